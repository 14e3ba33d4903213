"""The paged 8-bit cache without a GPU: argument checks of the C entry points
(made on the host before anything is launched), workspace sizes, the binding's
own checks, and pins of the oracle's e4m3."""
import ctypes

import numpy as np
import pytest
import torch

import attention_decode_b200 as nsnq
from attention_decode_b200 import build as nbuild
from oracle import paged as OP

FAKE = 0x10000  # a 128-byte aligned non-null address: validation never dereferences it
OTHER = 0x20000


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return nsnq.load()


def _cache(**kw):
    a = dict(k=FAKE, v=OTHER, ks=FAKE, vs=OTHER, pages=10, page=16, heads=2, status=None)
    a.update(kw)
    return nsnq._PagedCache(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page"], a["heads"], a["status"])


def _append(lib, **kw):
    a = dict(k=FAKE, v=OTHER, q=None, qo=None, dt=nsnq.NSNQ_BF16, n=4, kt=256, kh=128, vt=256, vh=128, qt=512,
             qh=128, cu=FAKE, lens=FAKE, B=2, Hq=4, Hkv=2, D=128, base=10000.0, cache={}, table=FAKE,
             cols=3, stride=3)
    a.update(kw)
    return lib.nsnq_paged_append(a["k"], a["v"], a["q"], a["qo"], a["dt"], a["n"], a["kt"], a["kh"], a["vt"],
                                 a["vh"], a["qt"], a["qh"], a["cu"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["D"],
                                 a["base"], _cache(**a["cache"]), a["table"], a["cols"], a["stride"], None)


def _attn(lib, **kw):
    a = dict(q=FAKE, qd=nsnq.NSNQ_BF16, n=4, qt=512, qh=128, cu=FAKE, mr=3, lens=FAKE, B=2, Hq=4, Hkv=2, D=128,
             cache={}, table=FAKE, cols=3, stride=3, window=0, sinks=0, scale=0.0, out=FAKE,
             od=nsnq.NSNQ_BF16, ws=FAKE, wsb=0)
    a.update(kw)
    return lib.nsnq_paged_attn(a["q"], a["qd"], a["n"], a["qt"], a["qh"], a["cu"], a["mr"], a["lens"], a["B"],
                               a["Hq"], a["Hkv"], a["D"], _cache(**a["cache"]), a["table"], a["cols"],
                               a["stride"], a["window"], a["sinks"], a["scale"], a["out"], a["od"], a["ws"], a["wsb"], None)


BOTH = [
    (dict(D=64), nsnq.NSNQ_ERR_UNSUPPORTED, b"D = 64"),
    (dict(B=-1), nsnq.NSNQ_ERR_INVALID_ARG, b"B"),
    (dict(n=-1), nsnq.NSNQ_ERR_INVALID_ARG, b"n_rows"),
    (dict(B=65536), nsnq.NSNQ_ERR_UNSUPPORTED, b"65535"),
    (dict(n=1 << 30), nsnq.NSNQ_ERR_UNSUPPORTED, b"2^31"),
    (dict(cu=None), nsnq.NSNQ_ERR_INVALID_ARG, b"cu_rows"),
    (dict(cache=dict(page=48)), nsnq.NSNQ_ERR_UNSUPPORTED, b"page_size"),
    (dict(cache=dict(page=256)), nsnq.NSNQ_ERR_UNSUPPORTED, b"page_size"),
    (dict(cache=dict(heads=3)), nsnq.NSNQ_ERR_INVALID_ARG, b"heads"),
    (dict(cache=dict(pages=-1)), nsnq.NSNQ_ERR_INVALID_ARG, b"num_pages"),
    (dict(cache=dict(pages=0)), nsnq.NSNQ_ERR_INVALID_ARG, b"num_pages"),
    (dict(cache=dict(pages=1 << 30)), nsnq.NSNQ_ERR_UNSUPPORTED, b"num_pages"),
    (dict(cache=dict(k=None)), nsnq.NSNQ_ERR_INVALID_ARG, b"NULL"),
    (dict(cache=dict(vs=None)), nsnq.NSNQ_ERR_INVALID_ARG, b"NULL"),
    (dict(cache=dict(v=OTHER + 16)), nsnq.NSNQ_ERR_INVALID_ARG, b"128-byte"),
    (dict(cache=dict(v=FAKE)), nsnq.NSNQ_ERR_INVALID_ARG, b"share"),
    (dict(cache=dict(vs=FAKE)), nsnq.NSNQ_ERR_INVALID_ARG, b"share"),
    (dict(cache=dict(ks=FAKE + 2)), nsnq.NSNQ_ERR_INVALID_ARG, b"4-byte"),
    (dict(cache=dict(status=FAKE + 1)), nsnq.NSNQ_ERR_INVALID_ARG, b"4-byte"),
    (dict(lens=None), nsnq.NSNQ_ERR_INVALID_ARG, b"seq_lens"),
    (dict(table=None), nsnq.NSNQ_ERR_INVALID_ARG, b"page_table"),
    (dict(table=FAKE + 1), nsnq.NSNQ_ERR_INVALID_ARG, b"4-byte"),
    (dict(cols=-1), nsnq.NSNQ_ERR_INVALID_ARG, b"table_cols"),
    (dict(stride=2), nsnq.NSNQ_ERR_INVALID_ARG, b"table_stride"),
    (dict(Hkv=0), nsnq.NSNQ_ERR_INVALID_ARG, b"Hkv"),
]


@pytest.mark.parametrize("call", ["append", "attn"])
@pytest.mark.parametrize("change,status,text", BOTH)
def test_refusals_of_both(lib, call, change, status, text):
    got = (_append if call == "append" else _attn)(lib, **change)
    assert got == status and text in lib.nsnq_last_error(), lib.nsnq_last_error()


@pytest.mark.parametrize("change,status,text", [
    (dict(dt=7), nsnq.NSNQ_ERR_UNSUPPORTED, b"dtype"),
    (dict(base=0.5), nsnq.NSNQ_ERR_INVALID_ARG, b"rope_base"),
    (dict(base=float("nan")), nsnq.NSNQ_ERR_INVALID_ARG, b"rope_base"),
    (dict(base=float("inf")), nsnq.NSNQ_ERR_INVALID_ARG, b"rope_base"),
    (dict(k=None), nsnq.NSNQ_ERR_INVALID_ARG, b"k is NULL"),
    (dict(v=OTHER + 2), nsnq.NSNQ_ERR_INVALID_ARG, b"v and its strides"),
    (dict(kt=260), nsnq.NSNQ_ERR_INVALID_ARG, b"k and its strides"),
    (dict(vh=-128), nsnq.NSNQ_ERR_INVALID_ARG, b"v has a negative"),
    (dict(q=FAKE), nsnq.NSNQ_ERR_INVALID_ARG, b"q_out"),
    (dict(q=FAKE, qo=FAKE, qt=640), nsnq.NSNQ_ERR_INVALID_ARG, b"contiguous"),
    (dict(q=FAKE, qo=OTHER, Hq=3), nsnq.NSNQ_ERR_INVALID_ARG, b"multiple"),
])
def test_append_refusals(lib, change, status, text):
    assert _append(lib, **change) == status and text in lib.nsnq_last_error(), lib.nsnq_last_error()


@pytest.mark.parametrize("change,status,text", [
    (dict(qd=5), nsnq.NSNQ_ERR_UNSUPPORTED, b"dtype"),
    (dict(od=-1), nsnq.NSNQ_ERR_UNSUPPORTED, b"dtype"),
    (dict(Hq=5), nsnq.NSNQ_ERR_INVALID_ARG, b"multiple"),
    (dict(window=-1), nsnq.NSNQ_ERR_INVALID_ARG, b"window"),
    (dict(sinks=-2), nsnq.NSNQ_ERR_INVALID_ARG, b"sinks"),
    (dict(mr=-1), nsnq.NSNQ_ERR_INVALID_ARG, b"max_rows"),
    (dict(scale=float("nan")), nsnq.NSNQ_ERR_INVALID_ARG, b"softmax_scale"),
    (dict(q=None), nsnq.NSNQ_ERR_INVALID_ARG, b"q is NULL"),
    (dict(qh=4), nsnq.NSNQ_ERR_INVALID_ARG, b"q and its strides"),
    (dict(out=FAKE + 8), nsnq.NSNQ_ERR_INVALID_ARG, b"out"),
    (dict(ws=None), nsnq.NSNQ_ERR_WORKSPACE, b"workspace"),
    (dict(wsb=16), nsnq.NSNQ_ERR_WORKSPACE, b"workspace"),
    (dict(ws=FAKE + 64, wsb=1 << 40), nsnq.NSNQ_ERR_INVALID_ARG, b"256-byte"),
])
def test_attn_refusals(lib, change, status, text):
    assert _attn(lib, **change) == status and text in lib.nsnq_last_error(), lib.nsnq_last_error()


def test_nothing_to_do(lib):
    for change in (dict(n=0), dict(B=0)):
        assert _append(lib, **change) == nsnq.NSNQ_OK
        assert _attn(lib, **change) == nsnq.NSNQ_OK
    assert _attn(lib, mr=0) == nsnq.NSNQ_OK
    assert lib.nsnq_last_error() == b""


def test_workspace_sizes(lib):
    ws = lib.nsnq_paged_attn_workspace
    assert ws(4, 2, 4, 2, 128, 3) > 0 and ws(32768, 8, 64, 8, 128, 4096) > 0
    for bad in ((-1, 2, 4, 2, 128, 3), (4, -2, 4, 2, 128, 3), (4, 2, 5, 2, 128, 3), (4, 2, 4, 2, 64, 3),
                (4, 2, 4, 2, 128, -1), (1 << 30, 2, 4, 2, 128, 3), (4, 2, 4, 0, 128, 3)):
        assert ws(*bad) == 0, bad


def test_binding_rejects_cpu_and_wrong_tensors():
    pc = nsnq.PagedCache.empty(4, 2, 16, device="cpu")
    assert (pc.num_pages, pc.heads, pc.page_size) == (4, 2, 16)
    pc.check()  # nothing reported
    with pytest.raises(ValueError, match="CUDA"):
        pc._c()
    pc.status.fill_(nsnq.PAGED_BAD_PAGE)
    with pytest.raises(nsnq.NSNQError, match="page table"):
        pc.check()
    pc.check()  # cleared
    bad = nsnq.PagedCache(pc.k.view(torch.uint8), pc.v, pc.k_scales, pc.v_scales)
    with pytest.raises(TypeError, match="float8"):
        bad._c()
    with pytest.raises(TypeError, match="scales"):
        nsnq.PagedCache(pc.k, pc.v, pc.k_scales.double(), pc.v_scales)._c()
    with pytest.raises(ValueError):
        nsnq.PagedCache(pc.k[..., :64], pc.v[..., :64], pc.k_scales, pc.v_scales)._c()


def test_oracle_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(OP.VALUES, want)
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 100
    x = torch.cat((x, torch.tensor([0.0, -0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10])))
    x = x.clamp(-448, 448)
    np.testing.assert_array_equal(OP.e4m3_codes(x.double().numpy()),
                                  x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    np.testing.assert_array_equal(OP.e4m3_codes(np.array([1e9, -1e9, np.inf, -np.inf, np.nan])),
                                  [0x7E, 0xFE, 0x7E, 0xFE, 0x7F])


def test_oracle_cover():
    for e in (-126, -30, 0, 7, 119):
        assert OP.cover(448.0 * 2.0 ** e) == 2.0 ** e
        assert OP.cover(np.nextafter(448.0 * 2.0 ** e, np.inf)) == 2.0 ** (e + 1)
    assert OP.cover(0.0) == OP.cover(1e-300) == 2.0 ** -126
