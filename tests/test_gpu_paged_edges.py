"""The paged 8-bit cache at the edges of what its calls allow, on the GPU: value
scales that lie far apart, rows and tokens that others do not see, queries with
one large channel, lengths and rows out of range, a caller's own scales, calls
in either order."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_decode_b200 as nsnq
from oracle import paged as OP
from test_gpu_paged import Batch, D, check_pool, dense64

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bounded(got, q, b, codes, scales, window=0, sinks=0, scale=1 / math.sqrt(D)):
    """Attention against fp64 with a bound that holds whatever the value scales
    are. Each weight is off by a relative e, as for test_gpu_paged.check_out: an
    output by 2 e sum p |v| / sum p. A term (weight times its page's value scale)
    is held in steps of 2^-23 of the row's largest such term, or finer, so half a
    step of it is lost at most, for each token, times a code of at most 448. Then
    half a step of the output type."""
    table, lens, cu = b.table.tolist(), b.lens, b.cu
    for s, length in enumerate(lens):
        for r in range(cu[s], cu[s + 1]):
            pos = length - (cu[s + 1] - r)
            seen = [t for t in range(pos + 1) if not window or t > pos - window or t < sinks]
            if not seen:
                assert (got[r] == 0).all()
                continue
            ids, at = np.array([table[s][t // b.page] for t in seen]), np.array([t % b.page for t in seen])
            for h in range(b.hq):
                g = h // (b.hq // b.hkv)
                kk = OP.VALUES[codes[0][ids, g, at]] * scales[0][ids, g].astype(np.float64)[:, None]
                vs = scales[1][ids, g].astype(np.float64)
                vv = OP.VALUES[codes[1][ids, g, at]] * vs[:, None]
                x = q[r, h].double().cpu().numpy()
                p = np.exp(kk @ x * scale - (kk @ x * scale).max())
                want, size = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
                reach = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
                e = 2.0 ** -18 + 160 * 2.0 ** -23 * reach + (2.0 ** -11 if got.dtype == torch.bfloat16 else 0.0)
                lost = len(seen) * 2.0 ** -24 * 448.0 * (p * vs).max() / p.sum()
                tol = torch.finfo(got.dtype).eps / 2 * np.abs(want) + 2 * e * size + lost
                err = np.abs(got[r, h].double().cpu().numpy() - want)
                assert (err <= tol).all(), (r, h, (err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 4, 2), (4, 4, 2), (16, 2, 2), (90, 4, 2), (40, 8, 2)])
def test_value_scales_far_apart(rows, hq, hkv, dtype):
    """Rows that see pages of tiny values only, rows behind them that see huge ones too, in either order."""
    for sign, seed in ((1, 1), (-1, 2), (0, 3)):
        b = Batch([rows, rows], [0, 60], hq, hkv, 16, dtype, seed=seed)
        slot = torch.arange(b.cols)[None, :, None].expand(2, b.cols, hkv)
        e = sign * (7 * slot - 30) if sign else torch.randint(-60, 30, slot.shape, generator=torch.Generator().manual_seed(rows))
        b.scales[1][b.table.long()] = torch.exp2(e.float())
        pc, (table, lens, cu) = b.cache(), b.dev()
        got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, out_dtype=dtype)
        bounded(got, b.q, b, *b.stored())


@pytest.mark.parametrize("rows", [1, 4, 60])
@pytest.mark.parametrize("small,large", [(-20, 10), (-60, 40), (-126, 0)])
def test_weight_on_a_page_of_small_values(rows, small, large):
    """Nearly all the weight on a token whose page holds far smaller values than the others' pages."""
    b = Batch([rows], [300], 4, 2, 16, seed=rows)
    b.q = b.q.abs() + 1
    b.scales[0].fill_(2.0 ** -9)
    b.scales[1].fill_(2.0 ** large)
    page = b.table[0, 5].long()
    b.codes[0][page, :, 3] = 0x7E                  # 448 / 512 in every channel
    b.scales[1][page] = 2.0 ** small
    b.scales[0][page] = 2.0 ** -9
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, softmax_scale=1.0)
    bounded(got, b.q, b, *b.stored(), scale=1.0)


@pytest.mark.parametrize("rows,hq,page,window,sinks", [(8, 4, 16, 0, 0), (3, 2, 16, 30, 2), (40, 4, 16, 0, 0),
                                                       (300, 2, 16, 0, 0), (200, 4, 32, 50, 3), (128, 2, 64, 0, 0)])
def test_unseen_tokens_change_no_bit(rows, hq, page, window, sinks):
    """Other keys, values and scales behind a row's position: the same bits, in both kernels."""
    before = page - 4
    b = Batch([rows], [before], hq, 2, page, seed=rows)
    for s in b.scales:
        s.copy_(torch.exp2(torch.randint(-9, -4, s.shape, generator=torch.Generator().manual_seed(rows)).float()))
    q, (table, lens, cu) = b.q.cuda(), b.dev()
    want = nsnq.nsnq_paged_attn(q, b.cache(), table, lens, cu, max_rows=rows, window=window, sinks=sinks)
    g = torch.Generator().manual_seed(rows + 1)
    for border in range(1, b.cols):                # pages from this one on are others
        for trial in range(3):
            pc, ids = b.cache(), b.table[0, border:].long().cuda()
            for c in (pc.k, pc.v):
                other = torch.randint(0, 256, (len(ids), *c.shape[1:]), generator=g).to(torch.uint8)
                c.view(torch.uint8)[ids] = other.cuda()
            for s, (lo, hi) in ((pc.k_scales, ((-9, 5), (-9, 0), (20, 60))[trial]), (pc.v_scales, ((20, 60), (-60, 60), (-9, 3))[trial])):
                s[ids] = torch.exp2(torch.randint(lo, hi, (len(ids), 2), generator=g).float()).cuda()
            got = nsnq.nsnq_paged_attn(q, pc, table, lens, cu, max_rows=rows, window=window, sinks=sinks)
            n = border * page - before
            assert torch.equal(got[:n], want[:n]), (border, trial)


ORDERS = """
import torch
import attention_decode_b200 as nsnq
dev = dict(device="cuda", dtype=torch.%(dtype)s)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
pc = nsnq.PagedCache.empty(4, 2, %(page)d)
k, v = torch.ones(9, 2, 128, **dev), torch.ones(9, 2, 128, **dev)
args = (pc, i32([[0, 1]]), i32([9]), i32([0, 9]))
graph = torch.cuda.CUDAGraph()
nsnq.nsnq_paged_append(k, v, *args, rope_base=%(first)s)
with torch.cuda.graph(graph):
    nsnq.nsnq_paged_append(k, v, *args, rope_base=%(second)s)
graph.replay()
cb = nsnq.Codebook(torch.randn(256, 8, device="cuda"))
cache = nsnq.Cache.empty(1, 1, 64, 8)
nsnq.nsnq_encode(torch.randn(1, 1, 64, 128, device="cuda"), cb, cache)
torch.cuda.synchronize()
assert cache.codes.any()
print("both orders fine")
"""


@pytest.mark.parametrize("page,dtype", [(16, "bfloat16"), (64, "bfloat16"), (64, "float32"), (128, "float32")])
@pytest.mark.parametrize("first,second", [("0.0", "10000.0"), ("10000.0", "0.0")])
def test_appends_with_and_without_rotation_in_either_order(first, second, page, dtype):
    """In a process of its own: what the first call sets up for a kernel is enough for the second, captured one,
    and no error is left for the next call of the library."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ORDERS % dict(first=first, second=second, page=page, dtype=dtype)
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "both orders fine" in run.stdout, run.stderr[-2000:]


@pytest.mark.parametrize("cu,lens", [([0, 10], [20]), ([-2, 6], [20]), ([-1000, 6, 8], [20, 9]), ([0, 3, 12], [9, 30]), ([0, 5, 3, 8], [9, 9, 9]),
                                     ([0, 1000000], [20]), ([0, 2, 40, 42], [7, 60, 8]), ([0, 2, 4, 6, 7, 20], [9, 20, 33, 17, 50])])
def test_rows_out_of_range_are_left_out(cu, lens):
    """A sequence whose rows the row tensors do not hold: nothing stored, zeros for the rows that there are."""
    B, n = len(lens), 8
    b = Batch([n] * B, [40] * B, 4, 2, 16, seed=B)
    pc, table = b.cache(), b.table.cuda()
    q, k, v = (x[:n].cuda() for x in (b.q, b.k, b.v))
    good = [s for s in range(B) if 0 <= cu[s] <= cu[s + 1] <= n]
    bad = [s for s in range(B) if s not in good]
    qr = torch.full_like(q, 7.0)
    nsnq.nsnq_paged_append(k, v, pc, table, i32(lens), i32(cu), q=q, q_out=qr, rope_base=b.base)
    assert int(pc.status) == nsnq.PAGED_BAD_LENGTH
    for s in bad:
        lo, hi = max(0, min(n, cu[s])), max(0, min(n, cu[s + 1]))
        if cu != [0, 5, 3, 8]:
            assert (qr[lo:hi] == 0).all()
    codes, scales = b.stored()
    for s in good:
        if cu != [0, 5, 3, 8]:                     # (overlapping rows: each sequence stores its own)
            OP.append(k.double().cpu().numpy(), v.double().cpu().numpy(), codes, scales, [b.table[s].tolist()], [lens[s]],
                      cu[s:s + 2], b.base)
    if cu != [0, 5, 3, 8]:
        check_pool(pc, codes, scales)
    pc = b.cache()
    got = nsnq.nsnq_paged_attn(q, pc, table, i32(lens), i32(cu), max_rows=100)
    assert int(pc.status) == nsnq.PAGED_BAD_LENGTH
    for s in bad:
        lo, hi = max(0, min(n, cu[s])), max(0, min(n, cu[s + 1]))
        if cu != [0, 5, 3, 8]:
            assert (got[lo:hi] == 0).all()
    for s in good:
        if cu != [0, 5, 3, 8]:
            alone = nsnq.nsnq_paged_attn(q[cu[s]:cu[s + 1]], pc, table[s:s + 1], i32(lens[s:s + 1]),
                                         i32([0, cu[s + 1] - cu[s]]), max_rows=100)
            assert (got[cu[s]:cu[s + 1]].float() - alone.float()).abs().max() <= 0.02 * alone.float().abs().max()


@pytest.mark.parametrize("rows", [1, 5, 40])
def test_nan_value_under_a_vanishing_weight(rows):
    """A NaN value counts wherever its row sees it, also where its weight is too small for fp32 in another
    CTA's part of the row."""
    b = Batch([rows], [20000 - rows], 4, 2, 128, seed=rows)
    b.q = b.q.abs() + 1
    b.codes[0][:] = 0
    b.codes[0][b.table[0, -1].long(), :, 31 - rows] = 0x7E     # a seen token of a large score
    b.codes[1][b.table[0, 0].long(), 1, 5, 77] = 0x7F
    b.scales[0].fill_(1.0)
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = torch.isnan(nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows)).cpu()
    want = torch.zeros(rows, 4, D, dtype=torch.bool)
    want[:, 2:, 77] = True
    assert torch.equal(got, want)


@pytest.mark.parametrize("hq,q_dtype,out_dtype", [(64, torch.float32, torch.float32), (32, torch.float32, torch.float32),
                                                  (64, torch.bfloat16, torch.float32), (32, torch.float32, torch.bfloat16)])
def test_fp32_weights_above_a_lagging_maximum(hq, q_dtype, out_dtype):
    """One token of the second tile takes nearly all the weight while the row's maximum lags behind it by 4 to 5
    bits: it keeps its 24 bits. Scores are one product each: off by 2^-21 of at most 4 (their scale's rounding, the
    product's and the exponent's), 2^-18 for exp2 and the sums, twice for the quotient. The other 200 tokens' weights
    are 2^-36 of the largest and less: what the six pieces, 4 bits and then 5 each from 2^2 or more down to 2^-34,
    hold of them is off by half that step each, 2^-37 of the largest, times a code of at most 448."""
    n = 24
    b = Batch([1] * n, [201] * n, hq, 8, 64, torch.float32, seed=hq)
    g = torch.Generator().manual_seed(hq)
    b.codes[0].zero_()
    b.scales[0].fill_(1.0)
    b.scales[1].fill_(1.0)
    for t, code in ((3, 0x00), (200, 0x38)):       # k . q = 0 and q_0; elsewhere -8 q_0
        for s in range(n):
            if t == 3:
                b.codes[0][b.table[s].long(), :, :, 0] = 0xD0
            b.codes[0][b.table[s, t // 64].long(), :, t % 64, 0] = code
    b.q.zero_()
    b.q[:, :, 0] = ((4.0 + torch.rand(n, hq, generator=g)) * math.log(2.0)).to(q_dtype).float()
    pc, (table, lens, _) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.to(q_dtype).cuda(), pc, table, lens, softmax_scale=1.0, out_dtype=out_dtype).double().cpu().numpy()
    codes, scales = b.stored()
    want, weight, _, _ = OP.attention(b.q.double().numpy(), codes, scales, b.table.tolist(), b.lens, list(range(n + 1)), 0, 0, 1.0)
    tol = 2 * (2.0 ** -18 + 4 * 2.0 ** -21) * weight + 200 * 2.0 ** -37 * 448 + torch.finfo(out_dtype).eps / 2 * np.abs(want)
    err = np.abs(got - want)
    assert (err <= tol).all(), ((err > tol).sum(), (err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("rows,dtype", [(1, torch.bfloat16), (3, torch.bfloat16), (50, torch.bfloat16), (50, torch.float32)])
@pytest.mark.parametrize("ratio", [2.0 ** 8, 2.0 ** 12])
def test_queries_with_one_large_channel(rows, dtype, ratio):
    """One query channel far above the others, where the keys are zero: the other channels make the scores. Their
    elements are within 2^13 of the largest, where a bf16 query is held exactly: no term for it in the bound."""
    b = Batch([rows], [200], 4, 2, 32, dtype, seed=rows)
    g = torch.Generator().manual_seed(rows)
    small = (1 + torch.rand(b.q.shape, generator=g)) * torch.where(torch.rand(b.q.shape, generator=g) < 0.5, -1.0, 1.0)
    b.q = (small / ratio).to(dtype)
    b.q[:, :, 64] = 1.9
    b.codes[0][..., 64] = 0
    b.scales[0].fill_(2.0 ** -8)
    scale = float(np.float32(0.5 * ratio))
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, softmax_scale=scale, out_dtype=dtype)
    bounded(got, b.q, b, *b.stored(), scale=scale)


@pytest.mark.parametrize("rows,page", [(1, 16), (2, 64), (9, 16), (40, 64)])
@pytest.mark.parametrize("scale", [1e-40, 2.0 ** -128, 2.0 ** -149, 3e38])
def test_append_under_extreme_scales_of_a_caller(rows, page, scale):
    """A page whose own scale is subnormal, or nearly the largest: zeros, tiny values and values that outgrow it."""
    for grow in (0.0, 1e-40, 1.0):
        b = Batch([rows, rows], [9, 3], 4, 2, page, torch.float32, seed=rows, base=0.0, grow=grow)
        b.scales = [torch.full_like(s, scale) for s in b.scales]
        pc, (table, lens, cu) = b.cache(), b.dev()
        nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, rope_base=b.base)
        codes, scales = b.stored()
        OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, b.base)
        check_pool(pc, codes, scales)


@pytest.mark.parametrize("rows", [1, 4, 70])
@pytest.mark.parametrize("scale", [1e-40, 2.0 ** -140, 2.0 ** -126])
def test_attention_under_extreme_scales_of_a_caller(rows, scale):
    """Value scales below fp32's normal range: finite results, within half a step of what the type holds there (fp32
    subnormals: 2^-150 for a part, its factor and the sum of each of up to 130 tokens). For bf16 a weight times a v
    scale below 2^-118 is held in steps of 2^-23 of that: off by 2^-142 each, times a code of at most 448."""
    b = Batch([rows], [60], 4, 2, 16, seed=rows)
    b.scales[1].fill_(scale)
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, out_dtype=torch.float32).double().cpu().numpy()
    codes, scales = b.stored()
    want, weight, reach, _ = OP.attention(b.q.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, 0, 0,
                                          1 / math.sqrt(D))
    e = 2.0 ** -18 + 160 * 2.0 ** -23 * reach[..., None]
    assert (np.abs(got - want) <= 2 * e * weight + 2.0 ** -24 * np.abs(want) + 200 * 2.0 ** -149).all()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows).double().cpu().numpy()
    assert (np.abs(got - want) <= 2 * (e + 2.0 ** -11) * weight + 2.0 ** -8 * np.abs(want) + 2.0 ** -133 + (60 + rows) * 448 * 2.0 ** -142).all()


def test_rows_of_a_sequence_without_max_rows():
    """cu_rows without max_rows: every row is attended, as with the largest count given."""
    b = Batch([6, 1, 30], [3, 70, 0], 4, 2, 16, seed=7)
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu)
    bounded(got, b.q, b, *b.stored())
    pc.check()


def test_a_cache_of_a_callers_own_tensors_reports():
    b = Batch([2, 2], [3, 70], 4, 2, 16, seed=8)
    full, (table, lens, cu) = b.cache(), b.dev()
    pc = nsnq.PagedCache(full.k, full.v, full.k_scales, full.v_scales)
    table[1, 4] = -1
    nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=2)
    with pytest.raises(nsnq.NSNQError, match="page table"):
        pc.check()
    lens[0] = 10 ** 6
    nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table.clamp(0), lens, cu)
    with pytest.raises(nsnq.NSNQError, match="lengths"):
        pc.check()


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_rows_left_out_hold_zeros(rows):
    """Rows of a sequence whose length is out of range: zeros in the queries and in the outputs of the calls."""
    b = Batch([rows] * 3, [3, 70, 40], 4, 2, 16, seed=rows)
    pc, (table, lens, cu) = b.cache(), b.dev()
    for bad in (10 ** 6, -1, rows - 1):
        lens[1] = bad
        qr = torch.full_like(b.q, 7.0).cuda()
        nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, q=b.q.cuda(), q_out=qr, rope_base=b.base)
        assert (qr[rows:2 * rows] == 0).all() and (qr[:rows] != 0).any() and (qr[2 * rows:] != 0).any()
        out = torch.full_like(b.q, 7.0).cuda()
        nsnq.nsnq_paged_attn(qr, pc, table, lens, cu, max_rows=rows, out=out)
        assert (out[rows:2 * rows] == 0).all() if bad != rows - 1 else (out[rows] == 0).all()


def test_rows_that_no_call_can_reach_hold_zeros():
    """An output made by the call, more rows in it than max_rows of every sequence can be: the rest is zero."""
    b = Batch([2, 2], [3, 70], 4, 2, 16, seed=9, spare_rows=60)
    pc, (table, lens, cu) = b.cache(), b.dev()
    for _ in range(3):
        torch.full((64, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")  # what the allocator may hand out again
        got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=2)
        assert (got[4:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,base,before", [(64, 10000.0, 0), (16, 500.0, 4000), (128, 1e6, 100000)])
def test_queries_are_rounded_once(page, base, before, dtype):
    """The rotation in fp64 and one rounding, whichever kernel the number of rows selects: half a step of the
    result's own binade, and 2^-30 (|a| + |b|) of an angle's fp64 error at the longest position here (2^17 * 2^-53
    twice over, and the sine's own). Many bf16 rows are rotated in fp32: 2^-21 (|a| + |b|) in its place."""
    rows, hq = 150, 12
    g = torch.Generator().manual_seed(page)
    q = torch.randn(rows, hq, D, generator=g).to(dtype)
    kv = torch.randn(rows, 1, D, generator=g).to(dtype).cuda()
    pages = -(-(before + rows) // page)
    pc = nsnq.PagedCache.empty(pages, 1, page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    got = nsnq.nsnq_paged_append(kv, kv, pc, table, i32([before + rows]), i32([0, rows]), q=q.cuda(), rope_base=base)
    each = torch.cat([nsnq.nsnq_paged_append(kv[i:i + 1], kv[i:i + 1], pc, table, i32([before + i + 1]),
                                             q=q[i:i + 1].cuda(), rope_base=base) for i in range(rows)])
    x = q.double().numpy()
    want = np.stack([OP.rotate(x[i], before + i, base) for i in range(rows)])
    size = np.abs(x[..., :64]) + np.abs(x[..., 64:])
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 1e-30)))) * torch.finfo(dtype).eps
    size = np.concatenate((size, size), -1)
    for out, extra in ((got, -21 if dtype == torch.bfloat16 else -30), (each, -30)):
        tol = step / 2 + 2.0 ** extra * size
        err = np.abs(out.double().cpu().numpy() - want)
        assert (err <= tol).all(), (np.argwhere(err > tol).shape, (err / tol).max())
    if dtype == torch.float32:
        assert (got != each).sum() <= got.numel() * 2.0 ** -18  # fp64 values on a border alone


def test_strides_of_a_single_row_or_head_do_not_count():
    """A dimension of one element is never stepped over: any stride, also that of an in-place single row."""
    b = Batch([1], [20], 4, 1, 16, seed=3)
    (table, lens, _), n = b.dev(), 6 * D + 3
    fused = torch.zeros(1, n, dtype=torch.bfloat16, device="cuda")
    fused[:, :6 * D] = torch.cat((b.q.flatten(1), b.k.flatten(1), b.v.flatten(1)), 1).cuda()
    q = fused.as_strided((1, 4, D), (n, D, 1))
    k, v = (fused.as_strided((1, 1, D), (n, 7, 1), at * D) for at in (4, 5))
    want = nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), b.cache(), table, lens, q=b.q.cuda(), rope_base=b.base)
    pc = b.cache()
    assert nsnq.nsnq_paged_append(k, v, pc, table, lens, q=q, q_out=q, rope_base=b.base) is q
    assert torch.equal(q, want)
    codes, scales = b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, b.base)
    check_pool(pc, codes, scales)
    got = nsnq.nsnq_paged_attn(q, pc, table, lens)
    assert torch.equal(got, nsnq.nsnq_paged_attn(want, pc, table, lens))


@pytest.mark.parametrize("rows,dtype", [(1, torch.bfloat16), (6, torch.bfloat16), (40, torch.bfloat16), (2, torch.float32)])
@pytest.mark.parametrize("exponent", [105, 119, -120])
def test_values_near_the_ends_of_the_range_over_many_ctas(rows, dtype, exponent):
    """Value scales near both ends of fp32, a context that many CTAs share: each part is of the values' own size."""
    b = Batch([rows], [30000], 4, 1, 128, dtype, seed=rows)
    b.scales[1].copy_(torch.exp2(exponent - torch.randint(0, 2, b.scales[1].shape, generator=torch.Generator().manual_seed(1))))
    b.codes[1] = (b.codes[1].int() % 0x70 + (b.codes[1].int() & 0x80)).to(torch.uint8)   # at most 240: finite sums of two
    pc, (table, lens, cu), q = b.cache(), b.dev(), b.q.cuda()
    got = nsnq.nsnq_paged_attn(q, pc, table, lens, cu, max_rows=rows, out_dtype=dtype).double()
    want, weight, reach, _ = dense64(q, b, pc, table, 0, 0, 1 / math.sqrt(D))
    e = 2.0 ** -18 + 160 * 2.0 ** -23 * reach + (2.0 ** -10 if dtype == torch.bfloat16 else 0.0)
    # besides, of each token half a step of 2^-23 of the largest product (at most 2^exponent), over a sum of weights of
    # at least 1, times a code; below 2^-118, of that; and fp32's own steps under its normal range
    lost = lens[0].item() * 2.0 ** -24 * 240 * max(2.0 ** exponent, 2.0 ** -118) if dtype == torch.bfloat16 else 0.0
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2 * e * weight + lost + 300 * 2.0 ** -149
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()
