"""The paged 8-bit cache on the GPU against the fp64 oracle: appends (codes,
scales and untouched bytes equal), attention, and both together.

Tolerances. Codes and scales are decisions on the exact value: equal. A rotated
query is rounded once (half a step of its type) from a value that an fp32
evaluation gets within 4 roundings of |a| + |b| (cos, sin, two products): 2^-22
(|a| + |b|). Attention: with weights off by a relative e each, an output is off
by at most 2 e weight (numerator and denominator), weight = sum p |v| / sum p;
e = 2^-11 (a weight rounded to 11 bits; none for fp32 outputs) + 2^-18 (exp2, sums)
+ the score's error, a sum of 128 products in fp32 whose additions may truncate:
160 * 2^-23 of scale * sum |q k| (reach). Weights under 2^-24 of the largest may
vanish: tokens * 2^-24 * max |v| (spread). Then half a step of the output type."""
import math

import numpy as np
import pytest
import torch

import attention_decode_b200 as nsnq
from oracle import paged as OP

pytestmark = pytest.mark.gpu

D = 128


class Batch:
    """Sequences of `before` stored tokens and `new` rows over a shuffled pool.
    The pool's other bytes are random codes, the rest of the last pages NaN."""

    def __init__(self, new, before, hq, hkv, page, dtype=torch.bfloat16, seed=0, base=10000.0, spare_rows=0,
                 grow=1.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.before, self.hq, self.hkv, self.page, self.base = new, before, hq, hkv, page, base
        self.lens = [n + c for n, c in zip(new, before)]
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.cols = max(1, max(-(-t // page) for t in self.lens))
        pages = len(new) * self.cols + 2
        order = torch.randperm(pages, generator=g)[:len(new) * self.cols]
        self.table = order.view(len(new), self.cols).to(torch.int32)
        shape = (pages, hkv, page, D)
        self.codes = [torch.randint(0, 256, shape, generator=g).to(torch.uint8) for _ in range(2)]
        for c in self.codes:
            c[(c & 0x7F) == 0x7F] = 0x3A
        self.scales = [torch.exp2(torch.randint(-9, -4, shape[:2], generator=g).float()) for _ in range(2)]
        rows = self.cu[-1] + spare_rows
        self.k = (torch.randn(rows, hkv, D, generator=g) * grow).to(dtype)
        self.v = (torch.randn(rows, hkv, D, generator=g) * grow).to(dtype)
        self.q = torch.randn(rows, hq, D, generator=g).to(dtype)

    def tails(self, code):
        """Bytes behind each sequence's last token."""
        for b, t in enumerate(self.lens):
            if t % self.page:
                for c in self.codes:
                    c[self.table[b, t // self.page].long(), :, t % self.page:] = code

    def cache(self):
        codes = [c.cuda().view(torch.float8_e4m3fn) for c in self.codes]
        return nsnq.PagedCache(codes[0], codes[1], self.scales[0].cuda(), self.scales[1].cuda(),
                               torch.zeros(1, dtype=torch.int32, device="cuda"))

    def dev(self):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return self.table.cuda(), i32(self.lens), i32(self.cu)

    def stored(self):
        return ([c.numpy().copy() for c in self.codes], [s.numpy().copy() for s in self.scales])


def check_rotated(got, x, b):
    for s, n in enumerate(b.new):
        for i in range(n):
            r = b.cu[s] + i
            xr = x[r].double().numpy()
            want = OP.rotate(xr, b.before[s] + i, b.base)
            size = np.abs(xr[..., :64]) + np.abs(xr[..., 64:])
            tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0 ** -22 * np.concatenate((size, size), -1)
            assert (np.abs(got[r].double().cpu().numpy() - want) <= tol + 1e-40).all(), r


def check_pool(pc, codes, scales):
    for have, want in zip((pc.k, pc.v), codes):
        np.testing.assert_array_equal(have.view(torch.uint8).cpu().numpy(), want)
    for have, want in zip((pc.k_scales, pc.v_scales), scales):
        np.testing.assert_array_equal(have.cpu().numpy(), want)


def check_out(got, q, b, codes, scales, window=0, sinks=0, scale=1 / math.sqrt(D)):
    n = b.cu[-1]
    want, weight, reach, spread = OP.attention(q[:n].double().cpu().numpy(), codes, scales, b.table.tolist(), b.lens,
                                               b.cu, window, sinks, scale)
    e = 2.0 ** -18 + 160 * 2.0 ** -23 * reach + (2.0 ** -11 if got.dtype == torch.bfloat16 else 0.0)
    tol = (torch.finfo(got.dtype).eps / 2 * np.abs(want) + 2 * e[..., None] * weight
           + 2.0 ** -24 * spread[..., None])
    err = np.abs(got[:n].double().cpu().numpy() - want)
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:5], (err / np.maximum(tol, 1e-300)).max())


APPENDS = [
    # new rows, tokens before, Hq, Hkv, page
    ([1], [0], 4, 4, 16),
    ([1, 1, 1], [15, 16, 31], 8, 2, 16),
    ([5, 0, 33, 1, 0], [0, 7, 30, 127, 0], 6, 3, 16),
    ([40, 1, 131], [9, 63, 250], 4, 1, 64),
    ([200, 129], [100, 1], 8, 8, 128),
    ([64, 63, 65], [0, 1, 31], 2, 2, 32),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,before,hq,hkv,page", APPENDS)
def test_append(new, before, hq, hkv, page, dtype):
    b = Batch(new, before, hq, hkv, page, dtype, seed=len(new) + page, spare_rows=3)
    pc, (table, lens, cu) = b.cache(), b.dev()
    qo = torch.full((b.q.shape[0], hq, D), 7.0, dtype=dtype, device="cuda")
    got = nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, q=b.q.cuda(), q_out=qo, rope_base=b.base)
    codes, scales = b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, b.base)
    check_pool(pc, codes, scales)
    check_rotated(got, b.q, b)
    assert (got[b.cu[-1]:] == 7.0).all()  # rows behind the last sequence
    pc.check()


@pytest.mark.parametrize("page", [16, 128])
def test_append_many_sequences_without_cu(page):
    """One row per sequence, more sequences than a warp has lanes, no rotation, no queries."""
    before = [(17 * i) % 300 for i in range(77)]
    b = Batch([1] * 77, before, 2, 2, page, seed=3, base=0.0)
    pc, (table, lens, _) = b.cache(), b.dev()
    assert nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens) is None
    codes, scales = b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, 0.0)
    check_pool(pc, codes, scales)


@pytest.mark.parametrize("count", [33, 1025, 2050])
def test_append_few_rows_of_many_sequences(count):
    """0, 1, 2 and more rows a sequence, two on average: every row finds its sequence."""
    new = [(0, 1, 2, 0, 5, 1, 2)[i % 7] for i in range(count)]
    b = Batch(new, [(29 * i) % 47 for i in range(count)], 1, 1, 16, seed=count)
    assert sum(new) <= 2 * count
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, q=b.q.cuda(), rope_base=b.base)
    codes, scales = b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, b.base)
    check_pool(pc, codes, scales)
    check_rotated(got, b.q, b)
    pc.check()


@pytest.mark.parametrize("count,page", [(2, 16), (33, 16), (33, 128), (1100, 32)])
def test_append_rows_of_many_sequences(count, page):
    """More than two rows a sequence on average, some with none, some over three pages."""
    new = [(0, 7, 2, 2 * page + 1, 1, 0, page)[(i + 3) % 7] for i in range(count)]
    b = Batch(new, [(29 * i) % (page + 3) for i in range(count)], 1, 1, page, seed=count)
    assert sum(new) > 2 * count
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, q=b.q.cuda(), rope_base=b.base)
    codes, scales = b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, b.base)
    check_pool(pc, codes, scales)
    check_rotated(got, b.q, b)
    pc.check()


def test_append_strides_and_in_place_queries():
    """Rows of a fused projection [rows][(Hq + 2 Hkv) D], heads of a [heads][rows] layout, q rotated in place."""
    b = Batch([6, 11], [20, 3], 4, 2, 16, seed=5)
    n, hq, hkv = b.cu[-1], 4, 2
    fused = torch.cat((b.q.flatten(1), b.k.flatten(1), b.v.flatten(1)), 1).cuda()
    q = fused[:, :hq * D].view(n, hq, D)
    k = fused[:, hq * D:(hq + hkv) * D].view(n, hkv, D)
    v = b.v.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    (table, lens, cu), codes_scales = b.dev(), b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), *codes_scales, b.table.tolist(), b.lens, b.cu, b.base)
    pc = b.cache()
    got = nsnq.nsnq_paged_append(k, v, pc, table, lens, cu, q=q, rope_base=b.base)
    check_pool(pc, *codes_scales)
    check_rotated(got, b.q, b)
    pc, inplace = b.cache(), b.q.cuda()
    assert nsnq.nsnq_paged_append(k, v, pc, table, lens, cu, q=inplace, q_out=inplace, rope_base=b.base) is inplace
    assert torch.equal(inplace, got)


def test_scale_grows_token_by_token():
    """Ever larger tokens: the page's scale grows again and again, its older codes are rounded again."""
    page, steps = 16, 40
    g = torch.Generator().manual_seed(9)
    b = Batch([1, 1], [steps, steps + 5], 2, 2, page, torch.float32, seed=8)
    pc, (codes, scales) = b.cache(), b.stored()
    table = b.table.cuda()
    for i in range(steps):
        k = torch.randn(2, 2, D, generator=g) * 1.6 ** i * 1e-3
        v = torch.randn(2, 2, D, generator=g) * 0.7 ** i
        lens = [i + 1, i + 6]
        nsnq.nsnq_paged_append(k.cuda(), v.cuda(), pc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               rope_base=500.0)
        OP.append(k.double().numpy(), v.double().numpy(), codes, scales, b.table.tolist(), lens, [0, 1, 2], 500.0)
    check_pool(pc, codes, scales)


def test_append_zeros_infinities_nan_and_edges():
    b = Batch([20], [3], 2, 2, 16, torch.float32, seed=11, base=0.0)
    b.k[0] = 0.0
    b.k[1, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e-42])
    b.v[:13] = 0.0                               # the page of older tokens keeps its scale
    b.v[13:, 0] = 448.0 * 2.0 ** -3              # exactly at the border of a scale
    b.v[13:, 1] = float(np.nextafter(np.float32(448.0 * 2.0 ** -3), np.float32(1e9)))
    b.k[19, 1] = 3.0e38
    pc, (table, lens, cu) = b.cache(), b.dev()
    nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu)
    codes, scales = b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, 0.0)
    check_pool(pc, codes, scales)
    b = Batch([4], [0], 1, 1, 16, seed=12)
    b.k.zero_(), b.v.zero_()
    pc, (table, lens, cu) = b.cache(), b.dev()
    nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, rope_base=10000.0)
    assert float(pc.k_scales[b.table[0, 0].long()]) == 2.0 ** -126


@pytest.mark.parametrize("rows,page", [(1, 16), (2, 64), (40, 16), (90, 128)])
def test_append_under_a_callers_own_scales(rows, page):
    """Pages filled by another quantizer: scales that are no power of two are kept, or grow to one."""
    b = Batch([rows, rows], [9, 13], 4, 4, page, seed=rows + page, base=300.0)
    b.scales = [torch.where(torch.arange(s.numel()).view(s.shape) % 3 == 0, s * 0.37, torch.full_like(s, 0.3)) for s in b.scales]
    pc, (table, lens, cu) = b.cache(), b.dev()
    nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, rope_base=b.base)
    codes, scales = b.stored()
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, b.table.tolist(), b.lens, b.cu, b.base)
    check_pool(pc, codes, scales)


@pytest.mark.parametrize("rows", [1, 5, 150])
def test_attention_under_a_callers_own_scales(rows):
    b = Batch([rows, rows], [300, 77], 8, 2, 16, seed=rows)
    b.scales = [s * (0.7 + torch.rand(s.shape, generator=torch.Generator().manual_seed(rows))) for s in b.scales]
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows)
    check_out(got, b.q, b, *b.stored())


@pytest.mark.parametrize("new,before,hq,hkv", [([1], [600], 64, 1), ([1, 1], [40, 300], 33, 1), ([3, 1], [200, 9], 40, 2)])
def test_attention_many_heads_to_a_kv_head(new, before, hq, hkv):
    b = Batch(new, before, hq, hkv, 32, seed=hq)
    b.tails(0x7F)
    pc, (table, lens, cu) = b.cache(), b.dev()
    check_out(nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=max(new)), b.q, b, *b.stored())


def test_append_feeds_the_other_attention():
    """q rotated by the append is read by nsnq_attn_decode, whose kernel may start under its predecessor."""
    hq, hkv, T = 8, 2, 400
    b = Batch([1, 1], [20, 33], hq, hkv, 16, seed=98)
    pc, (table, lens, _) = b.cache(), b.dev()
    g = torch.Generator(device="cuda").manual_seed(99)
    cb = nsnq.Codebook(torch.randn(256, 8, generator=g, device="cuda"))
    caches = [nsnq.Cache.empty(2, hkv, T, 8) for _ in range(2)]
    for c in caches:
        nsnq.nsnq_encode(torch.randn(2, hkv, T, D, generator=g, device="cuda"), cb, c)
    seq = torch.full((2,), T, dtype=torch.int32, device="cuda")
    k, v, q = b.k.cuda(), b.v.cuda(), b.q.cuda()
    want = None
    for i in range(20):
        q_out = torch.zeros(2, hq, D, dtype=torch.bfloat16, device="cuda")
        nsnq.nsnq_paged_append(k, v, pc, table, lens, q=q, q_out=q_out, rope_base=b.base)
        if i == 0:
            torch.cuda.synchronize()
        got = nsnq.nsnq_attn_decode(q_out, caches[0], caches[1], cb, cb, seq, T, hkv)
        want = got if i == 0 else want
        assert torch.equal(got, want)


def test_append_reports_bad_pages_and_lengths():
    b = Batch([20, 3, 2, 4], [3, 40, 1, 7], 2, 2, 16, seed=13)
    b.table[0, 1] = -1
    b.table[1, 2] = 10 ** 9
    pc, (table, lens, cu) = b.cache(), b.dev()
    lens[2] = 16 * b.cols + 1   # longer than its table row
    lens[3] = 3                 # fewer tokens than rows
    nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, table, lens, cu, q=b.q.cuda(), rope_base=b.base)
    codes, scales = b.stored()
    keep = [c.copy() for c in codes], [s.copy() for s in scales]
    fixed = b.table.clone()
    fixed[0, 1], fixed[1, 2] = len(b.codes[0]) - 1, len(b.codes[0]) - 2  # stand-ins, put back after
    OP.append(b.k.double().numpy(), b.v.double().numpy(), codes, scales, fixed.tolist()[:2], b.lens[:2], b.cu[:3], b.base)
    for which in range(2):
        for p in (fixed[0, 1], fixed[1, 2]):
            codes[which][p], scales[which][p] = keep[0][which][p], keep[1][which][p]
    check_pool(pc, codes, scales)
    assert int(pc.status) == nsnq.PAGED_BAD_PAGE | nsnq.PAGED_BAD_LENGTH
    with pytest.raises(nsnq.NSNQError):
        pc.check()
    # rows that the row tensors do not have
    pc = b.cache()
    cu = torch.tensor([-5, 2, 1, 10 ** 6, 10 ** 6 + 1], dtype=torch.int32, device="cuda")
    nsnq.nsnq_paged_append(b.k.cuda(), b.v.cuda(), pc, b.dev()[0].clamp(0, 3), b.dev()[1], cu, q=b.q.cuda())
    assert int(pc.status) & nsnq.PAGED_BAD_LENGTH


ATTNS = [
    # new rows, tokens before, Hq, Hkv, page, window, sinks
    ([1], [0], 1, 1, 16, 0, 0),
    ([1], [600], 8, 2, 16, 0, 0),
    ([1, 1, 1, 1, 1], [0, 127, 128, 300, 77], 8, 2, 64, 0, 0),
    ([1, 1, 1], [500, 3, 260], 12, 2, 32, 100, 3),
    ([1, 1], [700, 431], 5, 1, 128, 1, 0),
    ([1, 1], [700, 431], 16, 2, 16, 129, 200),
    ([4, 0, 3, 1], [100, 55, 258, 0], 8, 4, 32, 0, 0),
    ([6, 6], [511, 124], 16, 2, 64, 60, 2),
    ([9, 2], [140, 600], 8, 1, 16, 0, 0),
    ([17, 300], [130, 0], 4, 1, 64, 0, 0),
    ([150, 1, 40], [77, 350, 0], 6, 2, 16, 0, 0),
    ([260, 90], [40, 200], 3, 3, 128, 50, 7),
    ([130], [250], 24, 3, 32, 128, 0),
    ([33], [0], 32, 1, 16, 0, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,before,hq,hkv,page,window,sinks", ATTNS)
def test_attention(new, before, hq, hkv, page, window, sinks, dtype):
    b = Batch(new, before, hq, hkv, page, dtype, seed=sum(new) + page, spare_rows=2)
    b.tails(0x7F)
    pc, (table, lens, cu) = b.cache(), b.dev()
    out = torch.full((b.q.shape[0], hq, D), 7.0, dtype=dtype, device="cuda")
    nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=max(new), window=window, sinks=sinks, out=out)
    check_out(out, b.q, b, *b.stored(), window=window, sinks=sinks)
    assert (out[b.cu[-1]:] == 7.0).all()
    pc.check()


def dense64(q, b, pc, table, window, sinks, scale):
    """fp64 attention on the device, a sequence and kv-head at a time: out, weight, reach, spread as the oracle's."""
    n, hq = b.cu[-1], b.hq
    out, weight = (torch.zeros(n, hq, D, dtype=torch.float64, device="cuda") for _ in range(2))
    reach, spread = (torch.zeros(n, hq, 1, dtype=torch.float64, device="cuda") for _ in range(2))
    for s, length in enumerate(b.lens):
        ids = table[s, :-(-length // b.page)].long()
        rows, pos = slice(b.cu[s], b.cu[s + 1]), torch.arange(b.before[s], length, device="cuda")[:, None, None]
        t = torch.arange(length, device="cuda")
        seen = (t <= pos) & ((t > pos - window) | (t < sinks) if window else True)
        for h in range(b.hkv):
            k, v = ((c.view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double() * e[ids, h].double()[:, None, None])
                    .reshape(-1, D)[:length] for c, e in ((pc.k, pc.k_scales), (pc.v, pc.v_scales)))
            g = slice(h * (hq // b.hkv), (h + 1) * (hq // b.hkv))
            qq = q[rows, g].double()
            p = torch.softmax((qq @ k.T * scale).masked_fill(~seen, -math.inf), -1)
            out[rows, g], weight[rows, g] = p @ v, p @ v.abs()
            reach[rows, g] = (qq.abs() @ k.abs().T * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
            spread[rows, g] = seen.sum(-1, keepdim=True) * v.abs().max()
    return out, weight, reach, spread


@pytest.mark.parametrize("new,before,hq,hkv,page,window,sinks", [
    # enough tiles that a CTA takes several units, with last units of one row, of half a unit and less
    ([280, 65, 129, 320], [1500, 3000, 700, 0], 32, 8, 16, 0, 0),
    ([280, 280, 33, 97], [2500, 1111, 4000, 3000], 8, 8, 128, 0, 0),
    ([350, 77, 513], [3000, 2000, 900], 20, 4, 64, 600, 9),
    ([2048], [0], 16, 4, 32, 0, 0),
    ([1] * 70, [(97 * i) % 3000 for i in range(70)], 24, 8, 64, 0, 0),
    ([4, 1, 3] * 12, [(531 * i) % 5000 for i in range(36)], 16, 4, 16, 1000, 130),
    ([8, 5] * 9, [(731 * i) % 4000 for i in range(18)], 32, 8, 32, 0, 0),
    ([2] * 5, [30000, 7, 12000, 20001, 1], 32, 8, 128, 0, 0),
])
def test_attention_many_units(new, before, hq, hkv, page, window, sinks):
    b = Batch(new, before, hq, hkv, page, seed=sum(new) + page)
    b.tails(0x7F)
    pc, (table, lens, cu), q = b.cache(), b.dev(), b.q.cuda()
    want, weight, reach, spread = dense64(q, b, pc, table, window, sinks, 1 / math.sqrt(D))
    e = 2.0 ** -18 + 160 * 2.0 ** -23 * reach + 2.0 ** -11
    tol = 2.0 ** -8 * want.abs() + 2 * e * weight + 2.0 ** -24 * spread
    for _ in range(3):
        got = nsnq.nsnq_paged_attn(q, pc, table, lens, cu, max_rows=max(new), window=window, sinks=sinks).double()
        err = (got - want).abs()
        assert (err <= tol).all(), (torch.nonzero(~(err <= tol))[:5], (err / tol).max())
    pc.check()


@pytest.mark.parametrize("rows", [1, 5, 140])
def test_attention_types_mixed_scale_given(rows):
    b = Batch([rows, rows], [90, 300], 4, 2, 16, seed=rows)
    pc, (table, lens, cu) = b.cache(), b.dev()
    for q, od in ((b.q, torch.float32), (b.q.float(), torch.bfloat16)):
        got = nsnq.nsnq_paged_attn(q.cuda(), pc, table, lens, cu, max_rows=rows, softmax_scale=0.02, out_dtype=od)
        assert got.dtype == od
        check_out(got, q, b, *b.stored(), scale=float(np.float32(0.02)))
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, softmax_scale=-0.02)
    check_out(got, b.q, b, *b.stored(), scale=float(np.float32(-0.02)))


@pytest.mark.parametrize("rows", [1, 6, 200])
def test_freed_pages_are_not_read(rows):
    """Behind a window's pages (and between sinks and window) the table may hold anything."""
    b = Batch([rows, rows], [700, 520], 8, 2, 16, seed=21)
    pc, (table, lens, cu) = b.cache(), b.dev()
    window, sinks = 65, 18
    want = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, window=window, sinks=sinks)
    for s, c in enumerate(b.before):
        first = (c + 1 - window) // 16
        table[s, 2:first] = torch.tensor([-1, 1 << 30], device="cuda").repeat(50)[:first - 2].to(torch.int32)
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, window=window, sinks=sinks)
    pc.check()
    assert torch.equal(got, want)
    check_out(got, b.q, b, *b.stored(), window=window, sinks=sinks)


@pytest.mark.parametrize("rows,window,sinks", [(1, 0, 0), (1, 40, 2), (5, 0, 0), (7, 40, 2), (150, 0, 0), (150, 40, 2)])
def test_nan_reaches_only_rows_that_see_it(rows, window, sinks):
    """NaN codes in keys and values of tokens that some rows see and others do not."""
    b = Batch([rows], [200], 4, 2, 32, seed=31)
    total = 200 + rows
    places = [total - 1, total - max(1, rows // 2), 200 - 39, 3]
    for i, t in enumerate(places):
        for which in range(2):
            b.codes[which][b.table[0, t // 32].long(), i % 2, t % 32, 5 + 30 * i] = 0x7F if which else 0xFF
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows, window=window, sinks=sinks)
    got = got.float().cpu()
    codes, scales = b.stored()
    clean = [np.where((c & 0x7F) == 0x7F, 0, c) for c in codes]
    clear = []
    for r in range(rows):
        pos = 200 + r
        for h in range(4):
            hit = any(t <= pos and (not window or t > pos - window or t < sinks) and i % 2 == h // 2
                      for i, t in enumerate(places))
            assert torch.isnan(got[r, h]).all() == hit if hit else torch.isfinite(got[r, h]).all(), (r, h)
            clear.append(not hit)
    want, weight, reach, spread = OP.attention(b.q.double().numpy(), clean, scales, b.table.tolist(), b.lens, b.cu,
                                               window, sinks, 1 / math.sqrt(D))
    clear = np.array(clear).reshape(rows, 4)
    e = 2.0 ** -18 + 160 * 2.0 ** -23 * reach + 2.0 ** -11
    tol = 2.0 ** -8 * np.abs(want) + 2 * e[..., None] * weight + 2.0 ** -24 * spread[..., None]
    assert (np.abs(got.double().numpy() - want) <= tol)[clear].all()


@pytest.mark.parametrize("rows", [1, 5, 150])
def test_nan_values_alone(rows):
    """NaN in one value channel: exactly that channel of the rows that see the token."""
    b = Batch([rows], [200], 4, 2, 32, seed=32)
    t = 200 + rows // 2
    b.codes[1][b.table[0, t // 32].long(), 1, t % 32, 77] = 0x7F
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = torch.isnan(nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows)).cpu()
    want = torch.zeros(rows, 4, D, dtype=torch.bool)
    want[rows // 2:, 2:, 77] = True
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [1, 4, 130])
def test_queries_with_nan_and_zero(rows):
    b = Batch([rows, rows], [60, 100], 4, 2, 16, seed=41)
    b.q[0, 1, 3] = float("nan")
    b.q[rows, 2] = 0.0
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows).cpu()
    assert torch.isnan(got[0, 1]).all()
    b.q[0, 1, 3] = 0.0
    ref = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows)
    check_out(ref, b.q, b, *b.stored())
    rest = torch.ones(2 * rows, 4, dtype=torch.bool)
    rest[0, 1] = False
    assert torch.equal(got[rest], ref.cpu()[rest])


@pytest.mark.parametrize("rows", [1, 3, 160])
def test_wide_scales_and_peaked_scores(rows):
    """Pages whose scales differ by 2^40, one token far above the others in score."""
    b = Batch([rows], [420], 6, 2, 16, seed=51)
    g = torch.Generator().manual_seed(52)
    b.scales[1] = torch.exp2(torch.randint(-30, 11, b.scales[1].shape, generator=g).float())
    b.codes[0][b.table[0, 3].long(), :, 5] = 0x7E
    b.q[:, :, :] = b.q.abs()
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=rows)
    check_out(got, b.q, b, *b.stored())


def test_small_weights_add_up():
    """One token 2^13 times as likely as each of 40000 others: together they carry most of the weight."""
    page, n = 128, 40000
    b = Batch([1], [n - 1], 2, 1, page, seed=61)
    for c in b.codes:
        c.fill_(0)
    b.codes[1][:] = 0x38                                    # values 1 * scale
    b.scales[0].fill_(1.0), b.scales[1].fill_(1.0)
    first = b.table[0, 0].long()
    b.codes[0][first, 0, 9, 0] = 0x38                       # k . q = q_0
    b.codes[1][first, 0, 9] = 0xB8                          # its value: -1
    b.q.zero_()
    b.q[0, :, 0] = 13.0 * math.log(2.0) * math.sqrt(D)
    top = float(b.q[0, 0, 0]) / math.sqrt(D)
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, out_dtype=torch.float32)
    want = (n - 1 - math.exp(top)) / (n - 1 + math.exp(top))
    assert (got.double().cpu() - want).abs().max() <= 2 * (2.0 ** -18 + 160 * 2.0 ** -23 * top) + n * 2.0 ** -24


def test_attention_reports_bad_pages_and_lengths():
    for rows in (1, 4, 140):
        b = Batch([rows] * 4, [200, 90, 100, 50], 4, 2, 32, seed=71)
        bad = b.table.clone()
        bad[0, 2], bad[1, 0] = -3, 1 << 29
        pc, (_, lens, cu) = b.cache(), b.dev()
        lens[2] = 32 * b.cols + 1
        got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, bad.cuda(), lens, cu, max_rows=rows)
        assert int(pc.status) == nsnq.PAGED_BAD_PAGE | nsnq.PAGED_BAD_LENGTH
        assert (got[2 * rows:3 * rows] == 0).all() and torch.isfinite(got).all()
        b2 = Batch([rows], [50], 4, 2, 32, seed=71)
        one = nsnq.nsnq_paged_attn(b.q[3 * rows:].cuda(), pc, b.table[3:].cuda(), lens[3:], cu[:2], max_rows=rows)
        tail = got[3 * rows:].float() - one.float()
        assert tail.abs().max() <= 0.02, b2.lens
    # more rows than tokens: the rows in front of the first token see nothing
    b = Batch([6], [0], 2, 1, 16, seed=72)
    pc, (table, lens, cu) = b.cache(), b.dev()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens - 2, cu, max_rows=6)
    assert (got[:2] == 0).all() and (got[2:].float().abs().sum((1, 2)) > 0).all()
    # rows past max_rows are left as they were
    out = torch.full((6, 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    pc = b.cache()
    nsnq.nsnq_paged_attn(b.q.cuda(), pc, table, lens, cu, max_rows=4, out=out)
    assert (out[4:] == 5.0).all() and int(pc.status) == nsnq.PAGED_BAD_LENGTH


def test_serving_run_prompt_chunk_decode_graph():
    """Prompts in two chunks, then decode steps replayed from a CUDA graph, on the caches they build."""
    hq, hkv, page, window, sinks = 8, 2, 32, 90, 4
    prompts, steps = [150, 37, 64], 5
    b = Batch([1] * 3, [p + steps - 1 for p in prompts], hq, hkv, page, seed=81)
    pc, (codes, scales) = b.cache(), b.stored()
    table = b.table.cuda()
    g = torch.Generator().manual_seed(82)
    draw = lambda n, h: torch.randn(n, h, D, generator=g).to(torch.bfloat16)  # noqa: E731
    step = Batch([1] * 3, prompts, hq, hkv, page, seed=81)
    step.table = b.table

    def oracle(k, v, lens, cu, q, got):
        OP.append(k.double().numpy(), v.double().numpy(), codes, scales, b.table.tolist(), lens, cu, b.base)
        check_pool(pc, codes, scales)
        step.lens, step.cu = lens, cu
        check_out(got, q, step, codes, scales, window=window, sinks=sinks)

    done = [0, 0, 0]
    for part in (0.6, 1.0):
        new = [int(p * part) - d for p, d in zip(prompts, done)]
        done = [d + n for d, n in zip(done, new)]
        cu = [0, new[0], new[0] + new[1], sum(new)]
        k, v, q = draw(sum(new), hkv), draw(sum(new), hkv), draw(sum(new), hq)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        qr = nsnq.nsnq_paged_append(k.cuda(), v.cuda(), pc, table, i32(done), i32(cu), q=q.cuda(), rope_base=b.base)
        got = nsnq.nsnq_paged_attn(qr, pc, table, i32(done), i32(cu), max_rows=max(new), window=window, sinks=sinks)
        oracle(k, v, done, cu, qr, got)
    k, v, q = (torch.zeros(3, h, D, dtype=torch.bfloat16, device="cuda") for h in (hkv, hkv, hq))
    lens = i32(done)
    ws = torch.empty(nsnq.nsnq_paged_attn_workspace(3, 3, hq, hkv, 1), dtype=torch.uint8, device="cuda")
    out, qr = torch.empty_like(q), torch.empty_like(q)

    def call():
        lens.add_(1)
        nsnq.nsnq_paged_append(k, v, pc, table, lens, q=q, q_out=qr, rope_base=b.base)
        nsnq.nsnq_paged_attn(qr, pc, table, lens, window=window, sinks=sinks, out=out, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(steps):
        kc, vc, qc = draw(3, hkv), draw(3, hkv), draw(3, hq)
        k.copy_(kc), v.copy_(vc), q.copy_(qc)
        graph.replay()
        torch.cuda.synchronize()
        done = [d + 1 for d in done]
        assert lens.tolist() == done
        oracle(kc, vc, done, [0, 1, 2, 3], qr, out)
    del graph


@pytest.mark.parametrize("rows", [1, 6, 200])
def test_two_streams_and_repeats(rows):
    """Calls at once on two streams (a workspace each, made by the call), and the same bits every time."""
    b = [Batch([rows] * 3, [900, 20, 411], 8, 2, 64, seed=91 + i) for i in range(2)]
    pcs, devs, qs = [x.cache() for x in b], [x.dev() for x in b], [x.q.cuda() for x in b]
    want = [nsnq.nsnq_paged_attn(qs[i], pcs[i], *devs[i], max_rows=rows) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            stream = streams[i] if i else streams[i].cuda_stream
            got[i].append(nsnq.nsnq_paged_attn(qs[i], pcs[i], *devs[i], max_rows=rows, stream=stream))
    torch.cuda.synchronize()
    for i in range(2):
        check_out(want[i], b[i].q, b[i], *b[i].stored())
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("rows", [1, 200])
def test_two_captured_calls_at_once(rows):
    """Two captured calls, their workspaces allocated in the capture, replayed on two streams at once."""
    b = [Batch([rows] * 3, [700, 33, 250], 8, 2, 32, seed=191 + i) for i in range(2)]
    sides = []
    for x in b:
        pc, dev, q = x.cache(), x.dev(), x.q.cuda()
        want = nsnq.nsnq_paged_attn(q, pc, *dev, max_rows=rows)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = nsnq.nsnq_paged_attn(q, pc, *dev, max_rows=rows)
        sides.append((graph, out, want, torch.cuda.Stream(), (pc, dev, q)))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, out, _, stream, _ in sides:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (graph, out, want, _, _), x in zip(sides, b):
        assert torch.equal(out, want)
        check_out(out, x.q, x, *x.stored())
    del sides


@pytest.mark.parametrize("rows", [1, 70])
def test_pool_of_more_than_32_bits(rows):
    """Pages whose bytes lie past 4 GiB: the same codes, scales and outputs as in a small pool."""
    b = Batch([rows, rows], [300, 0], 8, 8, 128, seed=195)
    pages = len(b.codes[0])
    small, (table, lens, cu) = b.cache(), b.dev()
    q, k, v = b.q.cuda(), b.k.cuda(), b.v.cuda()
    big = nsnq.PagedCache.empty(33000, 8, 128)
    far = 33000 - pages
    assert far * 8 * 128 * D > 1 << 32
    for x, y in ((big.k, small.k), (big.v, small.v)):
        x[far:].view(torch.uint8).copy_(y.view(torch.uint8))
    big.k_scales[far:], big.v_scales[far:] = small.k_scales, small.v_scales
    outs = []
    for pc, t in ((small, table), (big, table + far)):
        qr = nsnq.nsnq_paged_append(k, v, pc, t, lens, cu, q=q, rope_base=b.base)
        outs.append(nsnq.nsnq_paged_attn(qr, pc, t, lens, cu, max_rows=rows))
    assert torch.equal(*outs)
    for x, y in ((big.k, small.k), (big.v, small.v)):
        assert torch.equal(x[far:].view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(big.k_scales[far:], small.k_scales) and torch.equal(big.v_scales[far:], small.v_scales)


def test_shared_prefix_pages_and_table_stride():
    """Two sequences over the same prefix pages; the table a slice of a wider one."""
    b = Batch([1, 1], [127, 140], 8, 2, 32, seed=95)
    b.table[1, :4] = b.table[0, :4]
    pc, (_, lens, cu) = b.cache(), b.dev()
    wide = torch.full((2, b.cols + 9), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + b.cols] = b.table.cuda()
    got = nsnq.nsnq_paged_attn(b.q.cuda(), pc, wide[:, 2:2 + b.cols], lens)
    check_out(got, b.q, b, *b.stored())


def test_query_strides():
    b = Batch([5, 40], [30, 10], 4, 2, 16, seed=96)
    pc, (table, lens, cu) = b.cache(), b.dev()
    wide = torch.zeros(b.cu[-1], 7, 2 * D, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5, D:] = b.q.cuda()
    got = nsnq.nsnq_paged_attn(wide[:, 1:5, D:], pc, table, lens, cu, max_rows=40)
    check_out(got, b.q, b, *b.stored())


def test_binding_refusals():
    b = Batch([2, 1], [4, 5], 4, 2, 16, seed=97)
    pc, (table, lens, cu) = b.cache(), b.dev()
    k, v, q = b.k.cuda(), b.v.cuda(), b.q.cuda()
    with pytest.raises(TypeError, match="int32"):
        nsnq.nsnq_paged_append(k, v, pc, table.long(), lens, cu)
    with pytest.raises(ValueError, match="cu_rows"):
        nsnq.nsnq_paged_append(k, v, pc, table, lens)
    with pytest.raises(ValueError):
        nsnq.nsnq_paged_append(k, v[:2], pc, table, lens, cu)
    with pytest.raises(ValueError):
        nsnq.nsnq_paged_append(k, v, pc, table, lens.cpu(), cu)
    with pytest.raises(TypeError, match="dtype"):
        nsnq.nsnq_paged_append(k.half(), v.half(), pc, table, lens, cu)
    with pytest.raises(ValueError):
        nsnq.nsnq_paged_attn(q.cpu(), pc, table, lens, cu, max_rows=2)
    with pytest.raises(ValueError):
        nsnq.nsnq_paged_attn(q, pc, table[:1], lens, cu, max_rows=2)
    with pytest.raises(nsnq.NSNQError, match="workspace"):
        nsnq.nsnq_paged_attn(q, pc, table, lens, cu, max_rows=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(nsnq.NSNQError, match="heads"):
        nsnq.nsnq_paged_append(k[:, :1], v[:, :1], pc, table, lens, cu)
