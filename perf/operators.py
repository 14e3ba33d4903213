"""Timed cases of the paged 8-bit cache: the append of rotated keys and values,
and attention over the pages with an optional sliding window and sinks.

A pool of pages holds keys and values in e4m3, laid out [pages][kv heads][page][128],
with one power-of-two scale per page and kv head. A table row lists the pages of a
sequence; seq_lens counts its tokens with the new ones, whose rows lie packed,
[rows][heads][128], sequence after sequence (cu_rows).
"""
import math
import random

import torch

own = False
D = 128
BASE = 10000.0


def _case(name, op, seqs, rows, ctx, hq, hkv, page, ragged=False, window=0, sinks=0, dtype="bf16"):
    c = dict(op=op, seqs=seqs, rows=rows, ctx=ctx, hq=hq, hkv=hkv, page=page, ragged=ragged,
             window=window, sinks=sinks, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # One sequence's next token: a chat turn's decode step, where latency is all.
        _case("append-1", "append", 1, 1, 4090, 32, 8, 16),
        # A serving batch's next tokens; every sequence is inside some page.
        _case("append-64", "append", 64, 1, 8192, 64, 8, 64, ragged=True),
        # The prompts of a batch, stored whole.
        _case("append-8x4096", "append", 8, 4096, 0, 32, 8, 64),
        # Chunks of prompts of odd lengths that continue inside pages, fp32 activations.
        _case("append-5x777-f32", "append", 5, 777, 3001, 12, 4, 32, ragged=True, dtype="f32"),
        # A short chat: one query per step over a few pages.
        _case("attn-1x600", "attn", 1, 1, 599, 8, 2, 16),
        # The decode batch over 32k tokens of context each, four query heads to a kv head.
        _case("attn-16x32k", "attn", 16, 1, 32767, 32, 8, 64),
        # One long document.
        _case("attn-1x128k", "attn", 1, 1, 131071, 32, 8, 128),
        # A ragged serving batch of a model with a sliding window and sink tokens.
        _case("attn-64x8k-window", "attn", 64, 1, 8191, 64, 8, 64, ragged=True, window=2048, sinks=4),
        # Four drafted tokens per sequence checked at once.
        _case("attn-13x4-8k", "attn", 13, 4, 8000, 32, 8, 32, ragged=True),
        # A whole prompt's attention.
        _case("attn-prompt-8192", "attn", 1, 8192, 0, 32, 8, 64),
        # Chunks of prompts behind a long context.
        _case("attn-2x500-32k", "attn", 2, 500, 32000, 32, 8, 128, ragged=True),
        # Prompts of odd lengths under a sliding window with sinks, small pages.
        _case("attn-4x2047-window", "attn", 4, 2047, 300, 24, 8, 16, ragged=True, window=511, sinks=5),
    ]


def _span(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hkv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 6, 8))
    page = rng.choice((16, 32, 64, 128))
    kind = rng.choice(("append", "append", "decode", "decode", "chunk"))
    if kind == "append":
        seqs = _span(rng, 1, 64)
        rows = rng.choice((1, _span(rng, 1, 32768 // seqs)))
        return _case("", "append", seqs, rows, _span(rng, 1, 8192) - 1, hkv * group, hkv, page,
                     ragged=rng.random() < 0.7, dtype=rng.choice(("bf16", "bf16", "f32")))
    windowed = rng.random() < 0.5
    window = _span(rng, 1, 4096) if windowed else 0
    sinks = rng.choice((0, 1, 4, rng.randint(1, 200))) if windowed else 0
    if kind == "decode":
        seqs = _span(rng, 1, 64)
        ctx = _span(rng, 1, min(131072, 4194304 // (seqs * hkv)))
        return _case("", "attn", seqs, rng.choice((1, 1, rng.randint(1, 6))), ctx - 1, hkv * group, hkv,
                     page, ragged=rng.random() < 0.7, window=window, sinks=sinks)
    seqs = _span(rng, 1, 8)
    pairs = 1.0e9 / (hkv * group * seqs)  # (query, token) pairs of a sequence and head
    rows = _span(rng, 8, min(4096 // seqs, int(math.sqrt(pairs))))
    ctx = _span(rng, 1, min(16384 // seqs, max(1, int(pairs / rows) - rows)))
    return _case("", "attn", seqs, rows, ctx - 1, hkv * group, hkv, page, ragged=rng.random() < 0.7,
                 window=window, sinks=sinks)


def _lengths(case):
    """New rows and tokens before them, for each sequence: given by the case alone."""
    n, before = [case["rows"]] * case["seqs"], [case["ctx"]] * case["seqs"]
    if case["ragged"]:
        r = random.Random("%(seqs)d %(rows)d %(ctx)d %(page)d %(hkv)d" % case)
        n = [r.randint((case["rows"] + 1) // 2, case["rows"]) for _ in n]
        before = [r.randint(case["ctx"] // 2, case["ctx"]) for _ in before]
    return n, before


def _seen(case, n, before):
    """(query, token) pairs that a query head sees, and tokens that some query sees."""
    w, s, pairs, tokens = case["window"], case["sinks"], 0, 0
    for m, c in zip(n, before):
        if not w:
            pairs += m * c + m * (m + 1) // 2
            tokens += c + m
            continue
        pairs += sum(min(p + 1, w) + min(s, max(0, p + 1 - w)) for p in range(c, c + m))
        first = max(0, c + 1 - w)
        tokens += c + m - first + min(s, first)
    return pairs, tokens


def work(case):
    n, before = _lengths(case)
    rows, hq, hkv = sum(n), case["hq"], case["hkv"]
    if case["op"] == "append":
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * D * (2 * hkv * (esz + 1) + 2 * hq * esz), "flops": 3 * rows * D * (hq + hkv)}
    pairs, tokens = _seen(case, n, before)
    return {"bytes": tokens * hkv * (2 * D + 8 / case["page"]) + 4 * rows * hq * D, "flops": 4 * pairs * hq * D}


def _exponent(amax):
    """Least e with amax <= 448 * 2^e: amax = m * 2^k with m in [0.5, 1), and 448 = 0.875 * 2^9."""
    m, k = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m > 0.875, k - 8, k - 9), torch.full_like(k, -126))


def _e4m3(v):
    """Values rounded to the nearest e4m3 (ties to even, held at +-448)."""
    _, k = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(k - 4, min=-9))
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _tokens(gen, *shape):
    """Key-like activations: four outlier channels, a scale of its own for each token."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    x[..., ::64] += 8.0
    x[..., 32::64] -= 8.0
    return x * torch.exp(0.5 * torch.randn(*shape[:-1], 1, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, before = _lengths(case)
    seqs, hq, hkv, page = case["seqs"], case["hq"], case["hkv"], case["page"]
    cols = max(-(-(m + c) // page) for m, c in zip(n, before))
    pages = seqs * cols + 3
    # the pool as earlier steps left it: every page full, pages in any order
    pool, scales = [], []
    for i in range(2):
        codes = torch.empty(pages, hkv, page, D, dtype=torch.float8_e4m3fn, device="cuda")
        exps = torch.empty(pages, hkv, device="cuda")
        part = max(1, (1 << 27) // (hkv * page * D))
        for at in range(0, pages, part):
            shape = (min(part, pages - at), hkv, page, D)
            x = _tokens(gen, *shape) if i == 0 else torch.randn(*shape, generator=gen, device="cuda")
            e = _exponent(x.abs().amax((2, 3)))
            exps[at:at + part] = torch.ldexp(torch.ones_like(x[:, :, 0, 0]), e)
            codes[at:at + part] = torch.ldexp(x, -e[:, :, None, None]).to(torch.float8_e4m3fn)
        pool.append(codes)
        scales.append(exps)
    table = torch.randperm(pages, generator=gen, device="cuda")[:seqs * cols].to(torch.int32).view(seqs, cols)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    s = {"case": case, "lens": dev([m + c for m, c in zip(n, before)]), "cu": dev(cu), "rows": max(n),
         "table": table, "k_pages": pool[0], "v_pages": pool[1], "k_scales": scales[0], "v_scales": scales[1]}
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s["q"] = torch.randn(cu[-1], hq, D, generator=gen, device="cuda").to(dtype)
    if case["op"] == "append":
        s["k"] = _tokens(gen, cu[-1], hkv, D).to(dtype)
        s["v"] = torch.randn(cu[-1], hkv, D, generator=gen, device="cuda").to(dtype)
    else:
        # what lies behind a sequence's last token was never written: NaN codes
        for b, (m, c) in enumerate(zip(n, before)):
            if (m + c) % page:
                for t in pool:
                    t.view(torch.uint8)[table[b, (m + c) // page].long(), :, (m + c) % page:] = 0x7F
    if own:
        import attention_decode_b200 as nsnq
        s["cache"] = nsnq.PagedCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        if case["op"] == "attn":
            s["workspace"] = torch.empty(
                nsnq.nsnq_paged_attn_workspace(cu[-1], seqs, hq, hkv, s["rows"]), dtype=torch.uint8, device="cuda")
    return s


def _places(s):
    """Of each new row: its sequence, its position, and the number of its sequence's rows before it."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["q"].shape[0])
    at = torch.arange(s["q"].shape[0], device="cuda") - s["cu"].long()[seq]
    return seq, (s["lens"].long() - n)[seq] + at, at


def _rotated(x, pos):
    """Channels i and i + 64 turned by pos * BASE^(-i/64), in fp64."""
    freq = BASE ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    ang = pos.double()[:, None, None] * freq
    a, b = x[..., :D // 2].double(), x[..., D // 2:].double()
    return torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), -1)


def _at(pages, ids):
    return pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn)


def _append(s):
    page, (seq, pos, at) = s["case"]["page"], _places(s)
    n, lens = (s["cu"][1:] - s["cu"][:-1]).long(), s["lens"].long()
    start = lens - n
    dest, row = s["table"][seq, pos // page].long(), pos % page
    # the page that a sequence's first new row goes to keeps its older tokens
    old_page = torch.gather(s["table"], 1, (start // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    old_rows = torch.where(n > 0, start % page, 0)
    for x, pages, scales in ((_rotated(s["k"], pos), s["k_pages"], s["k_scales"]),
                             (s["v"].double(), s["v_pages"], s["v_scales"])):
        top = torch.zeros(scales.shape, dtype=torch.float64, device="cuda")
        top.index_reduce_(0, dest, x.abs().amax(-1), "amax")
        e = _exponent(top)
        had = _exponent(448.0 * scales[old_page].double())  # the scale's own exponent
        now = torch.where(old_rows[:, None] > 0, torch.maximum(e[old_page], had), e[old_page])
        e[old_page] = torch.where(n[:, None] > 0, now, e[old_page])
        older = _at(pages, old_page).double()
        kept = _e4m3(torch.ldexp(older, torch.clamp(had - now, -40, 0)[:, :, None, None]))
        mine = torch.arange(page, device="cuda")[None, :] < old_rows[:, None]
        kept = torch.where(mine[:, None, :, None], kept, older).to(torch.float8_e4m3fn)
        pages.view(torch.uint8)[old_page] = kept.view(torch.uint8)
        codes = _e4m3(torch.ldexp(x, -e[dest][..., None])).to(torch.float8_e4m3fn)
        pages.view(torch.uint8)[dest, :, row] = codes.view(torch.uint8)
        scales[dest] = torch.ldexp(torch.ones_like(top[dest]), e[dest]).float()
    return {"q": _rotated(s["q"], pos).to(s["q"].dtype), "k": s["k_pages"], "v": s["v_pages"],
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _attn(s):
    c, (seq, pos, at) = s["case"], _places(s)
    seqs, hq, hkv, width = c["seqs"], c["hq"], c["hkv"], s["rows"]
    length = s["table"].shape[1] * c["page"]
    t = torch.arange(length, device="cuda")
    there = (t[None, :] < s["lens"][:, None])[:, None, :, None]
    k, v = (torch.where(there, (_at(p, s["table"].long()).float() * e[s["table"].long()][..., None, None])
                        .permute(0, 2, 1, 3, 4).reshape(seqs, hkv, length, D), 0.0)
            for p, e in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
    q = torch.zeros(seqs, width, hq, D, device="cuda")
    q[seq, at] = s["q"].float()
    where = torch.full((seqs, width), -1, device="cuda")
    where[seq, at] = pos
    seen = t[None, None, :] <= where[..., None]
    if c["window"]:
        seen &= (t[None, None, :] > where[..., None] - c["window"]) | (t < c["sinks"])
    seen = seen[:, None, :, None, :]
    q = q.view(seqs, width, hkv, hq // hkv, D).transpose(1, 2).reshape(seqs, hkv, -1, D)
    score = (q @ k.transpose(2, 3)).view(seqs, hkv, width, hq // hkv, length) / math.sqrt(D)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(seqs, hkv, -1, length) @ v).view(seqs, hkv, width, hq // hkv, D)
    o = torch.where(total > 0, o / total, 0.0).transpose(1, 2).reshape(seqs, width, hq, D)
    return o[seq, at].to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import attention_decode_b200 as nsnq
        if s["case"]["op"] == "append":
            q = nsnq.nsnq_paged_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], cu_rows=s["cu"], q=s["q"],
                                       rope_base=BASE)
            return {"q": q, "k": s["cache"].k, "v": s["cache"].v, "k_scales": s["cache"].k_scales,
                    "v_scales": s["cache"].v_scales}
        return nsnq.nsnq_paged_attn(s["q"], s["cache"], s["table"], s["lens"], cu_rows=s["cu"], max_rows=s["rows"],
                                    window=s["case"]["window"], sinks=s["case"]["sinks"],
                                    workspace=s["workspace"])
    return _append(s) if s["case"]["op"] == "append" else _attn(s)


def _nearest_e4m3(v):
    """The nearest of the 253 e4m3 values, the one with an even code where two are as near."""
    codes = torch.arange(127, dtype=torch.uint8, device=v.device)
    grid = codes.view(torch.float8_e4m3fn).double()
    mag = v.abs().contiguous()
    hi = torch.searchsorted(grid, mag).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - mag, mag - grid[lo]
    take = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (mag >= 448), hi, lo)
    return torch.copysign(grid[take], v)


def _exact_append(s):
    page, lens, cu, hkv = s["case"]["page"], s["lens"].tolist(), s["cu"].tolist(), s["case"]["hkv"]
    table = s["table"].tolist()
    freq = torch.tensor([BASE ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")

    def turn(x, first):
        z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double())
        ang = torch.arange(first, first + x.shape[0], dtype=torch.float64, device="cuda")[:, None] * freq
        z = z * torch.polar(torch.ones_like(ang), ang)[:, None, :]
        return torch.cat((z.real, z.imag), -1)

    got = {"q": torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), "k": s["k_pages"].double(),
           "v": s["v_pages"].double(), "k_scales": s["k_scales"].double(), "v_scales": s["v_scales"].double()}
    bound = 448.0 * torch.ldexp(torch.ones(247, dtype=torch.float64, device="cuda"),
                                torch.arange(-126, 121, device="cuda"))
    for b, length in enumerate(lens):
        rows, first = cu[b + 1] - cu[b], length - (cu[b + 1] - cu[b])
        mine = slice(cu[b], cu[b + 1])
        got["q"][mine] = turn(s["q"][mine], first)
        for name, x in (("k", turn(s["k"][mine], first)), ("v", s["v"][mine].double())):
            lead = first % page
            total = lead + rows
            x = torch.cat((torch.zeros(lead, hkv, D, dtype=torch.float64, device="cuda"), x,
                           torch.zeros(-total % page, hkv, D, dtype=torch.float64, device="cuda")))
            x = x.view(-1, page, hkv, D).transpose(1, 2)  # [pages][kv heads][page][D]
            ids = table[b][first // page: first // page + x.shape[0]]
            at = torch.searchsorted(bound, x.abs().amax((2, 3)))
            scale = bound[at] / 448.0
            if lead:
                old = got[name + "_scales"][ids[0]]
                scale[0] = torch.maximum(scale[0], old)
                keep = got[name][ids[0], :, :lead] * (old / scale[0])[:, None, None]
            codes = _nearest_e4m3(x / scale[..., None, None])
            fresh = torch.arange(codes.shape[0] * page, device="cuda").view(-1, 1, page, 1)
            fresh = (fresh >= lead) & (fresh < total)
            now = torch.where(fresh, codes, got[name][ids])
            if lead:
                now[0, :, :lead] = _nearest_e4m3(keep)
            got[name][ids] = now
            got[name + "_scales"][ids] = scale
    return got


def _exact_attn(s):
    c, lens, cu = s["case"], s["lens"].tolist(), s["cu"].tolist()
    page, hq, hkv = c["page"], c["hq"], c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        ids = s["table"][b, :-(-length // page)].long()
        first = length - (cu[b + 1] - cu[b])
        for h in range(hkv):
            k, v = ((_at(p, ids)[:, h].double() * e[ids, h].double()[:, None, None]).reshape(-1, D)[:length]
                    for p, e in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for r in range(cu[b], cu[b + 1], 512):
                rows = slice(r, min(r + 512, cu[b + 1]))
                score = torch.einsum("rhd,td->rht", s["q"][rows, heads].double(), k) * D ** -0.5
                gap = (first + torch.arange(rows.start - cu[b], rows.stop - cu[b], device="cuda")[:, None, None]
                       - torch.arange(length, device="cuda"))
                hidden = gap < 0
                if c["window"]:
                    hidden = hidden | ((gap >= c["window"]) & (torch.arange(length, device="cuda") >= c["sinks"]))
                out[rows, heads] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)
