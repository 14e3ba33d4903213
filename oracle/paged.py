"""fp64 oracle of the paged 8-bit cache (numpy, one sequence, head and page at a
time): the append with its rotation and scales, and attention over the pages
with a sliding window and sinks. Test infrastructure only."""
from __future__ import annotations

import math

import numpy as np

D = 128


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; no infinity, NaN at 0x7f and 0xff."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = -v if c & 128 else v
    out[0x7F] = out[0xFF] = np.nan
    return out


VALUES = e4m3_values()
_POSITIVE = VALUES[:127]


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """Nearest code of each value: ties to the even code, held at +-448, NaN to 0x7f."""
    mag = np.abs(np.asarray(v, dtype=np.float64))
    up = np.clip(np.searchsorted(_POSITIVE, mag), 0, 126)
    low = np.maximum(up - 1, 0)
    with np.errstate(invalid="ignore"):
        du, dl = _POSITIVE[up] - mag, mag - _POSITIVE[low]
        code = np.where((mag >= 448) | (du < dl) | ((du == dl) & (up % 2 == 0)), up, low)
    code = np.where(np.signbit(v), code | 128, code)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def cover(amax: float) -> float:
    """The least power of two 2^e, e >= -126, with amax <= 448 * 2^e."""
    if not amax > 0:
        return 2.0 ** -126
    e = math.ceil(math.log2(amax / 448.0)) - 1
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def rotate(x: np.ndarray, pos: int, base: float) -> np.ndarray:
    """x [..., D] turned to token position pos: channels i and i + D/2 by pos * base^(-2i/D)."""
    if not base:
        return np.array(x, dtype=np.float64)
    ang = pos * base ** (-2.0 * np.arange(D // 2) / D)
    a, b = x[..., :D // 2].astype(np.float64), x[..., D // 2:].astype(np.float64)
    return np.concatenate((a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)), -1)


def append(k, v, codes, scales, table, lens, cu, base):
    """Store rows k, v [rows][H][D] (fp64) into codes = (k, v) uint8
    [pages][H][page][D] and scales = (k, v) [pages][H], in place."""
    page = codes[0].shape[2]
    for b, length in enumerate(lens):
        rows = cu[b + 1] - cu[b]
        start = length - rows
        for slot in range(start // page, -(-length // page) if rows else 0):
            lo, hi = max(start, slot * page), min(length, (slot + 1) * page)
            ident = table[b][slot]
            for which, x in enumerate((k, v)):
                for h in range(x.shape[1]):
                    new = np.stack([rotate(x[cu[b] + t - start, h], t, 0.0 if which else base)
                                    for t in range(lo, hi)])
                    mine = codes[which][ident, h]
                    top = np.abs(new[np.isfinite(new)]).max(initial=0.0)
                    scale = cover(top)
                    if lo > slot * page:
                        old = float(scales[which][ident, h])
                        if top <= 448.0 * old:
                            scale = old
                        else:
                            older = mine[:lo - slot * page]
                            mine[:lo - slot * page] = np.where(np.isnan(VALUES[older]), older,
                                                               e4m3_codes(VALUES[older] * (old / scale)))
                    mine[lo - slot * page:hi - slot * page] = e4m3_codes(new / scale)
                    scales[which][ident, h] = scale


def attention(q, codes, scales, table, lens, cu, window, sinks, scale):
    """fp64 attention of rows q [rows][Hq][D]: returns (out, weight, reach, spread),
    with weight = sum p |v| / sum p per channel (the size that errors of the
    weights act on), reach = max over visible tokens of scale * sum |q_i k_i|
    per row and head (the size that errors of the scores act on) and spread =
    visible tokens * max |v| (what weights lost to underflow act on)."""
    n, hq, _ = q.shape
    hkv, page = codes[0].shape[1], codes[0].shape[2]
    out, weight = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    reach, spread = np.zeros((n, hq)), np.zeros((n, hq))
    for b, length in enumerate(lens):
        for r in range(cu[b], cu[b + 1]):
            pos = length - (cu[b + 1] - r)
            seen = [t for t in range(pos + 1) if not window or t > pos - window or t < sinks]
            if not seen:
                continue
            ids, at = np.array([table[b][t // page] for t in seen]), np.array([t % page for t in seen])
            for h in range(hq):
                g = h // (hq // hkv)
                kk = VALUES[codes[0][ids, g, at]] * scales[0][ids, g].astype(np.float64)[:, None]
                vv = VALUES[codes[1][ids, g, at]] * scales[1][ids, g].astype(np.float64)[:, None]
                s = kk @ q[r, h] * scale
                p = np.exp(s - s.max())
                out[r, h] = p @ vv / p.sum()
                weight[r, h] = p @ np.abs(vv) / p.sum()
                reach[r, h] = (np.abs(kk) @ np.abs(q[r, h])).max() * abs(scale)
                spread[r, h] = len(seen) * np.abs(vv).max()
    return out, weight, reach, spread
