"""Plain oracle of the FP8 non-routed path and the scored router, in numpy.

Codes are E4M3: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinity,
0x7F NaN, largest value 448. What the library defines as a step of FP32
(amax, scale, the product that is rounded to a code) is computed here in
numpy's float32; everything else in float64. Shares no code with csrc/.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
MAX = 448.0


def code_values() -> np.ndarray:
    """The value of each of the 256 codes (float64)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (c & 0x7F) == 0x7F else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 0x80 else v
    return out


_VALUES = code_values()
_POSITIVE = _VALUES[:0x7F]  # ascending, codes 0 .. 0x7E


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest code of each value, ties to the even code, saturating at +-448; NaN gives NaN."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.where(np.isnan(v), 0.0, np.abs(v)), MAX)
    hi = np.searchsorted(_POSITIVE, a)  # first code >= a
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(v), 0x7F, code) | np.where(np.signbit(v) & ~np.isnan(v), 0x80, 0)
    return code.astype(np.uint8)


def decode(codes: np.ndarray) -> np.ndarray:
    return _VALUES[np.asarray(codes)]


def nblocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def quantize(x: np.ndarray, block_rows: int, dtype=np.float32) -> tuple:
    """(codes, scales) of a matrix in block_rows x 128 blocks."""
    R, C = x.shape
    codes = np.zeros((R, C), np.uint8)
    scales = np.zeros((-(-R // block_rows), nblocks(C)), dtype)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            sl = (slice(i * block_rows, (i + 1) * block_rows), slice(j * BLOCK, (j + 1) * BLOCK))
            b = x[sl].astype(dtype)
            amax = np.max(np.abs(b))
            if not np.isfinite(amax):
                scales[i, j], codes[sl] = np.nan, 0x7F
                continue
            scales[i, j] = amax / dtype(MAX)
            if amax > 0:
                codes[sl] = encode(b * (dtype(1) / amax * dtype(MAX)))  # as PyTorch computes MAX / amax
    return codes, scales


def widen(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    R, C = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), block_rows, 0)[:R], BLOCK, 1)[:, :C]
    return decode(codes) * s


def matmul(xq, xs, wq, ws) -> np.ndarray:
    return widen(xq, xs, 1) @ widen(wq, ws, BLOCK).T


def shared_ffn(x, wg, sg, wu, su, wd, sd) -> dict:
    """y and what its error bounds need: h before rounding, and the sums of
    the products' magnitudes."""
    xq, xs = quantize(x, 1)
    xv = widen(xq, xs, 1)
    g, u = (xv @ widen(w, s, BLOCK).T for w, s in ((wg, sg), (wu, su)))
    ag, au = (np.abs(xv) @ np.abs(widen(w, s, BLOCK)).T for w, s in ((wg, sg), (wu, su)))
    h = g / (1.0 + np.exp(-g)) * u
    hq, hs = quantize(h, 1, np.float64)
    wdv = widen(wd, sd, BLOCK)
    hv = widen(hq, hs, 1)
    return {"y": hv @ wdv.T, "g": g, "u": u, "ag": ag, "au": au, "h": h, "hq": hq, "hs": hs,
            "ay": np.abs(hv) @ np.abs(wdv).T, "wd": wdv}


def route_scored(logits, k, score="softmax", n_groups=1, top_groups=1, group_rank="max", renorm=True, scale=1.0,
                 bias=None) -> tuple:
    """(ids, weights, bad tokens) token by token, by sorting."""
    l = np.asarray(logits).astype(np.float64)
    T, E = l.shape
    per = E // n_groups
    ids, w, bad = np.full((T, k), -1, np.int32), np.zeros((T, k)), 0
    for t in range(T):
        row = l[t]
        live = [e for e in range(E) if row[e] != -np.inf and (bias is None or bias[e] != -np.inf)]
        broken = np.isnan(row).any() or (row == np.inf).any() or (
            bias is not None and (np.isnan(bias).any() or (np.asarray(bias) == np.inf).any()))
        if broken or not live:
            bad += 1
            continue
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-row))
        else:
            s = np.exp(row - row.max())
            s = s / s.sum()
        biased = s if bias is None else s + np.asarray(bias, np.float64)
        v = row if bias is None else biased
        groups = []
        for g in range(n_groups):
            mem = [e for e in live if e // per == g]
            if not mem:
                worth = -np.inf
            elif group_rank == "max" or per == 1:
                worth = max(v[e] for e in mem)
            else:
                worth = sum(sorted((biased[e] for e in mem), reverse=True)[:2])
            groups.append((-worth, g))
        kept = {g for _, g in sorted(groups)[:top_groups]}
        order = sorted((e for e in live if e // per in kept), key=lambda e: (-v[e], e))[:k]
        ids[t, :len(order)] = order
        sel = s[order]
        w[t, :len(order)] = (sel / (sel.sum() + 1e-20) if renorm else sel) * scale
    return ids, w, bad


def closest_call(logits, k, score="softmax", n_groups=1, top_groups=1, group_rank="max", bias=None, **_) -> np.ndarray:
    """Per token, the smallest gap between two computed values whose order
    decides the result: below FP32's rounding either order is right."""
    l = np.asarray(logits).astype(np.float64)
    T, E = l.shape
    per = E // n_groups
    gap = np.full(T, np.inf)
    for t in range(T):
        row = l[t]
        with np.errstate(invalid="ignore"):
            s = 1.0 / (1.0 + np.exp(-row)) if score == "sigmoid" else np.exp(row - row.max())
            if score != "sigmoid":
                s = s / s.sum()
        b = s if bias is None else s + np.asarray(bias, np.float64)
        b = np.where(row == -np.inf, -np.inf, b)
        kept = range(n_groups)
        if n_groups > 1 and top_groups < n_groups:
            best = np.sort(b.reshape(n_groups, per), 1)[:, ::-1]
            if group_rank == "top2" and per > 1:
                worth = best[:, 0] + np.where(np.isfinite(best[:, 1]), best[:, 1], 0.0)
            else:
                worth = best[:, 0]
            order = np.argsort(-worth, kind="stable")
            kept = order[:top_groups]
            d = worth[order[top_groups - 1]] - worth[order[top_groups]]
            if (bias is not None or group_rank == "top2") and np.isfinite(d):
                gap[t] = min(gap[t], d)
        if bias is not None:
            c = np.sort(np.concatenate([b[g * per:(g + 1) * per] for g in kept]))[::-1][:k + 1]
            c = c[np.isfinite(c)]
            if len(c) > 1:
                gap[t] = min(gap[t], (c[:-1] - c[1:]).min())
    return gap
