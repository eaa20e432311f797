"""Paged e4m3 cache of the selection attention, float64 CPU oracle: the append
with its position rotation and page scales, and the attention of one query
token per sequence over the cache.

The operations are this library's own (the source pages end at whole
sequences); ``include/bsa.h`` states them.

TEST INFRASTRUCTURE: see the package docstring for who may import this.
"""

from __future__ import annotations

import numpy as np

from .nsa import LSE_EMPTY

E_MIN = -96  # exponent of the least page scale


def e4m3_values() -> np.ndarray:
    """Value of each of the 256 codes (NaN for 0x7f and 0xff)."""
    out = np.zeros(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[code] = np.nan if code & 127 == 127 else (-x if code & 128 else x)
    return out


VALUES = e4m3_values()


def e4m3_encode(x) -> np.ndarray:
    """Nearest code of each x, ties to the even code, past +-448 the largest."""
    x = np.asarray(x, dtype=np.float64)
    pos = VALUES[:127]  # 0 .. 448, ascending
    a = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), 448.0)
    hi = np.searchsorted(pos, a)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(hi % 2 == 0, hi, lo)))
    return np.where(np.isnan(x), 127, code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def rotate(x, pos, inv_freq, interleaved: bool) -> np.ndarray:
    """Rows x [..., n, D] at positions pos [n], in float64."""
    x = np.array(x, dtype=np.float64)
    r = 2 * len(inv_freq)
    j = np.arange(r // 2)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + r // 2)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang), np.sin(ang)
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = xa * c - xb * s, xa * s + xb * c
    return x


def least_scale(amax: float) -> float:
    """The least 2^e, e >= E_MIN, with amax <= 448 * 2^e."""
    e = E_MIN
    if amax > 0:
        m, x = np.frexp(amax)  # amax = m 2^x, 448 = 0.875 * 2^9
        e = max(E_MIN, int(x) - 9 + (1 if m > 0.875 else 0))
    return 2.0 ** e


def append(x, cache, scale, table, lens, new_lens):
    """Rows x [B, Hkv, n, D] (rotated already) behind `lens` tokens.

    cache [pages, Hkv, page, D] uint8 codes and scale [pages, Hkv]; returns
    new ``(codes, scales, exact)``, `exact` being the values before their
    rounding, over the page's scale (NaN where no new token lies).
    """
    codes, scale = np.array(cache), np.array(scale, dtype=np.float64)
    pages, Hkv, page, D = codes.shape
    exact = np.full(codes.shape, np.nan)
    for b in range(len(lens)):
        held, n = int(lens[b]), min(int(new_lens[b]), x.shape[2])
        if held < 0:
            continue
        for lp in range(held // page, table.shape[1]):
            t0, t1 = max(0, lp * page - held), min(n, (lp + 1) * page - held)
            pid = int(table[b, lp])
            if t0 >= t1 or not 0 <= pid < pages:
                continue
            r0 = held + t0 - lp * page
            for h in range(Hkv):
                new = x[b, h, t0:t1]
                fin = np.abs(new[np.isfinite(new)])
                amax = fin.max() if fin.size else 0.0
                s = scale[pid, h] if r0 else 0.0
                if not r0 or amax > 448 * s or s < 2.0 ** E_MIN:
                    grown = least_scale(amax)
                    codes[pid, h, :r0] = e4m3_encode(VALUES[codes[pid, h, :r0]] * (s / grown))
                    s = grown
                scale[pid, h] = s
                codes[pid, h, r0:r0 + t1 - t0] = e4m3_encode(new / s)
                exact[pid, h, r0:r0 + t1 - t0] = new / s
    return codes, scale, exact


def decode(q, k_cache, v_cache, k_scale, v_scale, table, lens, block_idx=None):
    """``(out [B, Hq, 1, D], lse [B, Hq, 1], sums)`` over uint8 codes.

    ``sums``: ``"p"`` = sum_t softmax_t |v_t| and ``"e"`` = the same weighted
    by how far an fp32 evaluation of the scores may be off, in rounding steps,
    ``"lse"`` the largest such number of a row, ``"v"`` = the sum of |v_t|.
    """
    q = np.asarray(q, dtype=np.float64)
    B, Hq, _, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, 1, D)), np.full((B, Hq, 1), LSE_EMPTY)
    sums = {n: np.zeros((B, Hq, 1, D)) for n in ("p", "e", "v")} | {"lse": np.zeros((B, Hq, 1))}
    for b in range(B):
        n = min(int(lens[b]), table.shape[1] * page)
        for h in range(Hkv):
            blocks = range(table.shape[1]) if block_idx is None else sorted({int(j) for j in block_idx[b, h, 0]})
            kk, vv = [], []
            for j in blocks:
                if j < 0 or j * page >= n or not 0 <= int(table[b, j]) < pages:
                    continue
                pid, m = int(table[b, j]), min(page, n - j * page)
                kk.append(VALUES[k_cache[pid, h, :m]] * float(k_scale[pid, h]))
                vv.append(VALUES[v_cache[pid, h, :m]] * float(v_scale[pid, h]))
            if not kk:
                continue
            kk, vv = np.concatenate(kk), np.concatenate(vv)
            x = q[b, h * G:(h + 1) * G, 0]
            s = (x @ kk.T) * D ** -0.5
            top = s.max(-1, keepdims=True)
            e = np.exp(s - top)
            p = e / e.sum(-1, keepdims=True)
            off = (D + 4) * D ** -0.5 * (np.abs(x) @ np.abs(kk).T) + 8
            hs = slice(h * G, (h + 1) * G)
            out[b, hs, 0] = p @ vv
            lse[b, hs, 0] = (top + np.log(e.sum(-1, keepdims=True)))[:, 0]
            sums["p"][b, hs, 0] = p @ np.abs(vv)
            sums["e"][b, hs, 0] = (p * (off + off.max(-1, keepdims=True))) @ np.abs(vv)
            sums["v"][b, hs, 0] = np.abs(vv).sum(0)
            sums["lse"][b, hs, 0] = off.max(-1)
    return out, lse, sums
