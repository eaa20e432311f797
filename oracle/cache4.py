"""Paged 4-bit cache of the selection attention, float64 CPU oracle: the codes
and scales of new rows, the values they stand for, and the attention of one
query token per sequence over them.

The operations are this library's own (the source pages end at whole
sequences); ``include/bsa.h`` states them.

TEST INFRASTRUCTURE: see the package docstring for who may import this.
"""

from __future__ import annotations

import numpy as np

from .cache import VALUES as E4M3
from .cache import e4m3_encode
from .nsa import LSE_EMPTY

GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def e2m1_encode(x) -> np.ndarray:
    """Nearest code of each x, ties to the even code, past +-6 the largest."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    dist = np.abs(a[..., None] - E2M1[:8])
    dist = np.where(dist == dist.min(-1, keepdims=True), np.arange(8) % 2, 2)  # the nearest; the even one of two
    return (dist.argmin(-1) | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def encode(x):
    """Rows x [..., D] (over the head's factor) as (codes [..., D], scale codes [..., D / 16])."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    sc = e4m3_encode(np.abs(g).max(-1) / 6.0)
    s = E4M3[sc][..., None]
    codes = e2m1_encode(np.where(s > 0, g / np.where(s > 0, s, 1.0), np.copysign(0.0, g)))
    return codes.reshape(x.shape), np.where(bad, 0x7F, sc).astype(np.uint8)


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def values(packed, scales, factor=1.0):
    """What codes [..., D / 2] and scales [..., D / 16] stand for."""
    c = E2M1[unpack(packed)]
    return c * np.repeat(E4M3[scales], GROUP, -1) * factor


def slots(table, pages, page, held, n):
    """(new token, pool page, slot) of the tokens behind `held` that have a place."""
    for t in range(n):
        pos = held + t
        if held < 0 or pos // page >= table.shape[0] or not 0 <= int(table[pos // page]) < pages:
            continue
        yield t, int(table[pos // page]), pos % page


def decode(q, k_cache, v_cache, k_scale, v_scale, table, lens, block_idx=None, k_factor=None, v_factor=None):
    """``(out [B, Hq, 1, D], lse [B, Hq, 1], sums)`` as ``oracle.cache.decode``."""
    q = np.asarray(q, dtype=np.float64)
    B, Hq, _, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    kf, vf = (np.ones(Hkv) if f is None else np.asarray(f, dtype=np.float64) for f in (k_factor, v_factor))
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
                kk.append(values(k_cache[pid, h, :m], k_scale[pid, h, :m], kf[h]))
                vv.append(values(v_cache[pid, h, :m], v_scale[pid, h, :m], vf[h]))
            if not kk:
                continue
            kk, vv = np.concatenate(kk), np.concatenate(vv)
            x = q[b, h * G:(h + 1) * G, 0]
            s = (x @ kk.T) * D ** -0.5
            top = s.max(-1, keepdims=True)
            e = np.exp(s - top)
            p = e / e.sum(-1, keepdims=True)
            off = (D + 5) * D ** -0.5 * (np.abs(x) @ np.abs(kk).T) + 8
            hs = slice(h * G, (h + 1) * G)
            out[b, hs, 0] = p @ vv
            lse[b, hs, 0] = (top + np.log(e.sum(-1, keepdims=True)))[:, 0]
            sums["p"][b, hs, 0] = p @ np.abs(vv)
            sums["e"][b, hs, 0] = (p * (off + off.max(-1, keepdims=True))) @ np.abs(vv)
            sums["v"][b, hs, 0] = np.abs(vv).sum(0)
            sums["lse"][b, hs, 0] = off.max(-1)
    return out, lse, sums
