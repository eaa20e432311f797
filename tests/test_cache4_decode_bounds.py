"""The single-token decode over every page of the 4-bit cache under bounds of each row's own length, narrow enough to
notice one stage of 128 tokens that is dropped or counted twice (CPU: that they are; GPU: the kernels within them).

In units of u = 2^-24 (half a step of fp32) and U = 4 u, for a sequence of n tokens; the largest magnitude that a score
can have is s = sum |q k| D^-1/2.

Weights.  A score and its exponential are off by what ``oracle.cache4.decode`` gives (``off``).  The reference moves by
4 binary places or more, at most 2 s log2(e) / 4 + 1 <= s + 1 times, each an exponential and a product: 5 u, 1.25 (s + 1)
U in all.

Their sum.  Of a range a warp has a fourth, so at most n / 4 + 32 tokens; a lane adds up two of each 16, twice at most,
one after the other, and the two to each other: n / 32 + 5 u.  Behind them 3 shuffles, 4 warps (an exponential, a product,
4 sums: 10), and either 8 blocks of a cluster (14) or the join: 5 for a part's exponential, at most 10 rounds of 5
shuffles, an exponential and a product and sum of what came before (12 each), 8 warps (14): 3 + 10 + 139 u, 38 U.  The
logarithm: 2 U, then 2^-23 of the result.

The products with the values.  A matrix product over 16 tokens counts as one operation of U of the magnitudes it adds up: n
/ 64 + 2; behind them as above.  Probabilities are f16: 2^-11 of themselves, or 2^-36 of the largest.  The quotient has
both errors, three roundings more (1 U), and is rounded to bf16.
"""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from oracle import cache4

U, STEP, STAGE = 2.0 ** -22, 2.0 ** -8, 128


def many(B, longest, seed):
    n = np.random.default_rng(seed).integers(0, longest + 1, B)
    n[::7], n[3::11] = 0, 1
    return [int(x) for x in n]


# B, Hq, Hkv, D, page, lengths, tokens for which the table has places behind the longest sequence's
CASES = {
    "one": (1, 4, 1, 128, 64, [40001], 0),
    "one of sixteen rows": (1, 16, 1, 128, 64, [40001], 0),
    "one of small pages": (1, 5, 1, 64, 16, [70017], 0),
    "one beside a short one": (2, 2, 2, 16, 16, [9000, 3], 0),
    "two kv heads": (2, 20, 2, 32, 32, [30000, 12345], 0),
    "long among a few": (4, 16, 1, 64, 64, [0, 20011, 9000, 777], 0),
    "long among many": (150, 5, 1, 64, 64, [20011, 9000] + many(148, 200, 1), 0),
    "many of nine rows": (90, 18, 2, 64, 64, many(88, 200, 2) + [20011, 9000], 0),
    "short tables": (40, 16, 1, 128, 128, [2048, 2047] + many(38, 1900, 3), 0),
    "clusters": (4, 8, 2, 64, 64, [4000, 3, 2500, 4096], 0),
    "short sequences of long tables": (9, 6, 3, 128, 32, many(9, 3000, 4), 40000),
    "as many ranges as pairs": (200, 6, 2, 32, 16, many(200, 1500, 5), 0),
}


def inputs(name):
    """q in bf16, the cache's four arrays and its table, the lengths."""
    B, Hq, Hkv, D, page, lens, room = CASES[name]
    r = np.random.default_rng(sum(map(ord, name)))
    places = max(1, -(-max(lens) // page))
    pages = B * places + 3
    codes = [r.integers(0, 256, (pages, Hkv, page, D // 2), dtype=np.uint8) for _ in range(2)]
    scales = [r.integers(0x10, 0x30, (pages, Hkv, page, D // 16), dtype=np.uint8) for _ in range(2)]  # 1/32 .. 1/2
    table = np.full((B, places + room // page), -1, dtype=np.int32)
    table[:, :places] = r.permutation(pages)[: B * places].reshape(B, places)
    q = torch.from_numpy(r.standard_normal((B, Hq, 1, D))).to(torch.bfloat16)
    return q, codes + scales + [table], lens


def bounds(q, cache, lens, out, lse, sums):
    """What a result and its logarithm may be off by, row by row."""
    n = np.maximum(np.array(lens, dtype=np.float64), 0.0)[:, None, None]
    D = q.shape[3]
    s = np.maximum(sums["lse"] - 8, 0.0) / (D + 5)  # off = (D + 5) s + 8
    moves = 1.25 * (s + 1)
    of_sum = n / 128 + 1.25 + 38
    of_products = n / 64 + 2 + 38
    tol_lse = U * (sums["lse"] + moves + of_sum + 2) + 2.0 ** -23 * np.abs(lse)
    rest = (2 * moves + of_sum + of_products + 1)[..., None]
    bound = (1 + STEP) * (2.0 ** -11 * sums["p"] + U * (sums["e"] + rest * sums["p"]) + 2.0 ** -36 * sums["v"])
    return bound + STEP * np.abs(out), tol_lse


def parts_of(q, cache, lens):
    """(b, head, weights [stages], their sum times values [stages, D]) of every query head whose sequence has two or more
    stages, the weights over the largest."""
    k, v, ks, vs, table = cache
    B, Hq, _, D = q.shape
    _, Hkv, page, _ = k.shape
    for b in range(B):
        if lens[b] <= STAGE:
            continue
        ids = table[b, : -(-lens[b] // page)]
        for h in range(Hkv):
            keys, values = (cache4.values(c[ids, h], s[ids, h]).reshape(-1, D)[: lens[b]] for c, s in ((k, ks), (v, vs)))
            for i in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                x = (keys @ q[b, i, 0]) * D ** -0.5
                e = np.exp(x - x.max())
                at = np.arange(0, lens[b], STAGE)
                yield b, i, np.add.reduceat(e, at), np.add.reduceat(e[:, None] * values, at)


@pytest.mark.parametrize("name", CASES)
def test_bounds_notice_a_stage_dropped_or_counted_twice(name):
    q, cache, lens = inputs(name)
    q = q.double().numpy()
    out, lse, sums = cache4.decode(q, *cache, lens)
    _, tol = bounds(q, cache, lens, out, lse, sums)
    seen = 0
    for b, i, w, wv in parts_of(q, cache, lens):
        share = (w / w.sum())[: lens[b] // STAGE]  # (the last one may hold a single token)
        assert np.allclose(wv.sum(0) / w.sum(), out[b, i, 0], rtol=0, atol=1e-9)
        # twice the bound, so that a result within it on the other side does not hide the change
        assert (np.minimum(-np.log1p(-share), np.log1p(share)) > 2 * tol[b, i, 0]).all(), (b, i)
        seen += len(share)
    assert seen > 2


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_decode_within_bounds_of_its_own_length(name):
    q, cache, lens = inputs(name)
    want, wl, sums = cache4.decode(q.double().numpy(), *cache, lens)
    bound, tol = bounds(q, cache, lens, want, wl, sums)
    on = [torch.from_numpy(c).cuda() for c in cache]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = bsa.nsa_cache4_decode(q.cuda(), *on, n, return_lse=True)
    again = bsa.nsa_cache4_decode(q.cuda(), *on, n, return_lse=True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # bit for bit
    worst = (np.abs(out.double().cpu().numpy() - want) / (bound + 1e-30)).max()
    assert worst <= 1, f"result: {worst:.2f} times its bound"
    worst = (np.abs(lse.double().cpu().numpy() - wl) / tol).max()
    assert worst <= 1, f"logarithm: {worst:.2f} times its bound"
