"""GPU: the paged e4m3 cache -- append with rotation and page scales, and the
single-token selection attention over it -- against the float64 oracle.

Tolerances.  The rotated value of a pair (a, b) is off by at most 8 fp32
roundings of |a| + |b| (sine and cosine 2 each, argument 2, products and sum):
E = 2^-21 (|a| + |b|).  A code must be a nearest one for some value within E of
the exact one: its distance from the exact value exceeds the nearest code's by
at most 2 E.  Scales must be equal unless the maximum is within E of a border.

Decode: probabilities are rounded to f16 (2^-11 relative, and 2^-25 of the
largest where they are subnormal), the result to bf16 (2^-8); scores and sums
run in fp32 on the tensor cores, taken as U = 2^-22 an operation; the bound
is spelled out in ``check_decode``.
"""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from oracle import cache as ocache

pytestmark = pytest.mark.gpu
U, BF = 2.0 ** -22, 2.0 ** -8
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_tra_gb300 import build

    build.build()
    bsa.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert bsa.device_error() == 0


class Pool:
    """A cache whose every byte holds something (NaN codes among it), and a scattered table."""

    def __init__(self, B, Hkv, D, page, max_pages, seed=0, spare=3):
        r = np.random.default_rng(seed)
        self.pages = B * max_pages + spare
        self.k = torch.from_numpy(r.integers(0, 256, (self.pages, Hkv, page, D), dtype=np.uint8)).cuda()
        self.v = torch.from_numpy(r.integers(0, 256, (self.pages, Hkv, page, D), dtype=np.uint8)).cuda()
        self.ks = torch.exp2(torch.from_numpy(r.integers(-9, -4, (self.pages, Hkv))).float()).cuda()
        self.vs = torch.exp2(torch.from_numpy(r.integers(-9, -4, (self.pages, Hkv))).float()).cuda()
        self.table = torch.from_numpy(r.permutation(self.pages)[: B * max_pages].reshape(B, max_pages).astype(
            np.int32)).cuda()

    def clean(self):
        """No NaN codes (for pages whose tokens are read)."""
        for c in (self.k, self.v):
            c[(c & 127) == 127] = 0x30
        return self

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table

    def copy(self):
        return [t.cpu().numpy().copy() for t in (self.k, self.v, self.ks, self.vs, self.table)]


def freqs(rotary, base=10000.0):
    return (base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)).float().cuda() if rotary else None


def check_append(B, Hq, Hkv, n, D, page, lens, new=None, dtype=torch.bfloat16, rotary=None, interleaved=False, seed=0,
                 scale=1.0, pool=None, with_q=True, **kw):
    g = torch.Generator().manual_seed(seed)
    rotary = D if rotary is None else rotary
    k, v = ((torch.randn((B, Hkv, n, D), generator=g) * scale).to(dtype).cuda() for _ in range(2))
    q = torch.randn((B, Hq, n, D), generator=g).to(dtype).cuda() if with_q else None
    max_pages = max(-(-(x + n) // page) for x in lens)
    pool = pool or Pool(B, Hkv, D, page, max(1, max_pages), seed)
    before = pool.copy()
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nt = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    f = freqs(rotary)
    got = bsa.nsa_cache_append(k, v, *pool.args(), lt, new_lens=nt, inv_freq=f, interleaved=interleaved, q=q, **kw)
    torch.cuda.synchronize()
    news = [n] * B if new is None else new
    fr = f.double().cpu().numpy() if rotary else np.zeros(0)

    def turned(x):
        x = x.double().cpu().numpy()
        return np.stack([ocache.rotate(x[b], lens[b] + np.arange(n), fr, interleaved) for b in range(B)])

    for x, c0, s0, c1, s1 in ((turned(k), before[0], before[2], pool.k, pool.ks),
                              (v.double().cpu().numpy(), before[1], before[3], pool.v, pool.vs)):
        codes, scales, exact = ocache.append(x, c0, s0, before[4], lens, news)
        assert np.array_equal(s1.double().cpu().numpy(), scales)
        c1 = c1.cpu().numpy()
        old = np.isnan(exact)
        assert np.array_equal(c1[old], codes[old])  # held, rescaled and untouched codes
        a = ocache.VALUES[c1[~old]]
        near = np.abs(ocache.VALUES[codes[~old]] - exact[~old])
        tol = 2 * 2.0 ** -21 * 2 * 448  # |a| + |b| <= 2 * 448 scales
        assert (np.abs(a - exact[~old]) <= near + tol * (c1[~old] != codes[~old])).all()
        assert (c1[~old] != codes[~old]).mean() <= 1e-3 or old.all()
    if with_q:
        want = turned(q)
        for b in range(B):
            m = max(0, min(news[b], n))
            x, w = got[b, :, :m].double().cpu().numpy(), want[b, :, :m]
            eps = BF if dtype == torch.bfloat16 else 2.0 ** -24
            assert (np.abs(x - w) <= eps * np.abs(w) + 2.0 ** -20 * float(q[b].abs().max())).all()
    return pool, got


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_shapes(D, page):
    check_append(2, 4, 2, 2 * page + 3, D, page, [5, page], seed=D + page)
    check_append(3, 6, 2, 1, D, page, [0, page - 1, 3 * page], seed=D + page + 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 48, 64])
def test_append_rotations(dtype, interleaved, rotary):
    check_append(2, 9, 3, 37, 64, 32, [0, 70], dtype=dtype, interleaved=interleaved, rotary=rotary, seed=rotary)


def test_append_ragged_batch_and_lengths_zero():
    check_append(5, 4, 2, 70, 32, 32, [0, 31, 32, 100, 7], new=[70, 0, 1, 33, 69], seed=3)
    check_append(2, 2, 2, 9, 64, 16, [4, 0], new=[-3, 100], seed=4)


def test_append_without_queries_and_without_rotation():
    check_append(1, 2, 2, 20, 64, 64, [50], rotary=0, with_q=False)


def test_append_far_positions():
    """Angles of positions near 2^30, where an fp32 product would be off by whole turns."""
    page, far = 64, (1 << 30) + 12345
    lens, B, Hkv, D = [far], 1, 1, 64
    pool = Pool(B, Hkv, D, page, 1, seed=8)
    # only the queries: the table has no page there, so nothing is written
    before = pool.copy()
    q = torch.randn((1, 4, 3, D), generator=torch.Generator().manual_seed(2)).cuda()
    k = torch.zeros((1, 1, 3, D), device="cuda")
    f = freqs(D)
    got = bsa.nsa_cache_append(k, k, *pool.args(), torch.tensor(lens, device="cuda"), inv_freq=f, q=q)
    want = ocache.rotate(q[0].double().cpu().numpy(), far + np.arange(3), f.double().cpu().numpy(), False)
    # float64's own product of 2^30 and a frequency is exact to 2^-22 of a radian
    assert np.abs(got[0].double().cpu().numpy() - want).max() <= 2.0 ** -19 * float(q.abs().max())
    for a, b in zip(before, pool.copy()):
        assert np.array_equal(a, b)


def test_append_token_by_token_grows_the_scale():
    """Tokens of rising magnitude: each step's codes and scales are the oracle's."""
    B, Hkv, D, page = 2, 2, 32, 32
    pool = Pool(B, Hkv, D, page, 2, seed=5).clean()
    for t in range(40):
        check_append(B, 2, Hkv, 1, D, page, [t, t], rotary=0, seed=100 + t, scale=2.0 ** ((t % 7) - 3), pool=pool)


def test_append_special_values():
    B, Hkv, D, page = 1, 1, 16, 16
    rows = torch.zeros((1, 1, 6, D))
    rows[0, 0, 0, 0], rows[0, 0, 1, 1], rows[0, 0, 1, 2] = float("nan"), float("inf"), -float("inf")
    rows[0, 0, 2, :4] = torch.tensor([448.0, 464.0, -448.0, 1.5 * 2 ** -9])  # 464 needs the next scale
    for dtype in (torch.float32, torch.bfloat16):
        x = rows.to(dtype).cuda()
        for cut in (3, 2):  # with and without the large row
            y = x[:, :, :cut].contiguous()
            pool = Pool(B, Hkv, D, page, 1, seed=6)
            before = pool.copy()
            bsa.nsa_cache_append(y, y, *pool.args(), torch.zeros(1, dtype=torch.int32, device="cuda"))
            codes, scales, _ = ocache.append(y.double().cpu().numpy(), before[0], before[2], before[4], [0], [cut])
            assert np.array_equal(pool.ks.double().cpu().numpy(), scales)
            a, b = pool.k.cpu().numpy(), codes
            nan = (b & 127) == 127
            assert np.array_equal(a[~nan], b[~nan]) and ((a[nan] & 127) == 127).all()
    assert float(pool.ks[pool.table[0, 0].item(), 0]) == 2.0 ** ocache.E_MIN  # nothing finite but zeros


def test_append_border_values_exactly():
    """Maxima on and next to 448 * 2^e."""
    for e in (-100, -20, 0, 5, 60):
        for m in (447.0, 448.0, 448.0 * (1 + 2.0 ** -23), 449.0):
            y = torch.zeros((1, 1, 1, 16))
            y[0, 0, 0, 3] = m * 2.0 ** e
            y = y.cuda()
            pool = Pool(1, 1, 16, 16, 1)
            bsa.nsa_cache_append(y, y, *pool.args(), torch.zeros(1, dtype=torch.int32, device="cuda"))
            assert float(pool.ks[pool.table[0, 0].item(), 0]) == ocache.least_scale(float(y[0, 0, 0, 3]))


def test_append_leaves_bad_pages_and_the_rest_alone():
    B, Hkv, D, page = 3, 2, 32, 16
    pool = Pool(B, Hkv, D, page, 3, seed=9)
    pool.table[0, 1], pool.table[1, 0] = pool.pages, -1
    check_append(B, 4, Hkv, 30, D, page, [3, 0, 18], seed=10, pool=pool)
    check_append(B, 4, Hkv, 30, D, page, [40, 45, -5], seed=11, pool=pool)  # past the table, and no sequence


def test_append_in_place_queries_and_uint8_or_float8():
    B, Hkv, D, page = 1, 1, 64, 64
    q = torch.randn((B, 4, 5, D)).to(torch.bfloat16).cuda()
    k = torch.randn((B, Hkv, 5, D)).to(torch.bfloat16).cuda()
    lens = torch.tensor([3], dtype=torch.int64, device="cuda")  # other integer types are converted
    a, b = Pool(B, Hkv, D, page, 1).clean(), Pool(B, Hkv, D, page, 1).clean()
    want = bsa.nsa_cache_append(k, k, *a.args(), lens, inv_freq=freqs(D), q=q)
    got = bsa.nsa_cache_append(k, k, b.k.view(F8), b.v.view(F8), b.ks, b.vs, b.table, lens, inv_freq=freqs(D), q=q,
                               q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(a.k, b.k) and torch.equal(a.vs, b.vs)


# ------------------------------------------------------------------- decode


def check_decode(got, lse, q, pool, lens, idx):
    p = pool.copy()
    out, wl, sums = ocache.decode(q.double().cpu().numpy(), p[0], p[1], p[2], p[3], p[4], lens,
                                  None if idx is None else idx.cpu().numpy())
    x = got.double().cpu().numpy()
    n = max(1, max(lens))
    # f16 probabilities; scores and sums in fp32 (numerator and denominator); the result.  An f16 below 2^-14 is off by
    # up to 2^-25; probabilities (largest 1) are rounded times their page's scale over a unit that is at most 2^3 of
    # it, so that is 2^-22 of a probability of 1 (pages further off the unit are rounded on their own)
    bound = (1 + BF) * (2.0 ** -11 * sums["p"] + U * (sums["e"] + 2 * n * sums["p"]) + 2.0 ** -22 * sums["v"])
    bound += BF * np.abs(out)
    assert np.isfinite(x).all()
    assert (np.abs(x - out) - bound).max() <= 1e-30, f"{(np.abs(x - out) - bound).max():.3e} over its bound"
    y = lse.double().cpu().numpy()
    tol = U * (sums["lse"] + n + 8) + 2.0 ** -23 * np.abs(wl)
    assert (np.abs(y - wl) <= tol).all()


def select(B, Hkv, S, lens, page, seed):
    r = np.random.default_rng(seed)
    idx = np.full((B, Hkv, 1, S), -1, dtype=np.int32)
    for b in range(B):
        nb = -(-max(lens[b], 0) // page)
        for h in range(Hkv):
            pick = r.permutation(nb)[: S]
            idx[b, h, 0, r.permutation(S)[: len(pick)]] = pick
    return torch.from_numpy(idx).cuda()


def run_decode(B, Hq, Hkv, D, page, lens, S=0, seed=0, pool=None, change=None):
    max_pages = max(1, max(-(-x // page) for x in lens))
    pool = pool or Pool(B, Hkv, D, page, max_pages, seed).clean()
    q = torch.randn((B, Hq, 1, D), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    idx = select(B, Hkv, S, lens, page, seed) if S else None
    if change is not None:
        idx = change(idx)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = bsa.nsa_select_decode(q, *pool.args(), lt, block_idx=idx, return_lse=True)
    torch.cuda.synchronize()
    check_decode(out, lse, q, pool, lens, idx)
    return out, lse


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("S", [0, 5])
def test_decode_shapes(D, page, S):
    run_decode(3, 8, 2, D, page, [1, 4 * page + 7, 9 * page], S=S, seed=D + page)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (5, 1), (16, 1), (12, 1), (32, 8), (15, 1)])
def test_decode_group_sizes(Hq, Hkv):
    run_decode(2, Hq, Hkv, 64, 32, [77, 200], seed=Hq)
    run_decode(2, Hq, Hkv, 128, 64, [700, 64], S=4, seed=Hq)


def test_decode_empty_and_full_sequences():
    out, lse = run_decode(6, 4, 2, 64, 16, [0, 16, 1, 0, 15, 17], seed=1)
    assert not out[0].any() and not out[3].any() and (lse[0] == -1.0e9).all()
    run_decode(4, 4, 2, 64, 16, [0, 0, 0, 5], S=3, seed=2)
    out, lse = run_decode(2, 4, 2, 64, 16, [0, 0], seed=3)
    assert not out.any() and (lse == -1.0e9).all()


@pytest.mark.parametrize("B", [1, 2, 130, 300])
def test_decode_ragged_batches(B):
    run_decode(B, 2, 1, 32, 16, [(37 * b) % 230 for b in range(B)], seed=B)


def test_decode_one_long_sequence_over_every_block():
    run_decode(1, 4, 1, 128, 64, [40001], seed=4)
    run_decode(2, 2, 2, 16, 16, [9000, 3], seed=5)


def test_decode_selection_is_a_set():
    page, lens = 32, [300, 95]

    def odd(idx):
        idx[:, :, 0, 1] = idx[:, :, 0, 0]  # repeated
        idx[0, 0, 0, 3] = 50  # past the sequence
        idx[1, 1] = -1  # nothing
        return idx

    out, lse = run_decode(2, 4, 2, 64, page, lens, S=6, seed=6, change=odd)
    assert not out[1, 2:].any() and (lse[1, 2:] == -1.0e9).all()


def many(B, page, longest, seed):
    """Lengths of B sequences: empty ones, single tokens, whole pages and anything else."""
    n = np.random.default_rng(seed).integers(0, longest + 1, B)
    n[::7], n[3::11], n[5::13] = 0, 1, longest // page * page
    return [int(x) for x in n]


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_selected_pages_of_many_sequences(D, page):
    run_decode(311, 3, 1, D, page, many(311, page, 6 * page, D), S=5, seed=D + page)


@pytest.mark.parametrize("B,Hq,Hkv,S", [(400, 1, 1, 1), (170, 32, 2, 3), (77, 20, 4, 16), (310, 5, 1, 2), (21, 240, 15, 9)])
def test_decode_selected_pages_of_many_heads(B, Hq, Hkv, S):
    run_decode(B, Hq, Hkv, 64, 16, many(B, 16, 200, B), S=S, seed=S)


@pytest.mark.parametrize("D,page,S", [(128, 64, 4), (32, 16, 32), (64, 128, 3), (16, 32, 7)])
def test_decode_many_selections_with_repeats_and_dead_slots(D, page, S):
    B, Hkv, pages = 320, 1, 40
    r = np.random.default_rng(S)

    def odd(idx):
        a = r.integers(-2, pages // 2, (B, Hkv, 1, S)).astype(np.int32)  # -1, -2, repeats, blocks past the sequence
        a[::5] = -1                                                      # nothing at all
        a[1::9, :, :, 1:] = a[1::9, :, :, :1]                            # one page throughout
        a[2::17, :, :, 0] = 2 ** 31 - 1
        a[3::17, :, :, -1] = -2 ** 31
        return torch.from_numpy(a).cuda()

    run_decode(B, 4, Hkv, D, page, many(B, page, 8 * page + 5, S), S=S, seed=S, change=odd)


def test_decode_many_sequences_with_garbage_and_bad_pages():
    B, Hkv, D, page, last = 330, 1, 64, 32, 3
    lens = [40 + b % 50 for b in range(B)]
    pool = Pool(B, Hkv, D, page, last + 1, seed=7).clean()
    for b, n in enumerate(lens):
        for c in (pool.k, pool.v):
            c[pool.table[b, n // page].item(), :, n % page:] = 0x7F  # NaN codes behind the last token
            c[pool.table[b, last].item()] = 0x7F
    pool.ks[pool.table[:, last].long()] = float("nan")
    pool.table[::6, 0] = pool.pages
    pool.table[1::6, 1] = -9
    run_decode(B, 4, Hkv, D, page, lens, S=4, pool=pool, seed=8)


def test_decode_garbage_behind_the_end_and_bad_pages():
    B, Hkv, D, page, lens = 2, 2, 64, 64, [70, 130]
    pool = Pool(B, Hkv, D, page, 4, seed=7).clean()
    for b, n in enumerate(lens):
        for c in (pool.k, pool.v):
            c[pool.table[b, n // page].item(), :, n % page:] = 0x7F  # NaN codes behind the last token
            c[pool.table[b, 3].item()] = 0x7F
    pool.ks[pool.table[:, 3].long()] = float("nan")
    run_decode(B, 4, Hkv, D, page, lens, pool=pool, seed=8)
    run_decode(B, 4, Hkv, D, page, lens, S=3, pool=pool, seed=8)
    pool.table[0, 0], pool.table[1, 1] = pool.pages + 1000000, -7  # never followed
    run_decode(B, 4, Hkv, D, page, lens, pool=pool, seed=9)


def test_decode_lengths_past_the_table_count_as_its_end():
    pool = Pool(1, 1, 32, 16, 4, seed=3).clean()
    q = torch.randn((1, 2, 1, 32)).to(torch.bfloat16).cuda()
    a = bsa.nsa_select_decode(q, *pool.args(), torch.tensor([64], device="cuda"))
    b = bsa.nsa_select_decode(q, *pool.args(), torch.tensor([1000], device="cuda"))
    assert torch.equal(a, b)


def test_decode_scales_far_apart():
    """Pages whose scales differ by 2^60, and one whose values are all zero under the least scale."""
    B, Hkv, D, page = 1, 1, 64, 16
    pool = Pool(B, Hkv, D, page, 4, seed=12).clean()
    t = pool.table[0].long()
    pool.vs[t] = torch.tensor([2.0 ** 40, 2.0 ** -20, 2.0 ** -96, 1.0], device="cuda")[:, None]
    pool.v[t[2]] = 0
    pool.ks[t] = 2.0 ** -8
    run_decode(B, 4, Hkv, D, page, [64], pool=pool, seed=13)
    # the small page alone: its values come out with their own precision
    run_decode(B, 4, Hkv, D, page, [64], S=1, pool=pool, seed=13, change=lambda i: torch.ones_like(i))


def test_decode_queries_of_any_magnitude():
    pool = Pool(1, 1, 64, 16, 2, seed=14).clean()
    lt = torch.tensor([29], device="cuda")
    base = torch.randn((1, 4, 1, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for e in (-140, -30, 0, 12):
        q = (base.float() * 2.0 ** e).to(torch.bfloat16).cuda()
        out, lse = bsa.nsa_select_decode(q, *pool.args(), lt, return_lse=True)
        check_decode(out, lse, q, pool, [29], None)


def test_decode_repeats_on_another_stream_and_in_graphs_at_once():
    B, Hq, Hkv, D, page = 4, 8, 2, 128, 64
    lens = [5000, 1, 777, 2048]
    pool = Pool(B, Hkv, D, page, 80, seed=20).clean()
    q = torch.randn((B, Hq, 1, D)).to(torch.bfloat16).cuda()
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = bsa.nsa_select_decode(q, *pool.args(), lt, return_lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    second = bsa.nsa_select_decode(q, *pool.args(), lt, return_lse=True, stream=s)
    s.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(bsa.nsa_select_decode(q, *pool.args(), lt, return_lse=True))
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for other in (second, *outs):
        assert torch.equal(first[0], other[0]) and torch.equal(first[1], other[1])


# ------------------------------------------------- append and decode together


def test_a_served_sequence_matches_the_forward():
    """A prompt appended at once, then tokens one by one, each attended over its selection: what the whole-sequence
    forward computes on the values the cache holds."""
    from oracle import nsa as onsa

    B, Hq, Hkv, D, page, T0, T = 2, 8, 2, 64, 32, 75, 128
    g = torch.Generator().manual_seed(3)
    q = torch.randn((B, Hq, T, D), generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn((B, Hkv, T, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    f = freqs(D)
    pool = Pool(B, Hkv, D, page, T // page, seed=30)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    bsa.nsa_cache_append(k[:, :, :T0], v[:, :, :T0], *pool.args(), lens, inv_freq=f)
    lens += T0
    for t in range(T0, T):
        qr = bsa.nsa_cache_append(k[:, :, t:t + 1], v[:, :, t:t + 1], *pool.args(), lens, inv_freq=f,
                                  q=q[:, :, t:t + 1])
        lens += 1
        idx = select(B, Hkv, 3, [t + 1] * B, page, t)
        out, lse = bsa.nsa_select_decode(qr, *pool.args(), lens, block_idx=idx, return_lse=True)
        if t % 9 == 0 or t == T - 1:
            check_decode(out, lse, qr, pool, [t + 1] * B, idx)
    # the last token against the forward's oracle on the dequantised cache
    kc, vc, ks, vs, table = pool.copy()
    kk, vv = (np.stack([np.concatenate([ocache.VALUES[c[p]] * s[p][:, None, None] for p in table[b]], 1)
                        for b in range(B)]) for c, s in ((kc, ks), (vc, vs)))
    full = np.zeros((B, Hq, T, D))
    full[:, :, T - 1] = qr[:, :, 0].double().cpu().numpy()
    rows = np.full((B, Hkv, T, 3), -1)
    rows[:, :, T - 1] = idx[:, :, 0].cpu().numpy()
    want, wl = onsa.nsa_select_forward(full, kk, vv, rows, page)
    assert np.abs(lse[:, :, 0].double().cpu().numpy() - wl[:, :, T - 1]).max() <= 1e-4
    # bf16 result, f16 probabilities over at most 96 tokens
    err = np.abs(out[:, :, 0].double().cpu().numpy() - want[:, :, T - 1])
    assert (err <= 2.0 ** -8 * np.abs(want[:, :, T - 1]) + 2.0 ** -9 * np.abs(vv).max()).all()
