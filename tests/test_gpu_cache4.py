"""GPU: the paged 4-bit cache -- append with norm, rotation and scales, read back, single-token selection attention --
against the float64 oracle.

Tolerances.  Values, and keys that are neither normalised nor rotated, have exactly the oracle's codes and scales: a
group's maximum over 6 and an element over the scale are correctly rounded quotients, of which one that is no border of
the exact quotients' rounding does not become one (numbers of 24 and 4 bits).  A normalised and rotated key is off by E =
2^-19 of its reach (``test_gpu_qk_norm_rope.py``): its scale is a nearest one for some maximum within E of the exact one,
its codes are nearest ones for some value within E of the exact one, under the scale it got.

Decode: as in ``test_gpu_nsa_cache.py``, but no page has a scale of its own: an f16 below 2^-14 is off by up to 2^-25,
which is 2^-36 of the largest probability's units.
"""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import BsaError, bsa
from oracle import cache4
from oracle import rows as orows

pytestmark = pytest.mark.gpu
F32, BF, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U, STEP = 2.0 ** -22, 2.0 ** -8


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


def host(t):
    return t.detach().double().cpu().numpy()


class Pool:
    """A cache whose every byte holds something (NaN scales among it), and a scattered table."""

    def __init__(self, B, Hkv, D, page, max_pages, seed=0, spare=3, factors=False):
        r = np.random.default_rng(seed)
        self.pages = B * max_pages + spare

        def fill(width):
            return torch.from_numpy(r.integers(0, 256, (self.pages, Hkv, page, width), dtype=np.uint8)).cuda()

        self.k, self.v, self.ks, self.vs = fill(D // 2), fill(D // 2), fill(D // 16), fill(D // 16)
        self.table = torch.from_numpy(r.permutation(self.pages)[: B * max_pages].reshape(B, max_pages).astype(
            np.int32)).cuda()
        self.factors = {}
        if factors:
            self.factors = {n: torch.from_numpy(np.exp2(r.uniform(-3, 3, Hkv))).float().cuda()
                            for n in ("k_factor", "v_factor")}

    def clean(self):
        """Scales of 1/32 to 1/2 (for pages whose tokens are read)."""
        for c in (self.ks, self.vs):
            c.copy_(c % 32 + 0x10)
        return self

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table

    def copy(self):
        return [t.cpu().numpy().copy() for t in self.args()]

    def factor(self, name):
        return host(self.factors[name]) if self.factors else None


def freqs(rotary):
    return bsa.rope_frequencies(rotary, device="cuda")[0] if rotary else None


def weights(D, dtype=F32, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple((1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2))


def check_codes(got, scales, y, e):
    """Codes [D] and scale codes [D / 16] of rows got for values y, each off by at most e."""
    y, e = y.reshape(-1, 16), e.reshape(-1, 16)
    s = cache4.E4M3[scales.reshape(-1)]
    top = np.abs(y).max(-1) / 6.0
    et = e.max(-1) / 6.0
    best = np.abs(cache4.E4M3[cache4.e4m3_encode(top)] - top)
    assert (np.abs(s - np.minimum(top, 448.0)) <= np.where(top > 448, 0, best) + 2 * et).all()
    c = cache4.E2M1[got.reshape(-1, 16)]
    some = s > 0
    q = np.clip(np.where(some[:, None], y / np.where(some, s, 1.0)[:, None], 0.0), -6, 6)
    eq = np.where(some[:, None], e / np.where(some, s, 1.0)[:, None], 0.0)
    best = np.abs(q[..., None] - cache4.E2M1).min(-1)
    assert (np.abs(c - q) <= best + 2 * eq + 1e-15).all()


def check_append(B, Hq, Hkv, n, D, page, lens, new=None, dtype=BF, rotary=None, interleaved=False, seed=0, size=1.0,
                 pool=None, with_q=True, norm=True, rotary_scale=1.0, factors=False, inputs=None, **kw):
    g = torch.Generator().manual_seed(seed)
    rotary = D if rotary is None else rotary
    if inputs is None:
        k, v = ((torch.randn((B, Hkv, n, D), generator=g) * size).to(dtype).cuda() for _ in range(2))
        q = torch.randn((B, Hq, n, D), generator=g).to(dtype).cuda() if with_q else None
    else:
        k, v, q = inputs
    wq, wk = weights(D) if norm else (None, None)
    max_pages = max(-(-(x + n) // page) for x in lens)
    pool = pool or Pool(B, Hkv, D, page, max(1, max_pages), seed, factors=factors)
    before = pool.copy()
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nt = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    f = freqs(rotary)
    q0 = None if q is None else host(q)  # (it may be overwritten)
    got = bsa.nsa_cache4_append(k, v, *pool.args(), lt, new_lens=nt, inv_freq=f, interleaved=interleaved, q=q,
                                q_weight=wq if q is not None else None, k_weight=wk, rotary_scale=rotary_scale,
                                **pool.factors, **kw)
    torch.cuda.synchronize()
    after = pool.copy()
    news = [n] * B if new is None else [max(0, min(x, n)) for x in new]
    pos = np.array(lens, dtype=np.float64)[:, None] + np.arange(n)
    fr = host(f) if rotary else np.zeros(0)
    kk, ek = orows.forward(host(k), host(wk) if norm else None, pos, fr, interleaved, rotary_scale, 1e-6)
    plain = not norm and not rotary
    vv = host(v)
    for h in range(Hkv):
        if pool.factors:  # quotients in fp32: 2^-24 of themselves
            kk[:, h] /= pool.factor("k_factor")[h]
            ek[:, h] /= pool.factor("k_factor")[h]
    ek = 2.0 ** -19 * ek
    table = before[4]
    ids, at, bb, tt = [], [], [], []
    for b in range(B):
        for t, pid, slot in cache4.slots(table[b], pool.pages, page, lens[b], news[b]):
            ids.append(pid), at.append(slot), bb.append(b), tt.append(t)
    left = np.ones((pool.pages, page), dtype=bool)
    left[ids, at] = False
    for x0, x1 in zip(before[:4], after[:4]):
        m = np.broadcast_to(left[:, None, :, None], x0.shape)
        assert np.array_equal(x0[m], x1[m])  # slots without a new token
    for h in range(Hkv):
        if not ids:
            break
        x = vv[bb, h, tt]
        if pool.factors:
            x = (x.astype(np.float32) / pool.factor("v_factor")[h].astype(np.float32)).astype(np.float64)
        codes, scales = cache4.encode(x)
        fine = np.repeat(scales != 0x7F, 16, -1)
        assert np.array_equal(after[3][ids, h, at], scales)
        assert np.array_equal(cache4.unpack(after[1][ids, h, at])[fine], codes[fine])
        x, e = kk[bb, h, tt], ek[bb, h, tt]
        if plain and not pool.factors:
            codes, scales = cache4.encode(x)
            fine = np.repeat(scales != 0x7F, 16, -1)
            assert np.array_equal(after[2][ids, h, at], scales)
            assert np.array_equal(cache4.unpack(after[0][ids, h, at])[fine], codes[fine])
        else:
            check_codes(cache4.unpack(after[0][ids, h, at]), after[2][ids, h, at], x, e)
    if q is not None:
        want, e = orows.forward(q0, host(wq) if norm else None, pos, fr, interleaved, rotary_scale, 1e-6)
        h = torch.finfo(dtype).eps / 2
        for b in range(B):
            m = news[b]
            x, w = host(got[b, :, :m]), want[b, :, :m]
            assert (np.abs(x - w) <= h * np.abs(w) + (1 + h) * 2.0 ** -19 * e[b, :, :m] + 1e-37).all()
            if new is not None and "q_out" not in kw:
                assert not got[b, :, m:].any()
    return pool, got


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_shapes(D, page):
    check_append(2, 4, 2, 2 * page + 3, D, page, [5, page], seed=D + page)
    check_append(3, 6, 2, 1, D, page, [0, page - 1, 3 * page], seed=D + page + 1)
    check_append(2, 2, 1, 2 * page + 3, D, page, [5, page], seed=D + page, rotary=0, norm=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotary", [(64, 0), (64, 16), (64, 32), (64, 48), (64, 64), (128, 112), (128, 80), (16, 16),
                                      (32, 16)])
def test_append_rotations(dtype, interleaved, D, rotary):
    """Every way in which the runs of eight of a group lie in one thread, in two, or in either half."""
    for norm in (True, False):
        check_append(2, 9, 3, 37, D, 32, [0, 70], dtype=dtype, interleaved=interleaved, rotary=rotary, seed=rotary,
                     norm=norm, rotary_scale=1.25)


def test_append_ragged_batch_and_lengths_zero():
    check_append(5, 4, 2, 70, 32, 32, [0, 31, 32, 100, 7], new=[70, 0, 1, 33, 69], seed=3)
    check_append(2, 2, 2, 9, 64, 16, [4, 0], new=[-3, 100], seed=4)


@pytest.mark.parametrize("B,n,Hq,Hkv", [(128, 1, 64, 4), (300, 2, 3, 3), (1, 1000, 16, 1), (40, 33, 2, 2), (1, 1, 240, 15)])
def test_append_batches(B, n, Hq, Hkv):
    check_append(B, Hq, Hkv, n, 64, 32, [(37 * b) % 130 for b in range(B)], seed=B)
    check_append(B, Hq, Hkv, n, 128, 64, [(37 * b) % 130 for b in range(B)], seed=B, rotary=0, norm=False, dtype=F32)


def test_append_without_queries():
    check_append(1, 2, 2, 20, 64, 64, [50], with_q=False)


@pytest.mark.parametrize("size", [2.0 ** -14, 2.0 ** -8, 0.02, 3.0, 300.0, 2.0 ** 14])
def test_append_magnitudes(size):
    """Scales from zero through e4m3's subnormals to saturation, with a factor and without."""
    for dtype in (BF, F32):
        check_append(1, 1, 1, 50, 64, 16, [3], rotary=0, norm=False, size=size, dtype=dtype)
        check_append(1, 3, 3, 50, 64, 16, [3], rotary=0, norm=False, size=size, dtype=dtype, factors=True)
    check_append(1, 2, 2, 20, 64, 16, [3], size=size, factors=True)


def test_append_on_the_borders_of_codes_and_scales():
    """Maxima whose sixth lies half way between two scales, elements half way between two codes: the even one."""
    scales = cache4.E4M3[1:127]
    mids = (scales[1:] + scales[:-1]) / 2
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in np.concatenate([scales, mids]):
        near = cache4.E4M3[cache4.e4m3_encode(s)]
        rows.append(np.concatenate([[6 * s], ties * near, -ties * near, [-near]]))
    x = np.array(rows, dtype=np.float64)
    one_up = np.nextafter(x.astype(np.float32), np.float32(np.inf))
    one_down = np.nextafter(x.astype(np.float32), np.float32(0))
    x = torch.from_numpy(np.concatenate([x, one_up, one_down]).astype(np.float32))
    x = x[: x.shape[0] // 4 * 4].reshape(1, 1, -1, 64)
    for dtype in (F32, BF):
        t = x.to(dtype).cuda()
        check_append(1, 1, 1, t.shape[2], 64, 16, [0], rotary=0, norm=False, dtype=dtype, inputs=(t, -t, None))


def test_append_quotients_are_the_divisions():
    """Elements over every scale, against torch's fp32 division."""
    g = torch.Generator(device="cuda").manual_seed(0)
    n = 20000
    x = torch.randn((1, 1, n, 128), generator=g, device="cuda") * torch.exp2(
        torch.randint(-9, 9, (1, 1, n, 1), generator=g, device="cuda").float())
    pool = Pool(1, 1, 128, 128, -(-n // 128))
    bsa.nsa_cache4_append(x, x, *pool.args(), torch.zeros(1, device="cuda", dtype=torch.int32))
    t = pool.table[0].long()
    s = pool.ks[t, 0].flatten(0, 1)[:n].view(F8).float()
    s = s.repeat_interleave(16, -1)
    y = torch.where(s > 0, x[0, 0] / s, 0.0 * x[0, 0])  # (a scale of zero has codes of zero, with their signs)
    codes = cache4.e2m1_encode(host(y))
    assert np.array_equal(cache4.unpack(pool.k[t, 0].flatten(0, 1)[:n].cpu().numpy()), codes)
    assert torch.equal(pool.k[t, 0].flatten(0, 1)[:n], pool.v[t, 0].flatten(0, 1)[:n])


def test_append_nan_and_infinity():
    """Their groups read back as NaN; neighbours, other tokens and pages are what they are without."""
    x = torch.randn((1, 2, 40, 64), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    y = x.clone()
    y[0, 0, 3, 17], y[0, 1, 20, 63], y[0, 0, 39, 0] = float("nan"), float("inf"), float("-inf")
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    a, b = Pool(1, 2, 64, 16, 3), Pool(1, 2, 64, 16, 3)
    bsa.nsa_cache4_append(x, y, *a.args(), lens)
    bsa.nsa_cache4_append(x, x, *b.args(), lens)
    va, vb = (bsa.nsa_cache4_read(*p.args(), lens + 40, 40, starts=lens)[1] for p in (a, b))
    bad = torch.zeros((1, 2, 40, 4), dtype=torch.bool, device="cuda")
    bad[0, 0, 3, 1] = bad[0, 1, 20, 3] = bad[0, 0, 39, 0] = True
    bad = bad.repeat_interleave(16, -1)
    assert va[bad].isnan().all() and torch.equal(va[~bad], vb[~bad]) and torch.equal(a.ks, b.ks)


def test_append_far_positions():
    page, far = 64, (1 << 30) + 12345
    pool = Pool(1, 2, 64, page, 2)
    table = torch.full((1, -(-far // page) + 2), -1, dtype=torch.int32, device="cuda")
    table[0, far // page: far // page + 2] = pool.table[0]
    pool.table = table
    check_append(1, 4, 2, 30, 64, page, [far], pool=pool)


def test_append_leaves_bad_pages_and_the_rest_alone():
    B, Hkv, D, page = 3, 2, 32, 16
    pool = Pool(B, Hkv, D, page, 3, seed=9)
    pool.table[0, 1], pool.table[1, 0] = pool.pages, -1
    check_append(B, 4, Hkv, 30, D, page, [3, 0, 18], seed=10, pool=pool)
    check_append(B, 4, Hkv, 30, D, page, [40, 45, -5], seed=11, pool=pool)  # past the table, and no sequence


def test_append_strides_and_types():
    """From one fused projection, copies where rows need them, results in place, other integers and views of scales."""
    B, Hq, Hkv, n, D, page = 2, 6, 2, 5, 64, 16
    x = torch.randn((B, n, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(2)).to(BF).cuda().transpose(1, 2)
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    a, _ = check_append(B, Hq, Hkv, n, D, page, [3, 14], inputs=(k, v, q), seed=1)
    cols = [t.transpose(2, 3).contiguous().transpose(2, 3) for t in (k, v, q)]
    b, _ = check_append(B, Hq, Hkv, n, D, page, [3, 14], inputs=cols, seed=1)
    flat = [torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape) for t in (k, v, q)]
    c, _ = check_append(B, Hq, Hkv, n, D, page, [3, 14], inputs=flat, seed=1)
    for p in (b, c):
        assert all(torch.equal(s, t) for s, t in zip(a.args(), p.args()))
    own = q.contiguous()
    d, got = check_append(B, Hq, Hkv, n, D, page, [3, 14], inputs=(k, v, own), seed=1, q_out=own)
    assert got is own
    one = k[:, :1, :1].expand(B, Hkv, n, D)
    check_append(B, Hq, Hkv, n, D, page, [3, 14], inputs=(one, one, q), seed=1)
    e = Pool(B, Hkv, D, page, 2, 1)
    w = weights(D)
    bsa.nsa_cache4_append(k, v, e.k, e.v, e.ks.view(F8), e.vs.view(F8), e.table.long(),
                          torch.tensor([3, 14], device="cuda"), inv_freq=freqs(D), q=q, q_weight=w[0], k_weight=w[1])
    assert all(torch.equal(s, t) for s, t in zip(a.args(), e.args()))


# --------------------------------------------------------------------- read


def check_read(pool, lens, n, starts=None, dtype=BF, **kw):
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    got = bsa.nsa_cache4_read(*pool.args(), lt, n, starts=st, dtype=dtype, **pool.factors, **kw)
    p = pool.copy()
    page, B = pool.k.shape[2], len(lens)
    for i, name in enumerate(("k_factor", "v_factor")):
        f = pool.factor(name)
        want = np.zeros(got[i].shape)
        for b in range(B):
            s = 0 if starts is None else starts[b]
            for t, pid, slot in cache4.slots(p[4][b], pool.pages, page, s, max(0, min(n, lens[b] - s))):
                want[b, :, t] = cache4.values(p[i][pid, :, slot], p[2 + i][pid, :, slot],
                                              1.0 if f is None else f[:, None])
        x = host(got[i])
        h = torch.finfo(dtype).eps / 2 + (2.0 ** -24 if pool.factors else 0.0)
        assert got[i].dtype == dtype and np.array_equal(np.isnan(x), np.isnan(want))
        fine = ~np.isnan(want)
        # six bits: exact in either type without a factor
        assert (np.abs(x - want)[fine] <= (h * np.abs(want[fine]) if pool.factors else 0.0)).all()
    return got


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_read_shapes(D, page):
    for factors in (False, True):
        pool = Pool(3, 2, D, page, 4, seed=D + page, factors=factors)
        for dtype in (BF, F32):
            check_read(pool, [4 * page, 1, page + 3], 4 * page, dtype=dtype)
            check_read(pool, [4 * page, 0, page + 3], 2 * page + 1, starts=[page - 1, 0, page + 2], dtype=dtype)


def test_read_borders():
    pool = Pool(4, 1, 64, 16, 3, seed=1)
    pool.table[0, 1], pool.table[1, 0] = pool.pages, -7
    check_read(pool, [48, 48, 10 ** 6, -5], 60, starts=[5, 0, 40, 0])  # past the table, no sequence
    check_read(pool, [48, 48, 48, 48], 9, starts=[-1, -2 ** 31, 2 ** 31 - 1, 48])
    out = torch.full((2, 4, 1, 9, 64), 7.0, device="cuda")
    got = check_read(pool, [48, 2, 0, 48], 9, starts=[44, 0, 0, 3], dtype=F32, k_out=out[0], v_out=out[1])
    assert got[0].data_ptr() == out[0].data_ptr()


def test_what_is_appended_is_read():
    """Within a code's step and a scale's rounding of what went in, and exactly for what codes can hold."""
    B, H, n, D = 2, 3, 200, 128
    x = torch.randn((2, B, H, n, D), generator=torch.Generator().manual_seed(3)).cuda()
    lens = torch.tensor([0, 37], dtype=torch.int32, device="cuda")
    pool = Pool(B, H, D, 64, 4, factors=True)
    bsa.nsa_cache4_append(x[0], x[1], *pool.args(), lens, **pool.factors)
    once = bsa.nsa_cache4_read(*pool.args(), lens + n, n, starts=lens, dtype=F32, **pool.factors)
    for y, z in zip(x, once):
        top = y.abs().unflatten(-1, (-1, 16)).amax(-1, keepdim=True).expand(-1, -1, -1, -1, 16).flatten(-2)
        assert ((y - z).abs() <= top * (1 / 6 + 2.0 ** -4)).all()
    pool.factors = {}
    bsa.nsa_cache4_append(x[0], x[1], *pool.args(), lens)
    once = bsa.nsa_cache4_read(*pool.args(), lens + n, n, starts=lens)  # bf16 holds every value
    bsa.nsa_cache4_append(*once, *pool.args(), lens)
    twice = bsa.nsa_cache4_read(*pool.args(), lens + n, n, starts=lens)
    full = once[0].abs().unflatten(-1, (-1, 16)).amax(-1)  # groups that use their largest code keep their scale
    keep = (full == 6.0 * (full / 6.0).to(F8).to(BF)).repeat_interleave(16, -1)
    assert keep.float().mean() > 0.5 and torch.equal(once[0][keep], twice[0][keep])


# ------------------------------------------------------------------- decode


def check_decode(got, lse, q, pool, lens, idx):
    p = pool.copy()
    out, wl, sums = cache4.decode(host(q), *p, lens, None if idx is None else idx.cpu().numpy(),
                                  pool.factor("k_factor"), pool.factor("v_factor"))
    x = host(got)
    n = max(1, max(lens))
    # f16 probabilities; scores and sums in fp32 (numerator and denominator); the result
    bound = (1 + STEP) * (2.0 ** -11 * sums["p"] + U * (sums["e"] + 2 * n * sums["p"]) + 2.0 ** -36 * sums["v"])
    bound += STEP * np.abs(out)
    assert np.isfinite(x).all()
    assert (np.abs(x - out) - bound).max() <= 1e-30, f"{(np.abs(x - out) - bound).max():.3e} over its bound"
    tol = U * (sums["lse"] + n + 8) + 2.0 ** -23 * np.abs(wl)
    assert (np.abs(host(lse) - wl) <= tol).all()


def select(B, Hkv, S, lens, page, seed):
    r = np.random.default_rng(seed)
    idx = np.full((B, Hkv, 1, S), -1, dtype=np.int32)
    for b in range(B):
        nb = -(-max(lens[b], 0) // page)
        for h in range(Hkv):
            pick = r.permutation(nb)[: S]
            idx[b, h, 0, r.permutation(S)[: len(pick)]] = pick
    return torch.from_numpy(idx).cuda()


def run_decode(B, Hq, Hkv, D, page, lens, S=0, seed=0, pool=None, change=None, factors=False, size=1.0,
               room=0):
    """``room``: tokens for which the table has places behind the longest sequence's, with no pages there."""
    max_pages = max(1, max(-(-x // page) for x in lens))
    pool = pool or Pool(B, Hkv, D, page, max_pages, seed, factors=factors).clean()
    if room:
        none = torch.full((B, -(-room // page)), -1, dtype=torch.int32, device="cuda")
        pool.table = torch.cat((pool.table, none), 1)
    q = (torch.randn((B, Hq, 1, D), generator=torch.Generator().manual_seed(seed)) * size).to(BF).cuda()
    idx = select(B, Hkv, S, lens, page, seed) if S else None
    if change is not None:
        idx = change(idx)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = bsa.nsa_cache4_decode(q, *pool.args(), lt, block_idx=idx, return_lse=True, **pool.factors)
    torch.cuda.synchronize()
    check_decode(out, lse, q, pool, lens, idx)
    return out, lse


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("S", [0, 5])
def test_decode_shapes(D, page, S):
    run_decode(3, 8, 2, D, page, [1, 4 * page + 7, 9 * page], S=S, seed=D + page, factors=page < 64)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (5, 1), (16, 1), (12, 1), (32, 8), (15, 1)])
def test_decode_group_sizes(Hq, Hkv):
    run_decode(2, Hq, Hkv, 64, 32, [77, 200], seed=Hq)
    run_decode(2, Hq, Hkv, 128, 64, [700, 64], S=4, seed=Hq)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("S", [0, 5])
@pytest.mark.parametrize("G", [8, 9, 16])
def test_decode_groups_of_eight_and_more(D, page, S, G):
    run_decode(3, 2 * G, 2, D, page, [2, 3 * page + 9, 7 * page - 1], S=S, seed=D + page + G, factors=page < 128)


def test_decode_empty_and_full_sequences():
    out, lse = run_decode(6, 4, 2, 64, 16, [0, 16, 1, 0, 15, 17], seed=1)
    assert not out[0].any() and not out[3].any() and (lse[0] == -1.0e9).all()
    run_decode(4, 4, 2, 64, 16, [0, 0, 0, 5], S=3, seed=2)
    out, lse = run_decode(2, 4, 2, 64, 16, [0, 0], seed=3)
    assert not out.any() and (lse == -1.0e9).all()
    for S in (0, 2):
        lt = torch.tensor([-2 ** 31, -1], dtype=torch.int32, device="cuda")
        pool = Pool(2, 1, 64, 32, 3, seed=1).clean()
        idx = torch.zeros((2, 1, 1, S), dtype=torch.int32, device="cuda") if S else None
        out, lse = bsa.nsa_cache4_decode(torch.ones((2, 2, 1, 64), device="cuda", dtype=BF), *pool.args(), lt,
                                         block_idx=idx, return_lse=True)
        assert not out.any() and (lse == -1.0e9).all()


@pytest.mark.parametrize("B", [1, 2, 130, 300])
def test_decode_ragged_batches(B):
    run_decode(B, 2, 1, 32, 16, [(37 * b) % 230 for b in range(B)], seed=B)


@pytest.mark.parametrize("B,H,D,page,longest", [(600, 1, 128, 64, 700), (9, 3, 128, 32, 3000), (5, 2, 64, 128, 9000)])
def test_decode_ranges_that_end_anywhere(B, H, D, page, longest):
    """Lists of many short pairs (several to a block, empty ones between) and of few long ones (several blocks to one)."""
    run_decode(B, 2 * H, H, D, page, [(61 * b * b) % longest for b in range(B)], seed=B)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [3, 8, 9, 16])
def test_decode_short_sequences_of_long_tables(D, page, G):
    """Tables that are too long for the form of short ones, whatever the sequences: empty ranges among them."""
    run_decode(4, 2 * G, 2, D, page, [2, 0, 4 * page + 9, 9 * page - 1], seed=D + page + G, factors=page < 64, room=20000)


@pytest.mark.parametrize("B,Hkv", [(2, 2), (33, 1), (130, 1), (300, 2), (600, 1)])
@pytest.mark.parametrize("room", [0, 1100, 20000])
def test_decode_batches_of_short_and_long_tables(B, Hkv, room):
    run_decode(B, 4 * Hkv, Hkv, 32, 16, [(37 * b) % 330 for b in range(B)], seed=B, room=room)
    run_decode(B, 9 * Hkv, Hkv, 128, 64, many(B, 64, 700, B), seed=B, room=room)


@pytest.mark.parametrize("stages", [1, 2, 3, 4, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65])
def test_decode_tables_around_the_rule_for_short_ones(stages):
    n = 128 * stages
    run_decode(2, 8, 2, 64, 64, [n, n - 63], seed=stages)
    run_decode(40, 16, 1, 128, 128, [n - 1] + [1, 0, 77, 130] * 9 + [n // 2, n, 128], seed=stages)


@pytest.mark.parametrize("B,Hkv,longest", [(31, 1, 4000), (32, 1, 4000), (33, 1, 4000), (20, 2, 3000), (22, 2, 3000)])
@pytest.mark.parametrize("D,page", [(128, 32), (64, 16)])
def test_decode_few_and_just_too_many_pairs_for_ranges_of_their_own(B, Hkv, longest, D, page):
    run_decode(B, 3 * Hkv, Hkv, D, page, many(B, page, longest, B), seed=B)
    run_decode(B, 3 * Hkv, Hkv, D, page, [longest] + [1] * (B - 2) + [0], seed=B)


@pytest.mark.parametrize("B,Hq,Hkv", [(4, 16, 1), (150, 5, 1), (90, 14, 2), (70, 15, 1), (170, 4, 1)])
def test_decode_long_sequences_among_many_short_ones(B, Hq, Hkv):
    """Many rows to join, of which some have parts from most blocks and most have none."""
    lens = many(B, 64, 200, B)
    lens[1], lens[B // 2] = 20011, 9000
    run_decode(B, Hq, Hkv, 64, 64, lens, seed=B)


def test_decode_one_long_sequence_over_every_block():
    run_decode(1, 4, 1, 128, 64, [40001], seed=4)
    run_decode(2, 2, 2, 16, 16, [9000, 3], seed=5)


def many(B, page, longest, seed):
    """Lengths of B sequences: empty ones, single tokens, whole pages and anything else."""
    n = np.random.default_rng(seed).integers(0, longest + 1, B)
    n[::7], n[3::11], n[5::13] = 0, 1, longest // page * page
    return [int(x) for x in n]


@pytest.mark.parametrize("D,page", [(16, 128), (32, 16), (64, 64), (128, 32), (128, 16)])
def test_decode_selected_pages_of_many_sequences(D, page):
    run_decode(311, 3, 1, D, page, many(311, page, 6 * page, D), S=5, seed=D + page)


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


@pytest.mark.parametrize("D,page,S", [(128, 64, 32), (64, 16, 9), (16, 128, 17)])
def test_decode_one_page_in_slots_of_several_blocks(D, page, S):
    """Few pairs, whose slots are shared out: a page that is listed again, in any block's slots, counts once."""
    r = np.random.default_rng(S)
    run_decode(2, 6, 2, D, page, [11 * page + 5, 3 * page], S=S, seed=S,
               change=lambda idx: torch.from_numpy(r.integers(-1, 6, tuple(idx.shape)).astype(np.int32)).cuda())


@pytest.mark.parametrize("B,D,page,S", [(2, 64, 64, 0), (2, 128, 32, 3), (330, 64, 32, 4), (330, 16, 16, 0)])
def test_decode_garbage_behind_the_end_and_bad_pages(B, D, page, S):
    """NaN scales behind the last token, on unused pages, and pages outside the pool."""
    last = 3
    lens = [2 * page - 20 + b % 25 for b in range(B)]
    pool = Pool(B, 1, D, page, last + 1, seed=7).clean()
    for b, n in enumerate(lens):
        for c in (pool.ks, pool.vs):
            if n % page:
                c[pool.table[b, n // page].item(), :, n % page:] = 0x7F
            c[pool.table[b, last].item()] = 0xFF
    run_decode(B, 4, 1, D, page, lens, S=S, pool=pool, seed=8)
    pool.table[::6, 0] = pool.pages + 1000000
    pool.table[1::6, 1] = -9
    run_decode(B, 4, 1, D, page, lens, S=S, pool=pool, seed=8)


def test_decode_nan_in_a_read_token_is_loud():
    pool = Pool(1, 2, 64, 16, 2, seed=3).clean()
    pool.ks[pool.table[0, 0].item(), 0, 5, 2] = 0x7F
    pool.vs[pool.table[0, 1].item(), 1, 3, 1] = 0x7F
    out = bsa.nsa_cache4_decode(torch.ones((1, 4, 1, 64), device="cuda", dtype=BF), *pool.args(),
                                torch.tensor([30], device="cuda"))
    assert out[0, :2].isnan().all() and out[0, 2:, :, 16:32].isnan().all()
    assert out[0, 2:, :, :16].isfinite().all() and out[0, 2:, :, 32:].isfinite().all()


def test_decode_lengths_past_the_table_count_as_its_end():
    pool = Pool(1, 1, 32, 16, 4, seed=3).clean()
    q = torch.randn((1, 2, 1, 32)).to(BF).cuda()
    a = bsa.nsa_cache4_decode(q, *pool.args(), torch.tensor([64], device="cuda"))
    b = bsa.nsa_cache4_decode(q, *pool.args(), torch.tensor([1000], device="cuda"))
    assert torch.equal(a, b)


@pytest.mark.parametrize("D,page", [(16, 16), (64, 64), (128, 32), (32, 128)])
@pytest.mark.parametrize("short", [0, 1, 15, 16, 127, 128, 32 * 128 + 1])
def test_decode_of_the_longest_sequences(D, page, short):
    """Tokens up to the largest number that a table may hold, almost all on pages that the table does not have."""
    max_pages = (2 ** 31 - 1) // page
    n = max_pages * page - short
    last = (n - 1) // page
    held = sorted({0, 5, last // 2, last - 32, last - 1, last})
    pool = Pool(1, 1, D, page, len(held), seed=D + short).clean()
    dense = pool.table
    q = torch.randn((1, 3, 1, D), generator=torch.Generator().manual_seed(short)).to(BF).cuda()
    tokens = (len(held) - 1) * page + (n - 1) % page + 1
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    table[0, held] = dense[0]
    idx = torch.tensor(held, dtype=torch.int32, device="cuda").view(1, 1, 1, -1)
    for length in (n, 2 ** 31 - 1) if short == 0 else (n,):
        lt = torch.tensor([length], dtype=torch.int32, device="cuda")
        for pick in (None, idx):
            out, lse = bsa.nsa_cache4_decode(q, *pool.args()[:4], table, lt, block_idx=pick, return_lse=True)
            torch.cuda.synchronize()
            check_decode(out, lse, q, pool, [tokens], None)


def test_decode_pools_past_32_bits():
    """Codes more than 2^32 bytes into the pool."""
    pages, H, page, D = 150000, 2, 128, 128
    k = torch.zeros((pages, H, page, D // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros((pages, H, page, D // 16), dtype=torch.uint8, device="cuda")
    small = Pool(1, H, D, page, 3, seed=4).clean()
    ids = torch.tensor([pages - 1, 140000, 7], device="cuda")
    x = torch.randn((1, H, 300, D), device="cuda").to(BF)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn((1, 8, 1, D), device="cuda").to(BF)
    got = []
    for cache, table in (((k, k, s, s), ids.int()[None]), ((small.k, small.k, small.ks, small.ks), small.table)):
        bsa.nsa_cache4_append(x, x, *cache, table, lens)
        back = bsa.nsa_cache4_read(*cache, table, lens + 300, 300)
        got.append((*back, *bsa.nsa_cache4_decode(q, *cache, table, lens + 300, return_lse=True),
                    bsa.nsa_cache4_decode(q, *cache, table, lens + 300,
                                          block_idx=torch.tensor([[[[0, 2]]] * 2], device="cuda"))))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_decode_queries_and_scores_of_any_magnitude():
    pool = Pool(1, 1, 64, 16, 40, seed=14).clean()
    for e in (-140, -30, 0, 12, 18, 22, 24, 40, 100):
        run_decode(1, 4, 1, 64, 16, [629], pool=pool, seed=e + 200, size=2.0 ** e)
        run_decode(1, 4, 1, 64, 16, [629], S=9, pool=pool, seed=e + 200, size=2.0 ** e)


def test_decode_factors_far_from_one():
    for e in (-60, -20, 20, 60):
        pool = Pool(2, 2, 64, 32, 4, seed=5, factors=True).clean()
        pool.factors["k_factor"] *= 2.0 ** (e / 4)
        pool.factors["v_factor"] *= 2.0 ** e
        for S in (0, 3):
            run_decode(2, 8, 2, 64, 32, [128, 65], S=S, pool=pool, seed=6, size=2.0 ** (-e / 4))


@pytest.mark.parametrize("below", [14, 20, 25, 28])
@pytest.mark.parametrize("D,page,S", [(64, 64, 0), (64, 64, 32), (128, 32, 0), (32, 16, 32)])
def test_decode_with_most_of_the_weight_on_a_token_of_no_value(D, page, S, below):
    """A first token of probability next to 1 and values of zero; the result is the sum of the many others, each of
    probability near 2^-below.  A probability p of the largest P is off by 2^-11 p, or by 2^-36 P where that is more;
    scores and sums are in fp32 (U an operation, one a product of 16 tokens and 16 to join the parts)."""
    pages, G = 32, 4
    r = np.random.default_rng(below + D)
    pool = Pool(1, 1, D, page, pages, seed=below).clean()
    at = pool.table[0].cpu().numpy()
    k = cache4.unpack(pool.k.cpu().numpy())
    k[..., 0] = 0
    k[at[0], 0, 0] = 0
    k[at[0], 0, 0, 0] = 7  # 6
    pool.k.copy_(torch.from_numpy(cache4.pack(k)))
    pool.ks.fill_(0x18)  # 1/16
    pool.v[at[0], 0, 0] = 0
    pool.v &= 0x77  # no signs
    q = 0.02 * torch.randn((1, G, 1, D), generator=torch.Generator().manual_seed(below))
    q[..., 0] = below * np.log(2.0) * D ** 0.5 / (6 / 16)
    q = q.to(BF).cuda()
    n = pages * page - 3
    idx = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, 1, 1, -1)[..., :S] if S else None
    out, lse = bsa.nsa_cache4_decode(q, *pool.args(), torch.tensor([n], device="cuda"), block_idx=idx, return_lse=True)
    p = pool.copy()
    want, wl, sums = cache4.decode(host(q), *p, [n], None if idx is None else idx.cpu().numpy())
    bound = (1 + STEP) * (2.0 ** -11 * sums["p"] + U * (sums["e"] + 2 * (n / 16 + 16) * sums["p"])
                          + 2.0 ** -36 * sums["v"])
    worst = (np.abs(host(out) - want) / (bound + STEP * np.abs(want))).max()
    assert worst <= 1, f"{worst:.2f} times its bound"
    assert (np.abs(host(lse) - wl) <= U * (sums["lse"] + n + 8) + 2.0 ** -23 * np.abs(wl)).all()


def test_decode_repeats_on_another_stream_and_in_graphs_at_once():
    B, Hq, Hkv, D, page = 4, 8, 2, 128, 64
    lens = [5000, 1, 777, 2048]
    pool = Pool(B, Hkv, D, page, 80, seed=20).clean()
    q = torch.randn((B, Hq, 1, D)).to(BF).cuda()
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for idx in (None, select(B, Hkv, 6, lens, page, 1)):
        first = bsa.nsa_cache4_decode(q, *pool.args(), lt, block_idx=idx, return_lse=True)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        second = bsa.nsa_cache4_decode(q, *pool.args(), lt, block_idx=idx, return_lse=True, stream=s)
        s.synchronize()
        graphs, outs = [], []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(bsa.nsa_cache4_decode(q, *pool.args(), lt, block_idx=idx, return_lse=True))
            graphs.append(graph)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(3):
            for graph, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        for got in (second, *outs):
            assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


def test_decode_workspace_is_what_it_says():
    pool = Pool(3, 2, 64, 32, 40, seed=2).clean()
    q = torch.randn((3, 8, 1, 64)).to(BF).cuda()
    lt = torch.tensor([1200, 3, 800], device="cuda")
    want = bsa.nsa_cache4_decode(q, *pool.args(), lt, return_lse=True)
    need = bsa.nsa_cache4_decode_workspace_size(3, 8, 2, 64, 32, 40, 0)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((3, 8, 1), device="cuda")
    got = bsa.nsa_cache4_decode(q, *pool.args(), lt, workspace=ws[:need], out=out, lse=lse, return_lse=True)
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1]) and (ws[need:] == 0xFF).all()
    with pytest.raises(BsaError) as e:
        bsa.nsa_cache4_decode(q, *pool.args(), lt, workspace=ws[: need - 1])
    assert e.value.status == 9


# ----------------------------------------------------------------- together


def test_a_prompt_then_tokens():
    """The whole path: a projection, normed and rotated, its prompt attended to and kept, then tokens over the cache;
    each step against the oracle over what the cache holds, and the cache's keys against the prompt's."""
    B, Hq, Hkv, T, D, page, S, steps = 2, 16, 2, 256, 64, 64, 3, 5
    g = torch.Generator(device="cuda").manual_seed(0)
    (wq, wk), (f, scale) = weights(D), bsa.rope_frequencies(D, scaling="bands", factor=4.0, original_length=64,
                                                            device="cuda")

    def projected(n):
        return torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF).transpose(1, 2).split(
            [Hq, Hkv, Hkv], 1)

    pool = Pool(B, Hkv, D, page, -(-(T + steps) // page), seed=1)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = projected(T)
    qr, kr = bsa.qk_norm_rope_forward(q, k, wq, wk, f, rotary_scale=scale)
    idx = torch.zeros((B, Hkv, T, S), dtype=torch.int32, device="cuda")
    idx[..., 1] = torch.arange(T, device="cuda") // page
    idx[..., 2] = -1
    out = bsa.nsa_select_attention(qr, kr, v, idx, page)
    assert torch.isfinite(out).all()
    bsa.nsa_cache4_append(kr, v, *pool.args(), lens)
    # the same prompt, normed and rotated on the way into the cache
    other = Pool(B, Hkv, D, page, -(-(T + steps) // page), seed=1)
    q2 = bsa.nsa_cache4_append(k, v, *other.args(), lens, inv_freq=f, q=q, q_weight=wq, k_weight=wk, rotary_scale=scale)
    assert torch.equal(q2, qr) and torch.equal(other.v, pool.v) and torch.equal(other.vs, pool.vs)
    lens = lens + T
    held, same = bsa.nsa_cache4_read(*pool.args(), lens, T)[0], bsa.nsa_cache4_read(*other.args(), lens, T)[0]
    # keys rounded to bf16 first (2^-8) may have other scales and codes; each is within a code's half step (1/6 of the
    # group's largest) and a scale's rounding (2^-4) of its key
    top = kr.float().abs().unflatten(-1, (-1, 16)).amax(-1).repeat_interleave(16, -1)
    assert ((held.float() - same.float()).abs() <= top * (2 * (1 / 6 + 2.0 ** -4) * (1 + 2.0 ** -7) + 2.0 ** -7)).all()
    for _ in range(steps):
        q, k, v = projected(1)
        q1 = bsa.nsa_cache4_append(k, v, *pool.args(), lens, inv_freq=f, q=q, q_weight=wq, k_weight=wk,
                                   rotary_scale=scale)
        lens = lens + 1
        n = lens.tolist()
        now = torch.tensor([[0, (x - 1) // page, -1] for x in n], dtype=torch.int32, device="cuda")
        now = now[:, None, None].expand(B, Hkv, 1, S)
        for pick in (None, now):
            got, lse = bsa.nsa_cache4_decode(q1, *pool.args(), lens, block_idx=pick, return_lse=True)
            check_decode(got, lse, q1, pool, n, pick)


def test_a_captured_step():
    """Append and decode in one graph, replayed while the lengths grow, against eager calls."""
    B, Hq, Hkv, D, page, steps = 3, 8, 2, 64, 32, 40
    w, f = weights(D), freqs(D)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((steps, B, 1, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
    pools = [Pool(B, Hkv, D, page, 4, seed=2).clean() for _ in range(2)]
    buf, lens = torch.empty_like(x[0]), torch.tensor([0, 31, 50], dtype=torch.int32, device="cuda")

    def step(pool, x, lens):
        q, k, v = x.transpose(1, 2).split([Hq, Hkv, Hkv], 1)
        q = bsa.nsa_cache4_append(k, v, *pool.args(), lens, inv_freq=f, q=q, q_weight=w[0], k_weight=w[1])
        return bsa.nsa_cache4_decode(q, *pool.args(), lens + 1)

    held = lens.clone()
    step(pools[0], buf, held)
    pools[0] = Pool(B, Hkv, D, page, 4, seed=2).clean()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(pools[0], buf, held)
        held.add_(1)
    held.copy_(lens)
    for i in range(steps):
        buf.copy_(x[i])
        graph.replay()
        want = step(pools[1], x[i], lens + i)
        assert torch.equal(out, want)
    assert all(torch.equal(a, b) for a, b in zip(pools[0].args(), pools[1].args()))


def test_calls_on_parameters_without_autograd_and_in_place_versions():
    pool = Pool(1, 1, 64, 16, 2, seed=3).clean()
    x = torch.randn((1, 1, 5, 64), device="cuda").to(BF).requires_grad_()
    w = weights(64)[0].requires_grad_()
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    with torch.no_grad():
        q = bsa.nsa_cache4_append(x, x, *pool.args(), n, q=x, q_weight=w, k_weight=w)
        assert not q.requires_grad
        bsa.nsa_cache4_decode(x[:, :, :1], *pool.args(), n + 5)
    d = x.detach()[:, :, :1].contiguous()
    out, lse = torch.empty_like(d), torch.empty((1, 1, 1), device="cuda")
    read = torch.empty((2, 1, 1, 5, 64), device="cuda", dtype=BF)
    p = torch.ones((), device="cuda", requires_grad=True)
    for saved, call in ((d, lambda: bsa.nsa_cache4_append(d, d, *pool.args(), n, q=d, q_out=d)),
                        (out, lambda: bsa.nsa_cache4_decode(d, *pool.args(), n + 1, out=out, lse=lse)),
                        (lse, lambda: bsa.nsa_cache4_decode(d, *pool.args(), n + 1, out=out, lse=lse)),
                        (read, lambda: bsa.nsa_cache4_read(*pool.args(), n + 5, 5, k_out=read[0], v_out=read[1]))):
        y = (p * saved).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


def test_two_threads_on_streams_of_their_own():
    """Calls of two host threads at once, each on its own tensors and stream, against the same calls one by one."""
    import threading

    def work(i):
        B, Hq, Hkv, D, page = (3, 8, 2, 64, 32) if i else (2, 16, 1, 128, 64)
        g = torch.Generator(device="cuda").manual_seed(i)
        x = torch.randn((B, 40, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
        q, k, v = x.transpose(1, 2).split([Hq, Hkv, Hkv], 1)
        w, f = weights(D), freqs(D)
        pool = Pool(B, Hkv, D, page, 30, seed=i).clean()
        lens = torch.tensor([700, 3, 40][:B], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        out = []
        for _ in range(20):
            q2, k2 = bsa.qk_norm_rope_forward(q, k, w[0], w[1], f)
            grads = bsa.qk_norm_rope_backward(q, k, q2, k2, w[0], w[1], f)
            q1 = bsa.nsa_cache4_append(k, v, *pool.args(), lens, inv_freq=f, q=q, q_weight=w[0], k_weight=w[1])
            out.append((q2, k2, *grads, q1, *bsa.nsa_cache4_read(*pool.args(), lens + 40, 50),
                        bsa.nsa_cache4_decode(q1[:, :, -1:], *pool.args(), lens + 40)))
        return out

    want, got, wrong = [work(i) for i in (0, 1)], [None, None], []
    torch.cuda.synchronize()

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = work(i)
        except BaseException as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for r, s in zip(a, b) for x, y in zip(r, s))
