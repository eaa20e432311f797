"""GPU: the selection operators at the borders of their launch rules and of
their documented ranges, against the float64 oracle (tolerances as in
``test_gpu_nsa_cache.py``)."""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from oracle import cache as ocache
from test_gpu_nsa_cache import BF, U, Pool, check_append, check_decode

pytestmark = pytest.mark.gpu


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


# ------------------------------------------------------------------- append


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_around_every_warp_of_threads(D, page):
    """As many new tokens as make the units of a page one more, one less or exactly what a number of warps takes."""
    for n in (2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129):
        check_append(2, 2, 1, n, D, page, [0, 3 * page - 2], seed=n + D + page)


@pytest.mark.parametrize("old", [0.0, 2.0 ** -140, 2.0 ** -97, 2.0 ** -96])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -110, 2.0 ** -104, 1.0])
def test_append_behind_tokens_of_a_scale_of_zero(old, scale):
    """A page begun elsewhere, all of whose values are zero or next to it: what is appended keeps its value."""
    pool = Pool(2, 1, 64, 32, 2, seed=2).clean()
    pool.ks.fill_(old)
    pool.vs.fill_(old)
    check_append(2, 2, 1, 7, 64, 32, [3, 30], rotary=0, scale=scale, dtype=torch.float32, pool=pool)
    for c in (pool.k, pool.v):
        assert ((c & 127) != 127).all()


# ------------------------------------------------------------------- decode


@pytest.mark.parametrize("D,page", [(16, 16), (64, 64), (128, 32), (32, 128)])
@pytest.mark.parametrize("short", [0, 1, 15, 16, 127, 128, 32 * 128 + 1])
def test_decode_of_the_longest_sequences(D, page, short):
    """Tokens up to the largest number that a table may hold (the next to 2^31), almost all on pages that the table does
    not have; without those the sequence is a short one over the same pages."""
    max_pages = (2 ** 31 - 1) // page
    n = max_pages * page - short
    last = (n - 1) // page
    held = sorted({0, 5, last // 2, last - 32, last - 1, last})
    pool = Pool(1, 1, D, page, len(held), seed=D + short).clean()
    dense = pool.table
    q = torch.randn((1, 3, 1, D), generator=torch.Generator().manual_seed(short)).to(torch.bfloat16).cuda()
    tokens = (len(held) - 1) * page + (n - 1) % page + 1
    pool.table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    pool.table[0, held] = dense[0]
    args = pool.args()
    pool.table = dense
    idx = torch.tensor(held, dtype=torch.int32, device="cuda").view(1, 1, 1, -1)
    for length in (n, 2 ** 31 - 1) if short == 0 else (n,):
        lt = torch.tensor([length], dtype=torch.int32, device="cuda")
        for pick in (None, idx):
            out, lse = bsa.nsa_select_decode(q, *args, lt, block_idx=pick, return_lse=True)
            torch.cuda.synchronize()
            check_decode(out, lse, q, pool, [tokens], None)


def test_decode_of_the_least_lengths():
    pool = Pool(2, 1, 64, 32, 3, seed=1).clean()
    q = torch.randn((2, 2, 1, 64)).to(torch.bfloat16).cuda()
    lt = torch.tensor([-2 ** 31, -1], dtype=torch.int32, device="cuda")
    for pick in (None, torch.zeros((2, 1, 1, 2), dtype=torch.int32, device="cuda")):
        out, lse = bsa.nsa_select_decode(q, *pool.args(), lt, block_idx=pick, return_lse=True)
        assert not out.any() and (lse == -1.0e9).all()


@pytest.mark.parametrize("below", [14, 20, 25, 28])
@pytest.mark.parametrize("D,page,S", [(64, 64, 0), (64, 64, 32), (128, 32, 0), (32, 16, 32)])
def test_decode_with_most_of_the_weight_on_a_token_of_no_value(D, page, S, below):
    """A first token of probability next to 1 and values next to 0; the result is the sum of the many others, each of
    probability near 2^-below, on pages whose scales differ by up to 2^3.

    A probability p of the largest P is off by 2^-11 p, or by 2^-36 P where that is more, which a page's scale of 2^-3
    of the accumulator's may make 2^-33 P; scores and sums are in fp32 (U an operation, one a product of 16 tokens and
    16 to join the parts), the result is rounded to bf16.
    """
    pages, G = 32, 4
    r = np.random.default_rng(below + D)
    pool = Pool(1, 1, D, page, pages, seed=below)
    k = ocache.VALUES[r.integers(0, 0x38, (pool.pages, 1, page, D))]  # 0 .. 0.9375
    k *= np.where(r.random(k.shape) < 0.5, 1.0, -1.0)
    at = pool.table[0].cpu().numpy()
    k[at[0], 0, 0, :] = 0.0
    k[..., 0], k[at[0], 0, 0, 0] = 0.0, 32.0
    v = r.integers(0, 0x7F, (pool.pages, 1, page, D)).astype(np.uint8)
    v[at[0], 0, 0] = 0x01  # 2^-9
    pool.k.copy_(torch.from_numpy(ocache.e4m3_encode(k)))
    pool.v.copy_(torch.from_numpy(v))
    pool.ks.fill_(0.25)
    q = 0.02 * torch.randn((1, G, 1, D), generator=torch.Generator().manual_seed(below))
    q[..., 0] = below * np.log(2.0) * D ** 0.5 / 8.0
    q = q.to(torch.bfloat16).cuda()
    n = pages * page - 3
    idx = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, 1, 1, -1)[..., :S] if S else None
    out, lse = bsa.nsa_select_decode(q, *pool.args(), torch.tensor([n], device="cuda"), block_idx=idx, return_lse=True)
    torch.cuda.synchronize()
    p = pool.copy()
    want, wl, sums = ocache.decode(q.double().cpu().numpy(), *p, [n], None if idx is None else idx.cpu().numpy())
    small = 2.0 ** -33 * sums["v"] if S == 0 else 2.0 ** -36 * sums["v"]
    bound = (1 + BF) * (2.0 ** -11 * sums["p"] + U * (sums["e"] + 2 * (n / 16 + 16) * sums["p"]) + small)
    worst = (np.abs(out.double().cpu().numpy() - want) / (bound + BF * np.abs(want))).max()
    assert worst <= 1, f"{worst:.2f} times its bound"
    assert (np.abs(lse.double().cpu().numpy() - wl) <= U * (sums["lse"] + n + 8) + 2.0 ** -23 * np.abs(wl)).all()


@pytest.mark.parametrize("S", [0, 3])
@pytest.mark.parametrize("e", [14, 18, 20, 22, 24, 40, 100])
def test_decode_scores_of_any_magnitude_are_finite(S, e):
    """Scores up to and past the numbers between which an fp32 has no room for one: the largest has all the weight."""
    B, D, page = 1, 64, 16
    pool = Pool(B, 1, D, page, 40, seed=e).clean()
    q = (torch.randn((B, 3, 1, D), generator=torch.Generator().manual_seed(e)) * 2.0 ** e).to(torch.bfloat16).cuda()
    idx = torch.tensor([3, 0, 39], dtype=torch.int32, device="cuda").view(1, 1, 1, 3) if S else None
    lt = torch.tensor([630], device="cuda")
    out, lse = bsa.nsa_select_decode(q, *pool.args(), lt, block_idx=idx, return_lse=True)
    check_decode(out, lse, q, pool, [630], idx)


# ----------------------------------------------------------------- autograd


def test_attention_beyond_the_backwards_limits():
    """More (batch, kv head) pairs than the backward takes: the forward alone runs, a graph is not begun."""
    B, T, D = 65536, 16, 16
    q, k, v = (torch.randn((B, 1, T, D), device="cuda").to(torch.bfloat16) for _ in range(3))
    idx = torch.zeros((B, 1, T, 1), dtype=torch.int32, device="cuda")
    want = bsa.nsa_select_forward(q, k, v, idx, 16)
    assert torch.equal(bsa.nsa_select_attention(q, k, v, idx, 16), want)
    for leaf in (q, k, v):
        leaf.requires_grad_()
        with pytest.raises(bsa.BsaError, match="no gradients for"):
            bsa.nsa_select_attention(q, k, v, idx, 16)
        with torch.no_grad():
            assert torch.equal(bsa.nsa_select_attention(q, k, v, idx, 16), want)
        leaf.requires_grad_(False)


def test_cache_calls_on_parameters_without_autograd():
    """Weights require gradients in a serving program too: under no_grad the calls are those on detached tensors."""
    pool = Pool(1, 1, 64, 16, 2, seed=3).clean()
    x = torch.randn((1, 1, 5, 64), device="cuda").to(torch.bfloat16).requires_grad_()
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    with torch.no_grad():
        q = bsa.nsa_cache_append(x, x, *pool.args(), n, q=x)
        a = bsa.nsa_select_decode(x[:, :, :1], *pool.args(), n + 5)
    d = x.detach()
    assert torch.equal(q, d) and not q.requires_grad
    assert torch.equal(a, bsa.nsa_select_decode(d[:, :, :1], *pool.args(), n + 5))


def test_what_a_call_writes_in_place_is_known_to_autograd():
    """A graph that saved a tensor which a call then overwrites refuses its backward, as after torch's own in-place
    operations; what a call only reads stays usable."""
    pool = Pool(1, 1, 64, 16, 2, seed=4).clean()
    x = torch.randn((1, 1, 1, 64), device="cuda").to(torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(x), torch.empty((1, 1, 1), device="cuda")
    w = torch.ones((), device="cuda", requires_grad=True)

    def backward_after(saved, call):
        y = (w * saved).sum()
        call()
        y.backward()

    append = lambda: bsa.nsa_cache_append(x, x, *pool.args(), n, q=x, q_out=x)  # noqa: E731
    decode = lambda: bsa.nsa_select_decode(x, *pool.args(), n + 1, out=out, lse=lse)  # noqa: E731
    for saved, call in ((x, append), (pool.ks, append), (pool.vs, append), (out, decode), (lse, decode)):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            backward_after(saved, call)
    backward_after(x, decode)
    backward_after(pool.ks, decode)
    with torch.inference_mode():
        y = torch.randn((1, 1, 1, 64), device="cuda").to(torch.bfloat16)
        assert bsa.nsa_cache_append(y, y, *pool.args(), n, q=y, q_out=y) is y
