"""GPU: the norm and rotation of query and key heads, and its gradients, against the float64 oracle.

Tolerances, in units of u = 2^-24 (half a step of fp32).  r = (mean x^2 + eps)^-1/2: at most 20 roundings of a sum of
squares, 2 of the mean, half of which reach the root, and 4 for the root's own 2 steps: 15 u.  An element of the
normalised row: 2 products, 17 u.  The rotated element x_a c - x_b s: the angle's fraction of a turn is off by 2^-25 of a
half-turn, 2 u; sine and cosine 2 steps, 4 u; the factor, product and sum 3 u: 26 u of |x_a| + |x_b| at most, taken as
32 u = 2^-19; then the result's rounding.

Backward: g as the rotation (9 u of |dy_a| + |dy_b|), h = r x (16 u); g w h: 27 u, their mean 22 more; dx = r (g w -
h mean): 15 + 16 + 27 + 22 and four more operations: under 128 u = 2^-17 of the sums that ``oracle.rows`` gives.  dw: a
row's product 26 u, and the roundings of its sum: at most 8 rows of a thread, 5 shuffles, 8 warps, 64 lanes and the
blocks of a tensor over 64: 2^-17 of the sum of magnitudes holds up to 1100 blocks.
"""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import BsaError, bsa
from oracle import rows as orows

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


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


def half_step(t):
    return torch.finfo(t).eps / 2


def host(t):
    return t.detach().double().cpu().numpy()


def freqs(rotary, base=10000.0):
    return bsa.rope_frequencies(rotary, base, device="cuda")[0] if rotary else None


def make(B, Hq, Hkv, T, D, dtype=BF, layout="heads", seed=0, size=1.0):
    """q, k in one of the layouts that a program holds them in."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "heads":
        return tuple((torch.randn((B, h, T, D), generator=g, device="cuda") * size).to(dtype) for h in (Hq, Hkv))
    x = (torch.randn((B, T, Hq + 2 * Hkv, D), generator=g, device="cuda") * size).to(dtype).transpose(1, 2)
    return x[:, :Hq], x[:, Hq:Hq + Hkv]  # "fused"


def check_forward(q, k, wq, wk, f, pos=None, got=None, **kw):
    got = got or bsa.qk_norm_rope_forward(q, k, wq, wk, f, positions=pos, **kw)
    B, T = q.shape[0], q.shape[2]
    p = np.broadcast_to(np.arange(T), (B, T)) if pos is None else np.broadcast_to(host(pos), (B, T))
    il, scale, eps = kw.get("interleaved", False), kw.get("rotary_scale", 1.0), kw.get("eps", 1e-6)
    fr = np.zeros(0) if f is None else host(f)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        want, e = orows.forward(host(x), None if w is None else host(w), p, fr, il, scale, eps)
        assert y.shape == x.shape and y.dtype == x.dtype and y.is_contiguous()
        assert (np.abs(host(y) - want) <= half_step(x.dtype) * np.abs(want) + (1 + half_step(x.dtype)) * 2.0 ** -19 * e
                + 1e-37).all()
    return got


def check_backward(q, k, wq, wk, f, pos=None, seed=1, got=None, grads=None, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dq, dk = grads or (torch.randn(x.shape, generator=g, device="cuda").to(x.dtype) for x in (q, k))
    got = got or bsa.qk_norm_rope_backward(q, k, dq, dk, wq, wk, f, positions=pos, **kw)
    B, T = q.shape[0], q.shape[2]
    p = np.broadcast_to(np.arange(T), (B, T)) if pos is None else np.broadcast_to(host(pos), (B, T))
    il, scale, eps = kw.get("interleaved", False), kw.get("rotary_scale", 1.0), kw.get("eps", 1e-6)
    fr = np.zeros(0) if f is None else host(f)
    for x, dy, w, dx, dw in ((q, dq, wq, got[0], got[2]), (k, dk, wk, got[1], got[3])):
        want, want_w, ex, ew = orows.backward(host(x), host(dy), None if w is None else host(w), p, fr, il, scale, eps)
        h = half_step(x.dtype)
        assert dx.shape == x.shape and dx.dtype == x.dtype
        assert (np.abs(host(dx) - want) <= h * np.abs(want) + (1 + h) * 2.0 ** -17 * ex + 1e-37).all()
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == F32 and (np.abs(host(dw) - want_w) <= 2.0 ** -17 * ew).all()
    return got


def weights(D, dtype=F32, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple((1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2))


@pytest.mark.parametrize("D", list(range(16, 129, 16)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_head_size(D, dtype):
    for B, Hq, Hkv, T, layout in ((2, 3, 1, 37, "heads"), (3, 2, 2, 5, "fused"), (1, 1, 1, 1, "heads")):
        q, k = make(B, Hq, Hkv, T, D, dtype, layout, seed=D)
        for il in (False, True):
            kw = {"interleaved": il, "rotary_scale": 1.25, "eps": 1e-4}
            check_forward(q, k, *weights(D), freqs(D), **kw)
            check_backward(q, k, *weights(D), freqs(D), **kw)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotary", [(64, 0), (64, 16), (64, 48), (96, 32), (128, 112), (80, 80), (48, 16)])
def test_part_of_the_head(D, rotary, interleaved):
    q, k = make(2, 5, 2, 19, D, BF, seed=rotary)
    for w in (weights(D), (None, None), (weights(D)[0], None), (None, weights(D)[1])):
        check_forward(q, k, *w, freqs(rotary), interleaved=interleaved)
        check_backward(q, k, *w, freqs(rotary), interleaved=interleaved)


@pytest.mark.parametrize("B,Hq,Hkv,T,D", [(1, 32, 2, 1, 128), (128, 64, 4, 1, 128), (7, 16, 16, 33, 64), (2, 32, 2, 2048, 128),
                                          (1, 1, 1, 5000, 16), (3, 40, 8, 300, 80), (64, 12, 1, 31, 32)])
def test_sizes_and_layouts(B, Hq, Hkv, T, D):
    for layout in ("heads", "fused"):
        q, k = make(B, Hq, Hkv, T, D, BF, layout, seed=T)
        check_forward(q, k, *weights(D), freqs(D))
        dq, dk, *_ = check_backward(q, k, *weights(D), freqs(D))
        # gradients lie as the tensors do
        if layout == "fused" and Hq > 1 and T > 1:
            assert dq.transpose(1, 2).is_contiguous()
        elif layout == "heads":
            assert dq.is_contiguous() and dk.is_contiguous()


def test_weights_of_either_type():
    q, k = make(2, 4, 2, 9, 64)
    check_forward(q, k, *weights(64, BF), freqs(64))
    check_backward(q, k, *weights(64, BF), freqs(64))
    mixed = weights(64)[0], weights(64, BF)[1]
    check_forward(q, k, *mixed, freqs(64))
    check_backward(q, k, *mixed, freqs(64))


def test_positions():
    """Given ones, shared over the batch or not, far and negative; angles keep their bits."""
    q, k = make(3, 2, 1, 11, 64, F32)
    g = torch.Generator().manual_seed(0)
    for pos in (torch.randint(-2 ** 31, 2 ** 31, (3, 11), generator=g), torch.randint(0, 2 ** 20, (11,), generator=g),
                torch.full((3, 11), 2 ** 31 - 1), torch.full((11,), -2 ** 31)):
        for kind in (torch.int32, torch.int64):
            check_forward(q, k, *weights(64), freqs(64), pos.to(kind).cuda())
        check_backward(q, k, *weights(64), freqs(64), pos.cuda())


def test_strides_of_every_kind():
    """Rows that follow each other oddly, broadcast inputs, rows that have to be copied, misaligned views."""
    B, H, T, D = 2, 4, 6, 64
    x = torch.randn((B, T, H, 3, D), device="cuda").to(BF)
    q, k = x[:, :, :, 0].transpose(1, 2), x[:, :, ::2, 2].transpose(1, 2)
    check_forward(q, k, *weights(D), freqs(D))
    check_backward(q, k, *weights(D), freqs(D))
    one = torch.randn((1, 1, T, D), device="cuda").to(BF).expand(B, H, T, D)  # broadcast over batch and heads
    same = torch.randn((B, H, 1, D), device="cuda").to(BF).expand(B, H, T, D)
    for q, k in ((one, same), (same, one)):
        check_forward(q, k, *weights(D), freqs(D))
        check_backward(q, k, *weights(D), freqs(D), grads=(k, q))
    cols = torch.randn((B, H, D, T), device="cuda").to(BF).transpose(2, 3)  # a row's elements apart
    flat = torch.randn(B * H * T * D + 1, device="cuda").to(BF)[1:].view(B, H, T, D)  # 2 bytes off
    odd = torch.randn((B, H, T, D + 4), device="cuda").to(BF)[..., :D]  # rows of 136 bytes
    rev = torch.randn((B, H, D, T), device="cuda").transpose(2, 3)
    check_forward(cols, flat, *weights(D), freqs(D))
    check_backward(flat, odd, *weights(D), freqs(D), grads=(cols, flat))
    check_forward(rev, rev, *weights(D), freqs(D))
    w = torch.randn(D + 1, device="cuda")[1:]
    f = torch.cat([torch.zeros(1, device="cuda"), freqs(D)])[1:]  # 4 bytes off
    check_forward(odd, cols, w, w, f)
    check_forward(odd, cols, torch.randn(2 * D, device="cuda")[::2], w, f)


def test_magnitudes_and_zero_rows():
    q, k = make(2, 3, 2, 7, 64, F32)
    for size in (2.0 ** -40, 2.0 ** 40):
        check_forward(q * size, k * size, *weights(64), freqs(64), eps=1e-30)
    q[0, 1, 3] = 0.0
    k[:, :, 2] = 0.0
    check_forward(q, k, *weights(64), freqs(64))
    check_backward(q, k, *weights(64), freqs(64))
    check_forward(q, k, *(torch.zeros_like(w) for w in weights(64)), freqs(64))


def test_other_rows_do_not_see_a_bad_one():
    q, k = make(1, 4, 4, 40, 128)
    want = bsa.qk_norm_rope_forward(q, k, *weights(128), freqs(128))
    q2, k2 = q.clone(), k.clone()
    q2[0, 1, 7, 3], q2[0, 2, 8] = float("nan"), float("inf")
    k2[0, 0, 0, 0] = float("-inf")
    got = bsa.qk_norm_rope_forward(q2, k2, *weights(128), freqs(128))
    keep_q, keep_k = (torch.ones((4, 40), dtype=torch.bool, device="cuda") for _ in range(2))
    keep_q[1, 7] = keep_q[2, 8] = keep_k[0, 0] = False
    assert torch.equal(got[0][0][keep_q], want[0][0][keep_q]) and torch.equal(got[1][0][keep_k], want[1][0][keep_k])


def test_results_given_and_in_other_streams():
    q, k = make(2, 8, 2, 100, 64, layout="fused")
    w, f = weights(64), freqs(64)
    want = bsa.qk_norm_rope_forward(q, k, *w, f)
    out = torch.empty(q.shape, dtype=BF, device="cuda"), torch.empty(k.shape, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bsa.qk_norm_rope_forward(q, k, *w, f, q_out=out[0], k_out=out[1], stream=s)
    s.synchronize()
    assert got[0] is out[0] and got[1] is out[1]
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    first = bsa.qk_norm_rope_backward(q, k, *want, *w, f)
    for _ in range(3):
        again = bsa.qk_norm_rope_backward(q, k, *want, *w, f, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    need = bsa.qk_norm_rope_backward_workspace_size(2, 8, 2, 100, 64)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every float
    again = bsa.qk_norm_rope_backward(q, k, *want, *w, f, workspace=ws[:need])
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and (ws[need:] == 0xFF).all()
    with pytest.raises(BsaError) as e:
        bsa.qk_norm_rope_backward(q, k, *want, *w, f, workspace=ws[: need - 256])
    assert e.value.status == 9


def test_autograd():
    """Through the selection attention, from one fused projection, against differences and against the raw calls."""
    B, Hq, Hkv, T, D = 1, 4, 2, 64, 32
    x = torch.randn((B, T, Hq + 2 * Hkv, D), device="cuda", dtype=F32)
    wq, wk = (w.requires_grad_() for w in weights(D))
    f = freqs(D)

    def loss(x, wq, wk, c):
        q, k, _ = x.transpose(1, 2).split([Hq, Hkv, Hkv], 1)
        q, k = bsa.qk_norm_rope(q, k, wq, wk, f, rotary_scale=1.1)
        return (q * c[0]).sum().double() + (k * c[1]).sum().double()

    g = torch.Generator(device="cuda").manual_seed(3)
    c = tuple(torch.randn((B, h, T, D), generator=g, device="cuda") for h in (Hq, Hkv))
    x.requires_grad_()
    loss(x, wq, wk, c).backward()
    q, k, _ = (t.detach() for t in x.transpose(1, 2).split([Hq, Hkv, Hkv], 1))
    dq, dk, dwq, dwk = bsa.qk_norm_rope_backward(q, k, *c, wq.detach(), wk.detach(), f, rotary_scale=1.1)
    got = x.grad.transpose(1, 2)
    assert torch.equal(got[:, :Hq], dq) and torch.equal(got[:, Hq:Hq + Hkv], dk) and not got[:, Hq + Hkv:].any()
    assert torch.equal(wq.grad, dwq) and torch.equal(wk.grad, dwk)
    check_backward(q, k, wq.detach(), wk.detach(), f, got=(dq, dk, dwq, dwk), grads=c, rotary_scale=1.1)
    # bf16 weights get bf16 gradients; what needs none gets none
    wb = wq.detach().to(BF).requires_grad_()
    q = q.to(BF).requires_grad_()
    out, _ = bsa.qk_norm_rope(q, k.to(BF), wb, wb.detach(), f)
    out.float().square().sum().backward()
    assert wb.grad.dtype == BF and q.grad.dtype == BF and torch.isfinite(q.grad).all()
    # an expanded gradient, and only one of the two results used
    q2 = q.detach().requires_grad_()
    bsa.qk_norm_rope(q2, k.to(BF), wb.detach(), wb.detach(), f)[0].sum().backward()
    check_backward(q2.detach(), k.to(BF), wb.detach(), wb.detach(), f,
                   got=(q2.grad, torch.zeros_like(k, dtype=BF), *bsa.qk_norm_rope_backward(
                       q2.detach(), k.to(BF), torch.ones_like(q2), torch.zeros_like(k, dtype=BF), wb.detach(),
                       wb.detach(), f)[2:]), grads=(torch.ones_like(q2), torch.zeros_like(k, dtype=BF)))


def test_gradient_against_differences():
    """Slopes of sum(y c) in fp32 along the gradient, of all tensors and of each alone.  y is off by 2^-19 of its reach,
    so a difference over 2 h by at most sum(2^-19 e |c|) / h; third derivatives along a unit direction are about
    |c| / |x|^2 of a row's norm |x| (5.7 here), under 100 with room, times h^2 / 6."""
    B, H, T, D = 1, 2, 8, 32
    q, k = make(B, H, H, T, D, F32, seed=7)
    wq, wk = weights(D)
    f = freqs(D)
    g = torch.Generator(device="cuda").manual_seed(9)
    c = [torch.randn(q.shape, generator=g, device="cuda") for _ in range(2)]
    grads = bsa.qk_norm_rope_backward(q, k, *c, wq, wk, f)
    h = 2.0 ** -6
    for only in (None, 0, 1, 2, 3):
        v = [t if only in (None, i) else torch.zeros_like(t) for i, t in enumerate(grads)]
        size = sum(t.square().sum() for t in v).sqrt()
        v = [t / size for t in v]
        up, down = (bsa.qk_norm_rope_forward(*(t + s * u for t, u in zip((q, k, wq, wk), v)), f) for s in (h, -h))
        got = sum((((a - b).double() / (2 * h)) * cc).sum() for a, b, cc in zip(up, down, c))
        want = sum((a.double() * b).sum() for a, b in zip(grads, v))
        noise = 0.0
        for x, w, cc in ((q, wq, c[0]), (k, wk, c[1])):
            _, e = orows.forward(host(x), host(w), np.arange(T)[None], host(f), False, 1.0, 1e-6)
            noise += (e * np.abs(host(cc))).sum() * 2.0 ** -19 / h
        assert abs(float(got - want)) <= noise + 100 * h * h


def test_captured_training_steps():
    """Forward and backward in one graph, replayed on new inputs, beside an eager call and on two streams at once."""
    B, Hq, Hkv, T, D = 2, 8, 2, 128, 64
    f = freqs(D)
    eager = [t.requires_grad_() for t in (*make(B, Hq, Hkv, T, D), *weights(D))]
    graphs = []
    for seed in (1, 2):
        leaves = [t.requires_grad_() for t in (*make(B, Hq, Hkv, T, D, seed=seed), *weights(D, seed=seed))]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(2):
                outs = bsa.qk_norm_rope(*leaves, f)
                torch.autograd.grad([o.float().square().sum() for o in outs], leaves)
                del outs
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = bsa.qk_norm_rope(*leaves, f)
            grads = torch.autograd.grad([o.float().square().sum() for o in outs], leaves)
        graphs.append((graph, leaves, [o.detach() for o in outs], grads))
    with torch.no_grad():
        for _, leaves, _, _ in graphs:
            for a, b in zip(leaves, eager):
                a.copy_(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (graph, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    outs = bsa.qk_norm_rope(*eager, f)
    grads = torch.autograd.grad([o.float().square().sum() for o in outs], eager)
    torch.cuda.synchronize()
    for _, _, o, g in graphs:
        assert all(torch.equal(a, b) for a, b in zip(o, outs)) and all(torch.equal(a, b) for a, b in zip(g, grads))


def test_what_is_written_in_place_is_known_to_autograd():
    q, k = make(1, 2, 1, 4, 32)
    out = torch.empty_like(q), torch.empty_like(k)
    w = torch.ones((), device="cuda", requires_grad=True)
    y = (w * out[0]).sum()
    bsa.qk_norm_rope_forward(q, k, q_out=out[0], k_out=out[1])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_long_and_many():
    """More than 2^31 bytes of rows, and more blocks than a grid's second axis: sampled rows."""
    B, Hq, Hkv, T, D = 1, 34, 1, 1 << 18, 128
    q, k = make(B, Hq, Hkv, T, D)
    w, f = weights(D), freqs(D)
    got = bsa.qk_norm_rope_forward(q, k, *w, f)
    grads = bsa.qk_norm_rope_backward(q, k, *got, *w, f)
    at = torch.tensor([0, 1, 12345, T // 2, T - 33, T - 1], device="cuda")
    pick = lambda t: t[:, :, at].contiguous()  # noqa: E731
    check_forward(pick(q), pick(k), *w, f, at, got=(pick(got[0]), pick(got[1])))
    dq, dk, _, _ = bsa.qk_norm_rope_backward(pick(q), pick(k), pick(got[0]), pick(got[1]), *w, f, at)
    assert torch.equal(pick(grads[0]), dq) and torch.equal(pick(grads[1]), dk)
    # the weights' gradients: the same sums in 64 bits, from the fp32 rows of torch (each off by 2^-20 of its terms)
    h = k.double() * (k.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    a = torch.arange(T, device="cuda").double()[:, None] * f.double()
    c, s = torch.cos(a), torch.sin(a)
    y0, y1 = got[1].double()[..., :64], got[1].double()[..., 64:]
    g = torch.cat([y0 * c + y1 * s, y1 * c - y0 * s], -1)
    terms = torch.cat([y0.abs() + y1.abs()] * 2, -1) * h.abs()
    assert ((grads[3].double() - (g * h).sum((0, 1, 2))).abs() <= 2.0 ** -16 * terms.sum((0, 1, 2))).all()
