"""GPU: gradients of the NSA selection attention against the float64 oracle.

Tolerances.  p and dS are rounded once to bf16 (relative 2^-8) before their
products, and the results once more; the sums run in fp32 on the tensor cores,
taken as U = 2^-22 per operation (their aligned additions may truncate).  So
    |dq error| <= 2^-8 sum |dS k| + U (sum e |k| + n sum |dS k|) + 2^-8 |dq|
with e the steps by which an evaluation in fp32 may move dS (the oracle's
``sums``), n the number of terms, and the same for dk and dv; the second
rounding acts on the already perturbed value, hence the factor 1 + 2^-8 on the
first two terms.
"""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa, workloads
from oracle import nsa as onsa

pytestmark = pytest.mark.gpu
U, BF = 2.0 ** -22, 2.0 ** -8


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


def inputs(B, Hq, Hkv, T, D, bs, S, seed):
    """Inputs and the forward's results, all on the GPU."""
    q, k, v, idx = (t.cuda() for t in workloads.nsa_inputs(B, Hq, Hkv, T, D, bs, S, seed=seed))
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16).cuda()
    return q, k, v, idx, dout


def forward(q, k, v, idx, bs):
    """out (bf16) and lse (fp32) of the float64 oracle (indices past the sequence dropped)."""
    n = q.shape[2] // bs
    ok = torch.where(idx < n, idx, -1)
    out, lse = onsa.nsa_select_forward(*(t.double().cpu().numpy() for t in (q, k, v)), ok.cpu().numpy(), bs)
    return torch.from_numpy(out).to(torch.bfloat16).cuda(), torch.from_numpy(lse).float().cuda()


def check(got, q, k, v, idx, out, lse, dout, bs):
    n = q.shape[2] // bs
    ok = torch.where(idx < n, idx, -1)
    h = [t.double().cpu().numpy() for t in (q, k, v, out, lse, dout)]
    *want, sums = onsa.nsa_select_backward(h[0], h[1], h[2], ok.cpu().numpy(), h[3], h[4], h[5], bs)
    terms = {"dq": idx.shape[-1] * bs, "dk": q.shape[2] * q.shape[1] // k.shape[1]}
    terms["dv"] = terms["dk"]
    for name, x, r in zip(("dq", "dk", "dv"), got, want):
        assert x.dtype == torch.bfloat16 and tuple(x.shape) == r.shape
        x = x.double().cpu().numpy()
        bound = (1 + BF) * (BF * sums[name] + U * (sums[name + "_e"] + terms[name] * sums[name])) + BF * np.abs(r)
        worst = (np.abs(x - r) - bound).max()
        assert np.isfinite(x).all() and worst <= 1e-30, f"{name}: {worst:.3e} over its bound"


def run(B, Hq, Hkv, T, D, bs, S, seed=0, change=None):
    q, k, v, idx, dout = inputs(B, Hq, Hkv, T, D, bs, S, seed)
    if change is not None:
        idx = change(idx)
    out, lse = forward(q, k, v, idx, bs)
    got = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    torch.cuda.synchronize()
    check(got, q, k, v, idx, out, lse, dout, bs)
    return got


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_every_head_dim_and_block_size(D, bs):
    run(1, 8, 2, 256, D, bs, 3, seed=D + bs)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (5, 1), (7, 1), (16, 1), (12, 1), (16, 8), (15, 1)])
def test_group_sizes(Hq, Hkv):
    run(2, Hq, Hkv, 192, 64, 64, 2, seed=Hq)
    run(1, Hq, Hkv, 128, 128, 32, 4, seed=Hq + 1)


@pytest.mark.parametrize("T,bs,S", [(16, 16, 1), (64, 64, 1), (128, 128, 32), (64, 64, 7), (448, 64, 32), (1040, 16, 5)])
def test_lengths_and_slots(T, bs, S):
    run(1, 4, 2, T, 64, bs, S, seed=T + S)


def odd_rows(idx, n_blk):
    """Empty rows, rows of future blocks only, repeats, block 0 everywhere else, out-of-range entries."""
    a = idx.clone()
    T = a.shape[2]
    a[:, :, : T // 8] = -1
    a[:, :, T // 8: T // 4, 0] = n_blk - 1
    a[:, :, T // 8: T // 4, 1:] = -1
    a[:, :, T // 4:, 1] = 0
    a[:, :, T // 2:, -1] = a[:, :, T // 2:, 0]
    a[:, :, -3:, 2] = n_blk + 5
    return a


@pytest.mark.parametrize("D,bs,Hq,Hkv", [(128, 64, 16, 1), (64, 64, 4, 2), (32, 32, 6, 2), (128, 128, 3, 1)])
def test_empty_rows_repeats_and_a_block_every_row_reads(D, bs, Hq, Hkv):
    T = 768  # block 0's list is longer than a work item
    dq, dk, dv = run(1, Hq, Hkv, T, D, bs, 5, seed=D, change=lambda i: odd_rows(i, T // bs))
    assert not dq[:, :, : T // 8].any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 128])
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (16, 1), (16, 2), (10, 2)])
def test_lists_of_several_items_at_every_block_size(D, bs, Hq, Hkv):
    T = 1024
    run(1, Hq, Hkv, T, D, bs, 6, seed=D + bs + Hq, change=lambda i: odd_rows(i, T // bs))


@pytest.mark.parametrize("D,bs,Hq", [(64, 16, 8), (128, 16, 3), (64, 32, 3), (128, 32, 16), (64, 128, 8), (128, 128, 5)])
def test_a_block_beside_garbage(D, bs, Hq):
    """Every other block is selected by nobody and holds NaN and infinities: nothing of it is read."""
    q, k, v, idx, dout = inputs(1, Hq, 1, 1024, D, bs, 4, seed=D + bs)
    idx = torch.where(idx >= 0, idx // 2 * 2, idx)
    out, lse = forward(q, k, v, idx, bs)
    clean = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    for t, x in ((k, float("nan")), (v, float("inf"))):
        t.view(1, 1, -1, 2, bs, D)[:, :, :, 1] = x
    got = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, clean))


def test_blocks_no_row_reads_get_zero():
    T, bs = 512, 64
    only = lambda idx: torch.full_like(idx, -1).index_fill_(3, torch.tensor([1], device="cuda"), 2)  # noqa: E731
    dq, dk, dv = run(1, 4, 2, T, 64, bs, 3, change=only)
    for x in (dk, dv):
        assert not x[:, :, : 2 * bs].any() and not x[:, :, 3 * bs:].any() and x[:, :, 2 * bs: 3 * bs].any()
    assert not dq[:, :, : 2 * bs].any()
    none = run(1, 4, 2, T, 64, bs, 3, change=lambda idx: torch.full_like(idx, -1))
    assert not any(x.any() for x in none)


def test_garbage_behind_the_mask_stays_out():
    """Blocks that no row selects, and rows that select none, may hold infinities and NaN."""
    B, Hq, Hkv, T, D, bs, S = 1, 8, 1, 256, 64, 64, 2
    q, k, v, idx, dout = inputs(B, Hq, Hkv, T, D, bs, S, 3)
    idx[:, :, :, 1:] = -1  # the current block only
    idx[:, :, 128:192] = -1  # block 2 is nobody's
    out, lse = forward(q, k, v, idx, bs)
    clean = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    kb, vb, qb, db = k.clone(), v.clone(), q.clone(), dout.clone()
    kb[:, :, 128:192], vb[:, :, 128:192] = float("nan"), float("inf")
    qb[:, :, 128:192], db[:, :, 128:192] = float("nan"), float("inf")
    got = bsa.nsa_select_backward(qb, kb, vb, idx, out, lse, db, bs)
    for x, y in zip(got, clean):
        assert torch.equal(x, y)


def test_gradient_agrees_with_differences():
    """d/de of sum(dout * forward(. + e w)) by central differences of the float64 forward."""
    B, Hq, Hkv, T, D, bs, S = 1, 4, 2, 96, 32, 32, 2
    q, k, v, idx, dout = inputs(B, Hq, Hkv, T, D, bs, S, 11)
    out, lse = forward(q, k, v, idx, bs)
    grads = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    h = [t.double().cpu().numpy() for t in (q, k, v)]
    d, n = dout.double().cpu().numpy(), idx.cpu().numpy()
    rng = np.random.default_rng(5)
    for which, g in enumerate(grads):
        w = rng.standard_normal(h[which].shape)
        side = []
        for e in (1e-4, -1e-4):
            x = [y + e * w if j == which else y for j, y in enumerate(h)]
            side.append((onsa.nsa_select_forward(*x, n, bs)[0] * d).sum())
        want = (side[0] - side[1]) / 2e-4
        g = g.double().cpu().numpy()
        # every element within 2^-8 of its value twice over (operand and result roundings) plus out's own
        # rounding in delta, 2^-8 of dout.out times p: bounded through the norms
        slack = 4 * BF * np.linalg.norm(g) * np.linalg.norm(w)
        assert abs((g * w).sum() - want) <= slack


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    B, Hq, Hkv, T, D, bs, S = 2, 16, 1, 512, 128, 64, 8
    q, k, v, idx, dout = inputs(B, Hq, Hkv, T, D, bs, S, 7)
    idx[:, :, 64:, 1] = 0
    out, lse = bsa.nsa_select_forward(q, k, v, idx, bs, return_lse=True)
    first = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    second = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    for x in third:
        x.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_autograd_matches_the_calls_and_takes_strided_views():
    B, Hq, Hkv, T, D, bs, S = 1, 8, 2, 256, 64, 64, 4
    q, k, v, idx, dout = inputs(B, Hq, Hkv, T, D, bs, S, 9)
    # [B, T, H, D] memory seen as [B, H, T, D], as projections give it
    leaves = [t.transpose(1, 2).contiguous().requires_grad_() for t in (q, k, v)]
    got = bsa.nsa_select_attention(*(t.transpose(1, 2) for t in leaves), idx, bs)
    got.backward(dout.transpose(2, 3).contiguous().transpose(2, 3))
    out, lse = bsa.nsa_select_forward(q, k, v, idx, bs, return_lse=True)
    want = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    assert torch.equal(got, out)
    for leaf, w in zip(leaves, want):
        assert torch.equal(leaf.grad.transpose(1, 2), w)


def test_autograd_with_a_broadcast_key_head():
    """Expanded keys: autograd sums the heads' gradients."""
    T, D, bs = 128, 32, 32
    q, k, v, idx, dout = inputs(1, 4, 2, T, D, bs, 3, 13)
    k1 = k[:, :1].clone().requires_grad_()
    out = bsa.nsa_select_attention(q, k1.expand(-1, 2, -1, -1), v, idx, bs)
    out.backward(dout)
    o, lse = bsa.nsa_select_forward(q, k[:, :1].expand(-1, 2, -1, -1).contiguous(), v, idx, bs, return_lse=True)
    _, dk, _ = bsa.nsa_select_backward(q, k[:, :1].expand(-1, 2, -1, -1), v, idx, o, lse, dout, bs)
    assert torch.equal(k1.grad, dk.sum(1, keepdim=True))


@pytest.mark.parametrize("D,bs", [(64, 64), (32, 32)])
def test_a_captured_training_step_and_an_eager_one_on_another_stream(D, bs):
    """Forward and backward replayed from a graph on new inputs while other calls run beside it."""
    shape = (1, 8, 2, 512, D)
    batches = [inputs(*shape, bs, 4, seed=s) for s in (31, 32)]
    other = inputs(*shape, bs, 4, seed=33)

    def step(q, k, v, idx, do):
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        return torch.autograd.grad(bsa.nsa_select_attention(*leaves, idx, bs), leaves, do)

    want = [step(*b) for b in batches]
    beside = step(*other)
    static = [t.clone() for t in batches[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step(*static)
    side = torch.cuda.Stream()
    for b, w in zip(batches, want):
        for s, t in zip(static, b):
            s.copy_(t)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            again = step(*other)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(grads, w))
        assert all(torch.equal(x, y) for x, y in zip(again, beside))


@pytest.mark.parametrize("Hq,Hkv,T,D,bs,S", [(4, 2, 96, 32, 32, 2), (4, 1, 128, 64, 64, 2), (2, 1, 64, 128, 16, 3),
                                             (4, 2, 64, 16, 16, 2), (5, 1, 256, 64, 128, 2)])
def test_slope_along_the_gradient_is_its_length(Hq, Hkv, T, D, bs, S):
    """Along the unit vector w of a gradient the float64 forward, by central differences, rises as fast as the gradient
    is long; the kernels' gradient may differ from that slope by its elements' bounds times |w| and by what the rounding
    of out to bf16 moves the formula.  That is under 5% of the slope: another length or sign is refused.
    """
    q, k, v, idx, dout = inputs(1, Hq, Hkv, T, D, bs, S, 11)
    out, lse = forward(q, k, v, idx, bs)
    grads = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    h, n, d = [t.double().cpu().numpy() for t in (q, k, v)], idx.cpu().numpy(), dout.double().cpu().numpy()
    o, m = onsa.nsa_select_forward(*h, n, bs)
    true = onsa.nsa_select_backward(*h, n, o, m, d, bs)
    *rounded, sums = onsa.nsa_select_backward(*h, n, out.double().cpu().numpy(), lse.double().cpu().numpy(), d, bs)
    for which, (name, terms) in enumerate((("dq", S * bs), ("dk", T * Hq // Hkv), ("dv", T * Hq // Hkv))):
        w, r = true[which] / np.linalg.norm(true[which]), rounded[which]
        side = []
        for e in (1e-3, -1e-3):
            x = [y + e * w if j == which else y for j, y in enumerate(h)]
            side.append((onsa.nsa_select_forward(*x, n, bs)[0] * d).sum())
        slope = (side[0] - side[1]) / 2e-3
        bound = (1 + BF) * (BF * sums[name] + U * (sums[name + "_e"] + terms * sums[name])) + BF * np.abs(r)
        # (differences: 1e-6 of the third derivative, at most 1e-4 of the slope here)
        slack = (bound * np.abs(w)).sum() + abs(((r - true[which]) * w).sum()) + 1e-4 * slope
        assert slack <= 0.05 * slope
        assert abs((grads[which].double().cpu().numpy() * w).sum() - slope) <= slack, name
        for factor in (-1.0, 0.5, 0.9, 1.1, 2.0):  # planted in the oracle's
            assert abs(factor * (r * w).sum() - slope) > slack


@pytest.mark.parametrize("D,bs,Hq,Hkv", [(64, 64, 8, 1), (128, 64, 16, 1), (128, 128, 3, 1), (64, 32, 4, 2),
                                         (128, 16, 8, 2), (32, 32, 4, 1), (64, 128, 5, 1)])
@pytest.mark.parametrize("cut", [1, 9])
@pytest.mark.parametrize("what", ["large", "inf", "nan"])
def test_a_padded_tail_of_anything_stays_out(D, bs, Hq, Hkv, cut, what):
    """Tokens behind a sequence's end, inside a block that its last rows select, hold numbers up to bf16's largest or
    none, and their rows select nothing: every other row's and key's gradient is the one beside a tail of zeros."""
    T, S = 512, 3
    q, k, v, idx, dout = inputs(1, Hq, Hkv, T, D, bs, S, D + bs + cut)
    idx[:, :, T - cut:] = -1
    for t in (q, k, v, dout):
        t[:, :, T - cut:] = 0
    out, lse = forward(q, k, v, idx, bs)
    clean = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    top = {"large": 3e38, "inf": float("inf"), "nan": float("nan")}[what]
    for t, x in ((k, top), (v, -top), (q, top / 2), (dout, top), (out, top), (lse, top)):
        t[:, :, T - cut:] = x
    k[:, :, T - cut:, ::3] = -1e30
    got = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    torch.cuda.synchronize()
    for x, y in zip(got, clean):
        assert torch.equal(x, y)
