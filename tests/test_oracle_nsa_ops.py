"""CPU: the oracles of the selection attention's backward and of the paged
e4m3 cache, pinned against independent formulations."""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import workloads
from oracle import cache as ocache
from oracle import nsa as onsa


@pytest.mark.parametrize("Hq,Hkv,T,D,bs,S", [(4, 2, 64, 16, 16, 2), (3, 1, 96, 32, 32, 3), (2, 2, 16, 16, 16, 1)])
def test_backward_oracle_is_the_forward_oracles_gradient(Hq, Hkv, T, D, bs, S):
    q, k, v, idx = workloads.nsa_inputs(1, Hq, Hkv, T, D, bs, S, seed=T)
    idx[:, :, T // 2: T // 2 + 3] = -1
    q, k, v = (t.double().requires_grad_() for t in (q, k, v))
    sel = torch.zeros((1, Hkv, T, T // bs + 1), dtype=torch.bool).scatter_(3, torch.where(idx >= 0, idx, T // bs).long(),
                                                                          True)
    keep = (sel[..., :-1].repeat_interleave(bs, 3) & torch.ones(T, T, dtype=torch.bool).tril()).repeat_interleave(
        Hq // Hkv, 1)
    kk, vv = (t.repeat_interleave(Hq // Hkv, 1) for t in (k, v))
    s = (q @ kk.transpose(2, 3) * D ** -0.5).masked_fill(~keep, -1e30)
    out = torch.where(keep.any(-1, keepdim=True), s.softmax(-1), 0.0) @ vv
    dout = torch.randn(out.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    want = torch.autograd.grad(out, (q, k, v), dout)
    h = [t.detach().numpy() for t in (q, k, v)]
    o, lse = onsa.nsa_select_forward(*h, idx.numpy(), bs)
    got = onsa.nsa_select_backward(*h, idx.numpy(), o, lse, dout.numpy(), bs)
    for g, w in zip(got, want):
        assert np.abs(g - w.numpy()).max() <= 1e-12
    for name, g in zip(("dq", "dk", "dv"), got):
        assert (got[3][name] >= np.abs(g) - 1e-12).all() and (got[3][name + "_e"] >= 0).all()


def test_codes_are_torchs_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ocache.VALUES, want, equal_nan=True)
    x = torch.cat([torch.randn(4000, dtype=torch.float64, generator=torch.Generator().manual_seed(0)) * s
                   for s in (1e-3, 1.0, 100.0)]).clamp(-448, 448).float()
    mid = torch.from_numpy((ocache.VALUES[:126] + ocache.VALUES[1:127]) / 2).float()  # ties
    x = torch.cat([x, mid, -mid])
    assert np.array_equal(ocache.e4m3_encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert ocache.e4m3_encode([1e9, -np.inf, np.nan]).tolist() == [126, 254, 127]


def test_least_scale():
    for a in (1e-30, 1.0, 447.9, 448.0, 448.1, 3e38):
        s = ocache.least_scale(a)
        assert a <= 448 * s and (s == 2.0 ** ocache.E_MIN or a > 224 * s)
    assert ocache.least_scale(0.0) == 2.0 ** ocache.E_MIN


def test_rotation_is_relative():
    """Rotated products depend on the distance only."""
    r = np.random.default_rng(0)
    q, k = r.standard_normal((1, 32)), r.standard_normal((1, 32))
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    for il in (False, True):
        a = ocache.rotate(q, [100], f, il) @ ocache.rotate(k, [93], f, il).T
        b = ocache.rotate(q, [7], f, il) @ ocache.rotate(k, [0], f, il).T
        assert np.abs(a - b).max() <= 1e-12
    part = ocache.rotate(q, [5], f[:8], False)
    assert np.array_equal(part[:, 16:], q[:, 16:]) and not np.array_equal(part[:, :16], q[:, :16])


def test_append_then_decode_is_the_forward():
    """Values that e4m3 holds exactly, appended in two steps and read back."""
    r = np.random.default_rng(2)
    B, Hq, Hkv, T, D, page = 1, 2, 1, 48, 16, 16
    k, v = (ocache.VALUES[r.integers(0, 127, (B, Hkv, T, D))] for _ in range(2))
    k[..., 0] = v[..., 0] = 448.0  # scale 1 on every page
    q = r.standard_normal((B, Hq, T, D)) / 200
    table = np.array([[2, 0, 1]])
    caches = []
    for x in (k, v):
        c, s = np.zeros((3, Hkv, page, D), dtype=np.uint8), np.zeros((3, Hkv))
        c, s, _ = ocache.append(x[:, :, :19], c, s, table, [0], [19])
        c, s, _ = ocache.append(x[:, :, 19:], c, s, table, [19], [T - 19])
        assert (s == 1).all()
        caches.append((c, s))
    (kc, ks), (vc, vs) = caches
    rows = np.full((B, Hkv, T, 2), -1)
    rows[:, :, T - 1] = [0, 2]
    want, wl = onsa.nsa_select_forward(q, k, v, rows, page)
    out, lse, _ = ocache.decode(q[:, :, T - 1:], kc, vc, ks, vs, table, [T], rows[:, :, T - 1:])
    assert np.abs(out[:, :, 0] - want[:, :, -1]).max() <= 1e-10 and np.abs(lse[:, :, 0] - wl[:, :, -1]).max() <= 1e-10


def test_growing_scale_moves_held_codes():
    table = np.array([[0]])
    c, s = np.zeros((1, 1, 16, 16), dtype=np.uint8), np.zeros((1, 1))
    x = np.full((1, 1, 1, 16), 1.0)
    c, s, _ = ocache.append(x, c, s, table, [0], [1])
    c, s, _ = ocache.append(x * 1000, c, s, table, [1], [1])
    assert s[0, 0] == 4.0 and (ocache.VALUES[c[0, 0, 0]] == 0.25).all() and (ocache.VALUES[c[0, 0, 1]] == 256.0).all()
    c, s, _ = ocache.append(x, c, s, table, [2], [1])  # a smaller one keeps it
    assert s[0, 0] == 4.0
