"""CPU: the oracles of the rows' norm and rotation and of the 4-bit cache, pinned against independent formulations."""

import numpy as np
import pytest
import torch

import block_sparse_attention_tra_gb300 as bsa_pkg
from block_sparse_attention_tra_gb300 import BsaError
from oracle import cache as ocache
from oracle import cache4, rows


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 32])
def test_rows_are_the_complex_product_and_its_gradient(interleaved, rotary):
    """Against torch's complex numbers and autograd, in 64 bits."""
    g = torch.Generator().manual_seed(rotary)
    x, dy = (torch.randn((2, 3, 5, 32), generator=g, dtype=torch.float64) for _ in range(2))
    w = 1.0 + 0.3 * torch.randn(32, generator=g, dtype=torch.float64)
    pos = torch.randint(-50, 1 << 20, (2, 5), generator=g)
    f = 100.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(1, rotary))
    for weight in (w, None):
        x.requires_grad_()
        w.requires_grad_()
        n = x if weight is None else torch.nn.functional.rms_norm(x, (32,), w, 1e-3)
        part = n[..., :rotary]
        z = (torch.view_as_complex(part.reshape(2, 3, 5, -1, 2)) if interleaved
             else torch.complex(part[..., : rotary // 2], part[..., rotary // 2:]))
        z = z * torch.polar(torch.full((2, 1, 5, rotary // 2), 1.5, dtype=torch.float64),
                            (pos[..., None] * f)[:, None])
        turned = (torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1))
        y = torch.cat([turned, n[..., rotary:]], -1)
        args = (None if weight is None else w.detach().numpy(), pos.numpy(), f.numpy(), interleaved, 1.5, 1e-3)
        got, e = rows.forward(x.detach().numpy(), *args)
        assert np.abs(got - y.detach().numpy()).max() <= 1e-9 and (e >= np.abs(got) - 1e-9).all()
        want = torch.autograd.grad(y, (x, w) if weight is not None else (x,), dy)
        dx, dw, ex, ew = rows.backward(x.detach().numpy(), dy.numpy(), *args)
        assert np.abs(dx - want[0].numpy()).max() <= 1e-8 and (ex >= np.abs(dx) - 1e-9).all()
        if weight is not None:
            assert np.abs(dw - want[1].numpy()).max() <= 1e-8 and (ew >= np.abs(dw) - 1e-9).all()


def test_rows_gradient_is_the_slope():
    """Differences along random directions."""
    r = np.random.default_rng(0)
    x, dy, w = r.standard_normal((1, 2, 3, 16)), r.standard_normal((1, 2, 3, 16)), r.standard_normal(16)
    pos, f = np.array([[0, 7, -3]]), np.array([1.0, 0.1])
    dx, dw, _, _ = rows.backward(x, dy, w, pos, f, False, 1.2, 1e-2)
    for _ in range(5):
        vx, vw, h = r.standard_normal(x.shape), r.standard_normal(16), 1e-5
        up, down = (rows.forward(x + s * vx, w + s * vw, pos, f, False, 1.2, 1e-2)[0] for s in (h, -h))
        assert abs(((up - down) / (2 * h) * dy).sum() - (dx * vx).sum() - (dw * vw).sum()) <= 1e-7


def test_codes_are_the_nearest():
    assert cache4.E2M1[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    # 1 sign, 2 exponent bits of bias 1, 1 mantissa bit
    for c in range(8):
        e, m = c >> 1, c & 1
        assert cache4.E2M1[c] == (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))
    x = np.linspace(-7, 7, 5601)
    got = cache4.E2M1[cache4.e2m1_encode(x)]
    assert np.array_equal(np.abs(got - np.clip(x, -6, 6)), np.abs(np.clip(x, -6, 6)[:, None] - cache4.E2M1).min(1))
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert cache4.e2m1_encode(ties).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert cache4.e2m1_encode([-5.0, -np.inf, np.inf, -0.0]).tolist() == [14, 15, 7, 8]


def test_encode_and_values():
    r = np.random.default_rng(1)
    x = r.standard_normal((7, 64)) * np.exp(r.standard_normal((7, 1)))
    x[0, :16] = 0.0
    x[1, 3], x[2, 20] = np.nan, np.inf
    codes, sc = cache4.encode(x)
    assert sc[0, 0] == 0 and sc[1, 0] == 0x7F and sc[2, 1] == 0x7F and (sc != 0x7F).sum() == sc.size - 2
    assert np.array_equal(cache4.unpack(cache4.pack(codes)), codes)
    v = cache4.values(cache4.pack(codes), sc, 2.0)
    assert np.isnan(v[1, :16]).all() and np.isfinite(v[3:]).all() and not v[0, :16].any()
    top = np.repeat(np.abs(x[3:]).reshape(4, 4, 16).max(-1), 16, -1)
    # a scale is off by 2^-4 and a code by half its step, which is at most 2 of 6
    assert (np.abs(v[3:] / 2.0 - x[3:]) <= top * (1 / 6 + 2.0 ** -4)).all()


def test_decode_is_the_e4m3_caches_on_the_same_values():
    """Codes and scales that both caches can hold: the two oracles agree."""
    r = np.random.default_rng(2)
    pages, H, page, D = 5, 2, 16, 32
    c4 = [r.integers(0, 256, (pages, H, page, D // 2), dtype=np.uint8) for _ in range(2)]
    scale = [np.repeat(np.repeat(ocache.e4m3_encode(2.0 ** r.integers(-3, 3, (pages, H))).astype(np.uint8)[..., None, None],
                                 page, 2), 2, 3) for _ in range(2)]
    c8 = [ocache.e4m3_encode(cache4.E2M1[cache4.unpack(c)]) for c in c4]
    s8 = [ocache.VALUES[s[:, :, 0, 0]] for s in scale]
    q, table, lens = r.standard_normal((2, 4, 1, D)), np.array([[3, 0], [4, 1]]), [20, 32]
    for idx in (None, np.array([1, -1, 1, 0, 0, 0, -1, -1]).reshape(2, 2, 1, 2)):
        a = cache4.decode(q, *c4, *scale, table, lens, idx, k_factor=[1.0, 2.0], v_factor=[0.5, 1.0])
        s8f = s8[0] * [1.0, 2.0], s8[1] * [0.5, 1.0]
        b = ocache.decode(q, *c8, *s8f, table, lens, idx)
        assert np.abs(a[0] - b[0]).max() <= 1e-12 and np.abs(a[1] - b[1]).max() <= 1e-12


def test_frequencies():
    f, s = bsa_pkg.rope_frequencies(64)
    assert s == 1.0 and f.dtype == torch.float32
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-7)
    lin, s = bsa_pkg.rope_frequencies(64, scaling="linear", factor=4.0)
    assert s == 1.0 and torch.allclose(lin * 4.0, f)
    base, _ = bsa_pkg.rope_frequencies(64, scaling="base", factor=4.0)
    assert base[0] == 1.0 and abs(float(base[-1] / f[-1]) - 0.25) < 1e-6 and (base[1:] < f[1:]).all()
    bands, s = bsa_pkg.rope_frequencies(64, scaling="bands", factor=4.0, original_length=4096)
    turns = f.double() * 4096 / (2 * np.pi)
    assert torch.equal(bands[turns > 32], f[turns > 32])
    assert torch.allclose(bands[turns < 1] * 4.0, f[turns < 1]) and (bands[1:] < bands[:-1]).all()
    assert abs(s - (0.1 * np.log(4.0) + 1.0)) < 1e-12
    one, s = bsa_pkg.rope_frequencies(64, scaling="bands", factor=1.0, original_length=4096)
    assert s == 1.0 and torch.allclose(one, f)
    for bad in ({"rotary_dim": 7}, {"rotary_dim": 64, "scaling": "other"}, {"rotary_dim": 64, "factor": 0.5},
                {"rotary_dim": 64, "scaling": "bands", "factor": 2.0}, {"rotary_dim": 64, "base": 1.0}):
        with pytest.raises(BsaError):
            bsa_pkg.rope_frequencies(**bad)
