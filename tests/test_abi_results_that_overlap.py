"""Results that the rows' norm and rotation and the 4-bit cache's read write into memory of the caller's: refused where
they lie over an input or over each other, allowed where a result is its own input (CPU: tensors that pass for a
device's, and raw functions that record; GPU: the results in place)."""

import pytest
import torch

from block_sparse_attention_tra_gb300 import BsaError, bsa

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


@pytest.fixture
def reached(monkeypatch):
    got = []
    monkeypatch.setattr(bsa, "_one_device", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bsa, "_raw_stream", lambda *a: 0)
    for name in ("qk_norm_rope_forward_raw", "nsa_cache4_read_raw"):
        monkeypatch.setattr(bsa, name, lambda *a, **k: got.append(a) or 0)
    return got


def rows(B=2, Hq=4, Hkv=4, T=3, D=64):
    """q, k, two results and the buffer they are all cut from, each with room of a row behind it."""
    n = B * max(Hq, Hkv) * T * D
    buf = torch.zeros(4 * n + 4 * D, dtype=BF)
    cut = [buf[i * (n + D): i * (n + D) + n] for i in range(4)]
    return [c.view(B, h, T, D) for c, h in zip(cut, (Hq, Hkv, Hq, Hkv))] + [buf]


def test_rows_refuse_results_over_inputs_and_each_other(reached):
    q, k, qo, ko, buf = rows()
    D, n = q.shape[3], q.numel()
    last = buf[n - D: 2 * n - D].view(q.shape)  # q's last row is its first
    w, f, pos = torch.ones(64), torch.ones(32), torch.zeros((2, 3), dtype=I32)
    for given in ({"q_out": k}, {"k_out": q}, {"q_out": qo, "k_out": qo}, {"q_out": last}, {"q_out": q, "k_out": q},
                  {"q_out": k, "k_out": q}, {"k_out": last}, {"k_out": buf[n: 2 * n].view(k.shape)}):
        with pytest.raises(BsaError, match="overlaps"):
            bsa.qk_norm_rope_forward(q, k, w, w, f, pos, **given)
    fp = [torch.zeros(q.shape) for _ in range(2)]
    for given in ({"q_weight": fp[0].view(-1)[:64]}, {"k_weight": fp[0].view(-1)[-64:]}, {"inv_freq": fp[0].view(-1)[64:96]},
                  {"positions": fp[0].view(I32).view(-1)[:6].view(2, 3)}):
        with pytest.raises(BsaError, match="overlaps"):
            bsa.qk_norm_rope_forward(fp[1], fp[1].clone(), **given, q_out=fp[0])
    assert not reached
    # results that only touch, results in place, and rows that are copied before the kernel reads them
    bsa.qk_norm_rope_forward(q, k, w, w, f, pos, q_out=qo, k_out=ko)
    bsa.qk_norm_rope_forward(q, k, w, w, f, pos, q_out=q, k_out=k)
    bsa.qk_norm_rope_forward(q, k, q_out=buf[2 * n + 2 * D: 3 * n + 2 * D].view(q.shape),
                             k_out=buf[3 * n + 2 * D: 4 * n + 2 * D].view(q.shape))
    cols = k.view(2, 4, 64, 3).transpose(2, 3)
    bsa.qk_norm_rope_forward(q, cols, q_out=k)
    fused = torch.zeros((1, 1, 6, 64), dtype=BF).transpose(1, 2)  # one token's heads: its parts in place
    bsa.qk_norm_rope_forward(fused[:, :4], fused[:, 4:], q_out=fused[:, :4], k_out=fused[:, 4:])
    assert len(reached) == 5


def test_read_refuses_results_over_each_other_and_the_cache(reached):
    cache = [torch.zeros((3, 2, 32, n), dtype=U8) for n in (32, 32, 4, 4)]
    rest = torch.zeros((1, 3), dtype=I32), torch.zeros(1, dtype=I32)
    buf = torch.zeros(4000, dtype=BF)
    a, b, c = (buf[i: i + 640].view(1, 2, 5, 64) for i in (0, 640, 1279))
    for given in ({"k_out": a, "v_out": a}, {"k_out": b, "v_out": c}, {"k_out": c, "v_out": b},
                  {"k_out": cache[0].view(-1)[:1280].view(BF).view(1, 2, 5, 64), "v_out": b},
                  {"k_out": b, "v_out": cache[1].view(-1)[-1280:].view(BF).view(1, 2, 5, 64)}):
        with pytest.raises(BsaError, match="overlaps"):
            bsa.nsa_cache4_read(*cache, *rest, 5, **given)
    assert not reached
    bsa.nsa_cache4_read(*cache, *rest, 5, k_out=a, v_out=b)
    assert len(reached) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("B,Hq,Hkv,T,D,rotary", [(1, 4, 2, 1, 64, 64), (3, 5, 2, 37, 80, 48), (2, 40, 8, 300, 128, 128),
                                                 (1, 1, 1, 5000, 16, 16), (2, 34, 1, 2048, 64, 0)])
def test_rows_in_place(dtype, B, Hq, Hkv, T, D, rotary):
    """A thread reads what it writes, and reads it first, however many rows it walks."""
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k = (torch.randn((B, h, T, D), generator=g, device="cuda").to(dtype) for h in (Hq, Hkv))
    w = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
    f = bsa.rope_frequencies(rotary, device="cuda")[0] if rotary else None
    for il in (False, True):
        want = bsa.qk_norm_rope_forward(q, k, w, w, f, interleaved=il)
        q2, k2 = q.clone(), k.clone()
        got = bsa.qk_norm_rope_forward(q2, k2, w, w, f, interleaved=il, q_out=q2, k_out=k2)
        assert got[0] is q2 and got[1] is k2
        assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
