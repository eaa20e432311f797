"""CPU: host-side argument checks of the selection attention's backward, cache
append and decode (nothing is enqueued), and the binding's own refusals."""

import pytest
import torch

from block_sparse_attention_tra_gb300 import BsaError, bsa

P = 4096  # a fake, aligned "device" address


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_sparse_attention_tra_gb300 import build

    build.build()
    bsa.load_library()


no_gpu = not torch.cuda.is_available()


def bwd(ws=P, nbytes=1 << 40, B=1, Hq=16, Hkv=1, T=128, D=128, bs=64, S=4, **kw):
    p = dict.fromkeys(("q", "k", "v", "idx", "out", "lse", "dout", "dq", "dk", "dv"), P) | kw
    return bsa.nsa_select_backward_raw(*p.values(), B, Hq, Hkv, T, D, bs, S, ws, nbytes, 0)


def test_backward_refusals():
    for name in ("q", "k", "v", "idx", "out", "lse", "dout", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == 1, name
    assert bwd(ws=None) == 1
    for name in ("q", "k", "v", "out", "dout", "dq", "dk", "dv"):
        assert bwd(**{name: P + 8}) == 7, name
    assert bwd(idx=P + 2) == 7 and bwd(lse=P + 1) == 7 and bwd(ws=P + 16) == 7
    assert bwd(T=100) == 2 and bwd(S=0) == 2 and bwd(S=33) == 2 and bwd(Hq=24, Hkv=16) == 2 and bwd(B=0) == 2
    assert bwd(D=96) == 4 and bwd(bs=48, T=192) == 4 and bwd(Hq=32) == 4
    need = bsa.nsa_select_backward_workspace_size(1, 16, 1, 128, 128, 64, 4)
    assert bwd(nbytes=need - 1) == 9
    if no_gpu:
        assert bwd(nbytes=need) == 6


def test_backward_workspace_size():
    size = bsa.nsa_select_backward_workspace_size
    assert size(1, 16, 1, 128, 128, 64, 4) % 256 == 0
    rows = 2 * 32 * 8192 * 16  # f16 dQ rows of 64-token blocks of 64 or 128 dims
    assert rows * 256 < size(2, 32, 2, 8192, 128, 64, 16) < rows * 256 + (1 << 29)
    assert size(2, 32, 2, 8192, 32, 64, 16) < 1 << 28
    assert size(1, 16, 1, 100, 128, 64, 4) == 0 and size(1, 16, 1, 128, 96, 64, 4) == 0
    assert size(70000, 1, 1, 16, 16, 16, 1) == 0  # (batch, kv head) pairs past a grid's second axis
    assert bwd(B=70000, Hq=1, T=16, D=16, bs=16, S=1) == 2
    assert size(64, 64, 16, 131072, 64, 64, 16) == 0  # list positions past 32 bits


def append(B=2, Hq=8, Hkv=2, n=3, D=64, page=64, max_pages=4, pages=8, rotary=64, il=0, dtype=1, **kw):
    p = dict.fromkeys(("k", "v", "q", "q_out", "kc", "vc", "ks", "vs", "table", "lens", "new", "freq"), P) | kw
    return bsa.nsa_cache_append_raw(*p.values(), B, Hq, Hkv, n, D, page, max_pages, pages, rotary, il, dtype, 0)


def test_append_refusals():
    for name in ("k", "v", "kc", "vc", "ks", "vs", "table", "lens", "q", "q_out", "freq"):
        assert append(**{name: None}) == 1, name
    for name in ("k", "v", "q", "q_out", "kc", "vc"):
        assert append(**{name: P + 8}) == 7, name
    for name in ("ks", "vs", "table", "lens", "new", "freq"):
        assert append(**{name: P + 2}) == 7, name
    assert append(dtype=2) == 3
    for bad in ({"B": 0}, {"n": 0}, {"Hq": 7}, {"pages": 0}, {"max_pages": 0}, {"max_pages": 1 << 26}, {"n": 1 << 30},
                {"pages": 1 << 30, "page": 128, "D": 128}):
        assert append(**bad) == 2, bad
    for bad in ({"D": 96}, {"page": 24}, {"page": 256}, {"Hq": 64}, {"rotary": 8}, {"rotary": 80}, {"rotary": -16}):
        assert append(**bad) == 4, bad
    if no_gpu:
        assert append() == 6 and append(new=None) == 6 and append(q=None, q_out=None) == 6
        assert append(rotary=0, freq=None) == 6


def decode(ws=P, nbytes=1 << 30, B=2, Hq=8, Hkv=2, D=64, page=64, max_pages=4, pages=8, S=4, **kw):
    p = dict.fromkeys(("q", "kc", "vc", "ks", "vs", "table", "lens", "idx", "out", "lse"), P) | kw
    return bsa.nsa_select_decode_raw(*p.values(), B, Hq, Hkv, D, page, max_pages, pages, S, ws, nbytes, 0)


def test_decode_refusals():
    for name in ("q", "kc", "vc", "ks", "vs", "table", "lens", "out"):
        assert decode(**{name: None}) == 1, name
    assert decode(ws=None) == 1
    for name in ("q", "kc", "vc", "out"):
        assert decode(**{name: P + 8}) == 7, name
    for name in ("ks", "vs", "table", "lens", "idx", "lse"):
        assert decode(**{name: P + 2}) == 7, name
    assert decode(ws=P + 8) == 7
    assert decode(S=0) == 2 and decode(S=33) == 2 and decode(idx=None, S=4) == 2 and decode(B=0) == 2
    assert decode(D=48) == 4 and decode(page=8) == 4 and decode(Hq=64) == 4
    need = bsa.nsa_select_decode_workspace_size(2, 8, 2, 64, 64, 4, 4)
    assert need > 0 and decode(nbytes=need - 1) == 9
    assert bsa.nsa_select_decode_workspace_size(2, 8, 2, 48, 64, 4, 4) == 0
    if no_gpu:
        assert decode(nbytes=need) == 6 and decode(idx=None, S=0, lse=None) == 6


def test_binding_has_no_cpu_path():
    x = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, 64, 1, dtype=torch.int32)
    c = torch.zeros(1, 1, 64, 64, dtype=torch.uint8)
    s, t, n = torch.ones(1, 1), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(BsaError, match="no CPU path"):
        bsa.nsa_select_backward(x, x, x, i, x, torch.zeros(1, 1, 64), x)
    with pytest.raises(BsaError, match="no CPU path"):
        bsa.nsa_select_attention(x, x, x, i, 64)
    with pytest.raises(BsaError, match="no CPU path"):
        bsa.nsa_cache_append(x, x, c, c, s, s, t, n)
    with pytest.raises(BsaError, match="no CPU path"):
        bsa.nsa_select_decode(x[:, :, :1], c, c, s, s, t, n)


def test_attention_refuses_what_its_backward_cannot_count():
    """The binding's rule is the library's, on both sides of each limit; the refusal comes before the forward runs."""
    size = bsa.nsa_select_backward_workspace_size
    for B, Hq, Hkv, T, S in ((65535, 1, 1, 16, 1), (65536, 1, 1, 16, 1), (5, 13107, 13107, 16, 1),
                             (16, 8192, 4096, 16, 1), (1, 1, 1, (1 << 26) - 16, 1), (1, 1, 1, 1 << 26, 1),
                             (1, 1, 1, (1 << 26) - 16, 32), (1, 32, 2, (1 << 26) - 16, 1),
                             (1, 31, 31, (1 << 26) - 16, 1), (64, 64, 16, 131072, 16), (64, 64, 16, 131072, 15),
                             (2048, 16, 16, 65536, 1)):
        assert bsa._nsa_backward_counts(B, Hq, Hkv, T, S) == (size(B, Hq, Hkv, T, 16, 16, S) > 0), (B, Hq, Hkv, T, S)
    q, i = (torch.empty(65536, 1, 16, n, dtype=torch.bfloat16, device="meta") for n in (16, 1))
    with pytest.raises(BsaError, match="no gradients for"):
        bsa.nsa_select_attention(q.requires_grad_(), q, q, i, 16)


def test_cache_calls_refuse_tensors_that_a_gradient_is_asked_of():
    def of(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype)

    x, c = of(1, 1, 1, 64, dtype=torch.bfloat16), of(1, 1, 64, 64, dtype=torch.uint8)
    t, n = of(1, 1, dtype=torch.int32), of(1, dtype=torch.int32)
    append = {"k": x, "v": x, "k_cache": c, "v_cache": c, "k_scale": of(1, 1), "v_scale": of(1, 1), "q": x, "q_out": x,
              "inv_freq": of(8)}
    decode = {"q": x, "k_cache": c, "v_cache": c, "k_scale": of(1, 1), "v_scale": of(1, 1), "out": x,
              "lse": of(1, 1, 1)}
    for call, args in ((bsa.nsa_cache_append, append), (bsa.nsa_select_decode, decode)):
        for name, tensor in args.items():
            if not tensor.is_floating_point():
                continue
            given = args | {name: tensor.clone().requires_grad_()}
            with pytest.raises(BsaError, match="has no gradient"):
                call(**given, page_table=t, cache_lens=n)
            with torch.no_grad(), pytest.raises(BsaError, match="no CPU path"):  # the next refusal
                call(**given, page_table=t, cache_lens=n)


def test_workspaces_are_contiguous(monkeypatch):
    """The elements of an expanded or strided tensor say nothing about the memory behind it.  (Tensors that pass for a
    device's: the refusal comes before anything is called.)"""
    monkeypatch.setattr(bsa, "_one_device", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bsa, "nsa_select_backward_raw", None)
    monkeypatch.setattr(bsa, "nsa_select_decode_raw", None)
    x = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, 64, 1, dtype=torch.int32)
    c = torch.zeros(1, 1, 64, 64, dtype=torch.uint8)
    s, t, n = torch.ones(1, 1), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for w in (torch.zeros(1, dtype=torch.uint8).expand(1 << 30), torch.zeros(1 << 10, dtype=torch.uint8)[::2]):
        with pytest.raises(BsaError, match="workspace must be contiguous"):
            bsa.nsa_select_backward(x, x, x, i, x, torch.zeros(1, 1, 64), x, workspace=w)
        with pytest.raises(BsaError, match="workspace must be contiguous"):
            bsa.nsa_select_decode(x[:, :, :1], c, c, s, s, t, n, workspace=w)
