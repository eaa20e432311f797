"""CPU: host-side argument checks of the rows' norm and rotation and of the 4-bit cache (nothing is enqueued), and the
binding's own refusals."""

import pytest
import torch

from block_sparse_attention_tra_gb300 import BsaError, bsa

P = 4096  # a fake, aligned "device" address
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_sparse_attention_tra_gb300 import build

    build.build()
    bsa.load_library()


no_gpu = not torch.cuda.is_available()


def fwd(strides=None, B=2, Hq=4, Hkv=2, T=5, D=64, rotary=64, scale=1.0, eps=1e-6, dtype=1, wdtype=0, **kw):
    p = dict.fromkeys(("q", "k", "qo", "ko", "qw", "kw", "pos", "freq"), P) | kw
    return bsa.qk_norm_rope_forward_raw(*p.values(), strides, B, Hq, Hkv, T, D, rotary, 0, scale, eps, dtype, wdtype, 0)


def bwd(ws=P, nbytes=1 << 30, strides=None, B=2, Hq=4, Hkv=2, T=5, D=64, rotary=64, scale=1.0, eps=1e-6, dtype=1,
        wdtype=0, **kw):
    p = dict.fromkeys(("q", "k", "dqo", "dko", "dq", "dk", "dqw", "dkw", "qw", "kw", "pos", "freq"), P) | kw
    return bsa.qk_norm_rope_backward_raw(*p.values(), strides, B, Hq, Hkv, T, D, rotary, 0, scale, eps, dtype, wdtype,
                                         ws, nbytes, 0)


@pytest.mark.parametrize("call,count,names", [(fwd, 12, ("q", "k", "qo", "ko")),
                                              (bwd, 18, ("q", "k", "dqo", "dko", "dq", "dk"))])
def test_rows_refusals(call, count, names):
    for name in (*names, "freq"):
        assert call(**{name: None}) == 1, name
    for name in (*names, "qw", "kw", "freq"):
        assert call(**{name: P + 8}) == 7, name
    assert call(pos=P + 2) == 7
    assert call(dtype=2) == 3 and call(wdtype=5) == 3
    for bad in ({"B": 0}, {"T": 0}, {"Hq": 0}, {"Hkv": 65536}, {"B": 1 << 16, "T": 1 << 15},
                {"B": 1 << 10, "T": 1 << 20, "Hq": 16384}):
        assert call(**bad) == 2, bad
    for bad in ({"D": 8}, {"D": 144}, {"D": 72}, {"rotary": 8}, {"rotary": 80}, {"rotary": -16}, {"eps": 0.0},
                {"eps": NAN}, {"eps": INF}, {"scale": NAN}, {"scale": INF}):
        assert call(**bad) == 4, bad
    good = [64] * count
    for i in range(count):
        assert call(strides=good[:i] + [-64] + good[i + 1:]) == 2
        assert call(strides=good[:i] + [1 << 40] + good[i + 1:]) == 2
        assert call(strides=good[:i] + [12] + good[i + 1:]) == 7  # 24 bytes
    if no_gpu:
        assert call() == 6 and call(strides=good) == 6 and call(qw=None, kw=None) == 6 and call(pos=None) == 6
        assert call(rotary=0, freq=None) == 6 and call(dtype=0, strides=[4] * count) == 6


@pytest.mark.parametrize("call,count,written", [(fwd, 12, 6), (bwd, 18, 12)])
def test_results_do_not_repeat_rows(call, count, written):
    """A stride of 0 repeats rows of an input; of a result it would leave several rows in one place."""
    for i in range(written, count):
        s = [0] * written + [64] * (count - written)
        s[i] = 0
        assert call(strides=s) == 2
        if no_gpu:
            axis = i % 3
            assert call(strides=s, **({"B": 1}, {"Hq": 1, "Hkv": 1}, {"T": 1})[axis]) == 6


def test_rows_backward_workspace():
    assert bwd(ws=None) == 1 and bwd(ws=P + 16) == 7 and bwd(dqw=None) == 1 and bwd(dkw=None) == 1
    need = bsa.qk_norm_rope_backward_workspace_size(2, 4, 2, 5, 64)
    assert need > 0 and need % 256 == 0 and bwd(nbytes=need - 1) == 9
    assert bsa.qk_norm_rope_backward_workspace_size(2, 4, 2, 5, 72) == 0
    assert bsa.qk_norm_rope_backward_workspace_size(1 << 16, 4, 2, 1 << 15, 64) == 0
    if no_gpu:
        assert bwd(nbytes=need) == 6 and bwd(dqw=None, dkw=None, qw=None, kw=None) == 6


CACHE = ("kc", "vc", "ks", "vs")


def append(strides=None, B=2, Hq=8, Hkv=2, n=3, D=64, page=64, max_pages=4, pages=8, rotary=64, scale=1.0, eps=1e-6,
           dtype=1, wdtype=0, **kw):
    p = dict.fromkeys(("k", "v", "q", "qo", *CACHE, "kf", "vf", "table", "lens", "new", "qw", "kw", "freq"), P) | kw
    return bsa.nsa_cache4_append_raw(*p.values(), strides, B, Hq, Hkv, n, D, page, max_pages, pages, rotary, 0, scale,
                                     eps, dtype, wdtype, 0)


def test_append_refusals():
    for name in ("k", "v", "q", "qo", *CACHE, "table", "lens", "freq"):
        assert append(**{name: None}) == 1, name
    for name in ("k", "v", "q", "qo", *CACHE, "qw", "kw", "freq"):
        assert append(**{name: P + 8}) == 7, name
    for name in ("kf", "vf", "table", "lens", "new"):
        assert append(**{name: P + 2}) == 7, name
    assert append(dtype=2) == 3 and append(wdtype=-1) == 3
    for bad in ({"B": 0}, {"n": 0}, {"Hq": 7}, {"pages": 0}, {"max_pages": 0}, {"max_pages": 1 << 26}, {"n": 1 << 30},
                {"pages": 1 << 30, "page": 128, "D": 128}, {"n": 1 << 28, "B": 8}):
        assert append(**bad) == 2, bad
    for bad in ({"D": 96}, {"page": 24}, {"page": 256}, {"Hq": 64}, {"rotary": 8}, {"rotary": 80}, {"eps": -1.0},
                {"scale": INF}):
        assert append(**bad) == 4, bad
    good = [64] * 9
    for i in range(9):
        assert append(strides=good[:i] + [-64] + good[i + 1:]) == 2
        assert append(strides=good[:i] + [4] + good[i + 1:]) == 7
    if no_gpu:
        assert append() == 6 and append(new=None, kf=None, vf=None, qw=None, kw=None) == 6
        assert append(q=None, qo=None, qw=None) == 6 and append(rotary=0, freq=None) == 6


def read(B=2, Hkv=2, n=3, D=64, page=64, max_pages=4, pages=8, dtype=1, **kw):
    p = dict.fromkeys((*CACHE, "kf", "vf", "table", "starts", "lens", "ko", "vo"), P) | kw
    return bsa.nsa_cache4_read_raw(*p.values(), B, Hkv, n, D, page, max_pages, pages, dtype, 0)


def test_read_refusals():
    for name in (*CACHE, "table", "lens", "ko", "vo"):
        assert read(**{name: None}) == 1, name
    for name in (*CACHE, "ko", "vo"):
        assert read(**{name: P + 8}) == 7, name
    for name in ("kf", "vf", "table", "starts", "lens"):
        assert read(**{name: P + 2}) == 7, name
    assert read(dtype=7) == 3
    assert read(B=0) == 2 and read(n=0) == 2 and read(pages=0) == 2 and read(max_pages=1 << 26) == 2
    assert read(D=48) == 4 and read(page=8) == 4
    if no_gpu:
        assert read() == 6 and read(starts=None, kf=None, vf=None) == 6


def decode(ws=P, nbytes=1 << 30, B=2, Hq=8, Hkv=2, D=64, page=64, max_pages=4, pages=8, S=4, **kw):
    p = dict.fromkeys(("q", *CACHE, "kf", "vf", "table", "lens", "idx", "out", "lse"), P) | kw
    return bsa.nsa_cache4_decode_raw(*p.values(), B, Hq, Hkv, D, page, max_pages, pages, S, ws, nbytes, 0)


def test_decode_refusals():
    for name in ("q", *CACHE, "table", "lens", "out"):
        assert decode(**{name: None}) == 1, name
    assert decode(ws=None, idx=None, S=0) == 1 and decode(ws=P + 8) == 7
    for name in ("q", *CACHE, "out"):
        assert decode(**{name: P + 8}) == 7, name
    for name in ("kf", "vf", "table", "lens", "idx", "lse"):
        assert decode(**{name: P + 2}) == 7, name
    assert decode(S=0) == 2 and decode(S=33) == 2 and decode(idx=None, S=4) == 2 and decode(B=0) == 2
    assert decode(D=48) == 4 and decode(page=8) == 4 and decode(Hq=64) == 4
    for S in (0, 4):
        need = bsa.nsa_cache4_decode_workspace_size(2, 8, 2, 64, 64, 4, S)
        assert need > 0 and decode(nbytes=need - 1, S=S, **({} if S else {"idx": None})) == 9
    assert bsa.nsa_cache4_decode_workspace_size(2, 8, 2, 48, 64, 4, 4) == 0
    if no_gpu:
        assert decode() == 6 and decode(idx=None, S=0, lse=None, kf=None, vf=None) == 6
        assert decode(ws=None, nbytes=0) == 6  # selected pages need no workspace


# ---------------------------------------------------------------- the binding


def of(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def cache_args(page=64, D=64):
    return {"k_cache": of(1, 1, page, D // 2, dtype=torch.uint8), "v_cache": of(1, 1, page, D // 2, dtype=torch.uint8),
            "k_scale": of(1, 1, page, D // 16, dtype=torch.float8_e4m3fn),
            "v_scale": of(1, 1, page, D // 16, dtype=torch.uint8),
            "page_table": of(1, 1, dtype=torch.int32), "cache_lens": of(1, dtype=torch.int32)}


def calls():
    x, w = of(1, 1, 1, 64), of(64, dtype=torch.float32)
    f = of(8, dtype=torch.float32)
    return [(bsa.qk_norm_rope_forward, {"q": x, "k": x, "q_weight": w, "k_weight": w, "inv_freq": f, "q_out": x, "k_out": x}),
            (bsa.nsa_cache4_append, {"k": x, "v": x, "q": x, "q_out": x, "q_weight": w, "k_weight": w, "inv_freq": f,
                                     "k_factor": w[:1], "v_factor": w[:1]} | cache_args()),
            (bsa.nsa_cache4_read, {"n": 1, "k_out": x, "v_out": x, "k_factor": w[:1], "v_factor": w[:1]} | cache_args()),
            (bsa.nsa_cache4_decode, {"q": x, "out": x, "lse": of(1, 1, 1, dtype=torch.float32), "k_factor": w[:1],
                                     "v_factor": w[:1]} | cache_args())]


def test_binding_has_no_cpu_path():
    for call, args in calls():
        with pytest.raises(BsaError, match="no CPU path"):
            call(**args)
    x = of(1, 1, 1, 64)
    with pytest.raises(BsaError, match="no CPU path"):
        bsa.qk_norm_rope(x, x)
    with pytest.raises(BsaError, match="no CPU path"):
        bsa.qk_norm_rope_backward(x, x, x, x)


def test_calls_without_a_gradient_refuse_tensors_that_one_is_asked_of():
    for call, args in calls():
        for name, t in args.items():
            if not isinstance(t, torch.Tensor) or t.dtype not in (torch.float32, torch.bfloat16):
                continue
            given = args | {name: t.clone().requires_grad_()}
            with pytest.raises(BsaError, match="has no gradient"):
                call(**given)
            with torch.no_grad(), pytest.raises(BsaError, match="no CPU path"):  # the next refusal
                call(**given)
    x, f = of(1, 1, 1, 64), of(8, dtype=torch.float32)
    with pytest.raises(BsaError, match="inv_freq has no gradient"):
        bsa.qk_norm_rope(x, x, inv_freq=f.requires_grad_())


@pytest.fixture
def on_device(monkeypatch):
    """Tensors that pass for a device's: the refusals come before anything is called."""
    monkeypatch.setattr(bsa, "_one_device", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name in ("qk_norm_rope_forward_raw", "qk_norm_rope_backward_raw", "nsa_cache4_append_raw", "nsa_cache4_read_raw",
                 "nsa_cache4_decode_raw"):
        monkeypatch.setattr(bsa, name, None)


def refused(call, args, **change):
    with pytest.raises(BsaError) as e:
        call(**(args | change))
    return e.value.status


def test_binding_checks_shapes_and_types(on_device):
    f32 = torch.float32
    forward, append, read, decode = calls()
    call, args = forward
    for change in ({"k": of(1, 1, 2, 64)}, {"q": of(1, 1, 64)}, {"q_weight": of(32, dtype=f32)},
                   {"inv_freq": of(1, 8, dtype=f32)}, {"q_out": of(1, 2, 1, 64)},
                   {"positions": of(2, dtype=torch.int32)}, {"k_out": of(1, 1, 1, 128)[..., ::2]}):
        assert refused(call, args, **change) == 2, change
    for change in ({"k": of(1, 1, 1, 64, dtype=f32)}, {"q_weight": of(64, dtype=torch.float16)},
                   {"q_out": of(1, 1, 1, 64, dtype=f32)}):
        assert refused(call, args, **change) == 3, change
    x = of(1, 1, 1, 64)
    back = {"q": x, "k": x, "dq_out": x, "dk_out": x}
    assert refused(bsa.qk_norm_rope_backward, back, dq_out=of(1, 2, 1, 64)) == 2
    assert refused(bsa.qk_norm_rope_backward, back, dk_out=x.float()) == 3
    assert refused(bsa.qk_norm_rope_backward, back, workspace=of(1 << 20, dtype=torch.uint8)[::2]) == 2
    for call, args in (append, read, decode):
        for change in ({"k_cache": of(1, 1, 64, 64, dtype=torch.uint8)}, {"v_scale": of(1, 1, 64, 3, dtype=torch.uint8)},
                       {"cache_lens": of(2, dtype=torch.int32)}, {"page_table": of(1, dtype=torch.int32)},
                       {"k_factor": of(2, dtype=f32)}, {"v_cache": of(1, 1, 32, 64, dtype=torch.uint8).transpose(2, 3)}):
            assert refused(call, args, **change) == 2, change
        for change in ({"k_cache": of(1, 1, 64, 32, dtype=torch.int8)}, {"k_scale": of(1, 1, 64, 4)},
                       {"v_factor": of(1)}):
            assert refused(call, args, **change) == 3, change
    call, args = append
    for change in ({"v": of(1, 1, 2, 64)}, {"q": of(1, 1, 2, 64)}, {"new_lens": of(2, dtype=torch.int32)}):
        assert refused(call, args, **change) == 2, change
    assert refused(call, args, v=x.float()) == 3
    with pytest.raises(BsaError, match="without q"):
        call(**(args | {"q": None, "q_out": None}))
    call, args = read
    assert refused(call, args, k_out=None, v_out=None, n=0) == 2
    assert refused(call, args, starts=of(2, dtype=torch.int32)) == 2 and refused(call, args, dtype=f32) == 3
    with pytest.raises(BsaError, match="together"):
        call(**(args | {"v_out": None}))
    call, args = decode
    assert refused(call, args, block_idx=of(1, 1, 2, 1, dtype=torch.int32)) == 2
    assert refused(call, args, q=x.float(), out=None) == 3 and refused(call, args, lse=of(1, 1, dtype=f32)) == 2
    for w in (of(1, dtype=torch.uint8).expand(1 << 30), of(1 << 10, dtype=torch.uint8)[::2]):
        with pytest.raises(BsaError, match="workspace must be contiguous"):
            call(**(args | {"workspace": w}))
