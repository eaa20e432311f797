"""CPU: every call of the rows and the 4-bit cache goes to the library through its ``*_raw`` function, the one that the
refusals' tests hold shut.  (Tensors that pass for a device's; the library itself is out of reach.)"""

import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa

NAMES = ("qk_norm_rope_forward", "qk_norm_rope_backward", "nsa_cache4_append", "nsa_cache4_read", "nsa_cache4_decode")


def of(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def calls():
    """Of each name the arguments of a call that nothing refuses."""
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    q, k, w, f = of(2, 4, 3, 64), of(2, 2, 3, 64), of(64, dtype=f32), of(32, dtype=f32)
    cache = [of(4, 2, 32, n, dtype=u8) for n in (32, 32, 4, 4)] + [of(2, 2, dtype=i32), of(2, dtype=i32)]
    rows = {"q_weight": w, "k_weight": w, "inv_freq": f}
    return {"qk_norm_rope_forward": ([q, k], rows),
            "qk_norm_rope_backward": ([q, k, q.clone(), k.clone()], rows | {"workspace": of(1 << 16, dtype=u8)}),
            "nsa_cache4_append": ([k, k.clone(), *cache], rows | {"q": q}),
            "nsa_cache4_read": ([*cache, 5], {}),
            "nsa_cache4_decode": ([q[:, :, :1].contiguous(), *cache], {"workspace": of(1 << 24, dtype=u8)})}


@pytest.mark.parametrize("name", NAMES)
def test_calls_go_through_their_raw_functions(monkeypatch, name):
    def out_of_reach(*a, **k):
        raise AssertionError("the library was reached past the raw function")

    monkeypatch.setattr(bsa, "_one_device", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bsa, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(bsa, "load_library", out_of_reach)
    got = []
    for n in NAMES:
        monkeypatch.setattr(bsa, n + "_raw", lambda *a, n=n, **k: got.append((n, a)) or 0)
    args, more = calls()[name]
    getattr(bsa, name)(*args, **more)
    assert len(got) == 1 and got[0][0] == name
    first = args[0].data_ptr()
    assert got[0][1][0] == first
    # and a status that is not success is an error
    monkeypatch.setattr(bsa, "load_library", lambda: type("L", (), {"bsa_status_string": lambda self, s: b"shape"})())
    monkeypatch.setattr(bsa, name + "_raw", lambda *a, **k: 2)
    with pytest.raises(bsa.BsaError) as e:
        getattr(bsa, name)(*args, **more)
    assert e.value.status == 2
