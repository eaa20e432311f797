"""CPU: a selection without a slot is no selection of every page.  (Tensors that pass for a device's, and no library
behind them: a refusal that is missed ends in Python.)"""

import types

import pytest
import torch

from block_sparse_attention_tra_gb300 import BsaError, bsa


class Reached(Exception):
    pass


@pytest.fixture
def on_device(monkeypatch):
    def reached(*a, **k):
        raise Reached

    monkeypatch.setattr(bsa, "_one_device", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(bsa, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(bsa, "load_library", reached)


def of(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def calls():
    u8, f32 = torch.uint8, torch.float32
    rest = of(1, 4, dtype=torch.int32), of(1, dtype=torch.int32)
    e4m3 = (of(4, 2, 64, 64, dtype=u8), of(4, 2, 64, 64, dtype=u8), of(4, 2, dtype=f32), of(4, 2, dtype=f32))
    e2m1 = tuple(of(4, 2, 64, w, dtype=u8) for w in (32, 32, 4, 4))
    return [(bsa.nsa_select_decode, (of(1, 8, 1, 64), *e4m3, *rest)),
            (bsa.nsa_cache4_decode, (of(1, 8, 1, 64), *e2m1, *rest))]


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("shape", [(1, 2, 1, 0), (1, 2, 0), (0,), (), (1, 2, 1, 33)])
def test_empty_and_oversized_selections_are_refused(on_device, which, workspace, shape):
    call, args = calls()[which]
    ws = of(1 << 24, dtype=torch.uint8) if workspace else None
    with pytest.raises(BsaError) as e:
        call(*args, block_idx=of(*shape, dtype=torch.int32), workspace=ws)
    assert e.value.status == 2
    with torch.no_grad(), pytest.raises(Reached):  # what is a selection, and none, get past it
        call(*args, block_idx=of(1, 2, 1, 32, dtype=torch.int32), workspace=ws)
    with pytest.raises(Reached):
        call(*args, workspace=ws)
