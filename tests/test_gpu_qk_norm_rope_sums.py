"""GPU: the weights' gradients of the norm and rotation of rows under a bound that counts the kernels' sums.

In units of u = 2^-24: a row's product is off by 26 u of its magnitude (``test_gpu_qk_norm_rope.py``).  Its sum: at most
16 rows of a thread, 5 shuffles, 8 warps; in the second launch every 256th of the blocks one after the other, 3 shuffles,
32 warps: 64 + blocks / 256 roundings.  90 + blocks / 256 u of the sum of magnitudes, 1 for products of roundings: 2^-17
of it up to 9400 blocks.
"""

import numpy as np
import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from oracle import rows as orows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hq,Hkv,T,D,rotary", [(1, 1, 1, 1, 64, 64), (2, 33, 2, 2047, 128, 128), (1, 1, 1, 150001, 16, 16),
                                                 (3, 16, 1, 5000, 48, 32), (1, 5, 17, 9000, 64, 0)])
def test_weights_gradients_under_their_own_bound(dtype, B, Hq, Hkv, T, D, rotary):
    g = torch.Generator().manual_seed(T)
    q, k, dq, dk = (torch.randn((B, h, T, D), generator=g).to(dtype) for h in (Hq, Hkv, Hq, Hkv))
    wq, wk = (1.0 + 0.3 * torch.randn(D, generator=g) for _ in range(2))
    f = bsa.rope_frequencies(rotary)[0] if rotary else None
    on = [None if t is None else t.cuda() for t in (q, k, dq, dk, wq, wk, f)]
    *_, gq, gk = bsa.qk_norm_rope_backward(*on)
    *_, aq, ak = bsa.qk_norm_rope_backward(*on)
    assert torch.equal(gq, aq) and torch.equal(gk, ak)
    blocks = bsa.qk_norm_rope_backward_workspace_size(B, Hq, Hkv, T, D) / (4 * D)  # of both tensors: each has fewer
    pos = np.broadcast_to(np.arange(T), (B, T))
    fr = np.zeros(0) if f is None else f.double().numpy()
    for x, dy, w, got in ((q, dq, wq, gq), (k, dk, wk, gk)):
        _, want, _, sums = orows.backward(x.double().numpy(), dy.double().numpy(), w.double().numpy(), pos, fr, False, 1.0,
                                          1e-6)
        off = np.abs(got.double().cpu().numpy() - want) / (2.0 ** -24 * (91 + blocks / 256) * sums)
        assert off.max() <= 1, f"{off.max():.2f} times its bound"
