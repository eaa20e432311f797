"""GPU: the selection operators through the debug build.

The library compiled with -DBSA_DEBUG checks gather indices and TMA
coordinates against their tensors before the access and records a violation
in the device error word.  The backward, the cache append and the decode run
on odd and degenerate inputs through it: no violation may be recorded, and
every output must equal the release build's bit for bit.
"""

import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_tra_gb300 import build

    build.build()
    bsa.load_library()
    torch.cuda.set_device(0)
    path = build.build(debug=True)
    yield path
    assert bsa.device_error() == 0


def both(path, fn):
    a = fn()
    torch.cuda.synchronize()
    with bsa.using_library(path):
        assert bsa.device_error() == 0
        b = fn()
        torch.cuda.synchronize()
        err = bsa.device_error()
    assert err == 0, f"debug build recorded device error {err}"
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def odd_rows(idx, n_blk):
    """Empty rows, future-only rows, repeats and out-of-range entries."""
    a = idx.clone()
    T = a.shape[2]
    a[:, :, : T // 8] = -1
    a[:, :, T // 8: T // 4, 0] = n_blk - 1
    a[:, :, T // 8: T // 4, 1:] = -1
    a[:, :, T // 2:, -1] = a[:, :, T // 2:, 0]
    a[:, :, -3:, 1] = n_blk + 5
    return a


@pytest.mark.parametrize("Hq,Hkv,D,bs,S", [(16, 2, 128, 64, 8), (16, 1, 64, 64, 16), (12, 4, 64, 64, 5), (5, 1, 128, 64, 3),
                                           (8, 2, 32, 32, 6), (2, 2, 16, 16, 4), (6, 2, 128, 128, 4)])
def test_backward_debug_build(debug_lib, Hq, Hkv, D, bs, S):
    q, k, v, idx = workloads.nsa_inputs(1, Hq, Hkv, 512, D, bs, S, seed=D + bs)
    q, k, v, idx = q.cuda(), k.cuda(), v.cuda(), odd_rows(idx, 512 // bs).cuda()
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(D)).to(torch.bfloat16).cuda()
    out, lse = bsa.nsa_select_forward(q, k, v, idx, bs, return_lse=True)
    both(debug_lib, lambda: bsa.nsa_select_backward(q, k, v, idx, out, lse, do, bs))


@pytest.mark.parametrize("B,Hq,Hkv,D,page,S", [(3, 8, 2, 64, 32, 0), (3, 8, 2, 128, 64, 4), (320, 4, 1, 32, 16, 3),
                                               (310, 3, 1, 128, 64, 2), (2, 16, 1, 16, 128, 0)])
def test_cache_debug_build(debug_lib, B, Hq, Hkv, D, page, S):
    n, pages = 2 * page + 3, 4
    g = torch.Generator().manual_seed(D)
    k, v, q = (torch.randn(B, h, n, D, generator=g).to(torch.bfloat16).cuda() for h in (Hkv, Hkv, Hq))
    table = torch.randperm(B * pages, generator=g).view(B, pages).int()
    table[0, 1] = B * pages + 7  # a page outside the pool
    held = torch.arange(B) % (page + 1)
    held, table = held.int().cuda(), table.cuda()
    freq = (100.0 ** (-torch.arange(0, D, 2) / D)).cuda()
    idx = torch.randint(-1, pages + 1, (B, Hkv, 1, S), generator=g).cuda() if S else None

    def run():
        codes = [torch.zeros(B * pages, Hkv, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.ones(B * pages, Hkv, device="cuda") for _ in range(2)]
        qr = bsa.nsa_cache_append(k, v, *codes, *scales, table, held, inv_freq=freq, q=q)
        out, lse = bsa.nsa_select_decode(qr[:, :, -1:], *codes, *scales, table, held + n, block_idx=idx, return_lse=True)
        return (qr, *codes, *scales, out, lse)

    both(debug_lib, run)
