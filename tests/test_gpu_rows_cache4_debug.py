"""GPU: the 4-bit cache and the rows' norm and rotation through the debug build, which checks page and token indexes
before the access: no violation may be recorded, and outputs must equal the release build's bit for bit."""

import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from test_gpu_nsa_ops_debug import both, debug_lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,Hkv,D,page,S", [(3, 8, 2, 64, 32, 0), (3, 8, 2, 128, 64, 4), (320, 4, 1, 32, 16, 3),
                                               (310, 3, 1, 128, 64, 2), (2, 16, 1, 16, 128, 0), (600, 2, 1, 128, 16, 0)])
def test_cache4_debug_build(debug_lib, B, Hq, Hkv, D, page, S):  # noqa: F811
    n, pages = 2 * page + 3, 4
    g = torch.Generator().manual_seed(D)
    k, v, q = (torch.randn(B, h, n, D, generator=g).to(torch.bfloat16).cuda() for h in (Hkv, Hkv, Hq))
    table = torch.randperm(B * pages, generator=g).view(B, pages).int()
    table[0, 1] = B * pages + 7  # a page outside the pool
    held = torch.arange(B) % (page + 1)
    held, table = held.int().cuda(), table.cuda()
    freq, w = (100.0 ** (-torch.arange(0, D, 2) / D)).cuda(), torch.linspace(0.5, 1.5, D).cuda()
    idx = torch.randint(-1, pages + 1, (B, Hkv, 1, S), generator=g).cuda() if S else None

    def run():
        codes = [torch.zeros(B * pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(B * pages, Hkv, page, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
        qr = bsa.nsa_cache4_append(k, v, *codes, *scales, table, held, inv_freq=freq, q=q, q_weight=w, k_weight=w)
        out, lse = bsa.nsa_cache4_decode(qr[:, :, -1:], *codes, *scales, table, held + n, block_idx=idx, return_lse=True)
        back = bsa.nsa_cache4_read(*codes, *scales, table, held + n, n, starts=held)
        rows = bsa.qk_norm_rope_forward(q, k, w, w, freq)
        return (qr, *codes, *scales, out, lse, *back, *rows, *bsa.qk_norm_rope_backward(q, k, *rows, w, w, freq))

    both(debug_lib, run)


@pytest.mark.parametrize("B,Hq,Hkv,D,page", [(3, 8, 2, 64, 32), (2, 16, 1, 128, 128), (600, 2, 1, 128, 16), (40, 9, 1, 32, 64)])
def test_cache4_debug_build_of_long_tables(debug_lib, B, Hq, Hkv, D, page):  # noqa: F811
    g = torch.Generator().manual_seed(B)
    pages = 5
    codes = [torch.randint(0, 256, (B * pages, Hkv, page, D // 2), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = [torch.randint(0x30, 0x40, (B * pages, Hkv, page, D // 16), generator=g, dtype=torch.uint8).cuda()
              for _ in range(2)]
    table = torch.full((B, 20000 // page), -1, dtype=torch.int32)
    table[:, :pages] = torch.randperm(B * pages, generator=g).view(B, pages)
    table[0, 1] = B * pages + 7  # a page outside the pool
    held = (torch.arange(B) * 37 % (pages * page + 1)).int().cuda()
    held[-1] = 19000  # most of it on pages that the table does not have
    table, q = table.cuda(), torch.randn((B, Hq, 1, D), generator=g).to(torch.bfloat16).cuda()
    both(debug_lib, lambda: bsa.nsa_cache4_decode(q, *codes, *scales, table, held, return_lse=True))
