"""GPU: the selection operators at the borders of their launch rules and of
their documented ranges, against the float64 oracle (tolerances as in
``test_gpu_nsa_cache.py``)."""

import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from test_gpu_nsa_cache import Pool, check_append, check_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_tra_gb300 import build

    build.build()
    bsa.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert bsa.device_error() == 0


# ------------------------------------------------------------------- append


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_around_every_warp_of_threads(D, page):
    """As many new tokens as make the units of a page one more, one less or exactly what a number of warps takes."""
    for n in (2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129):
        check_append(2, 2, 1, n, D, page, [0, 3 * page - 2], seed=n + D + page)


# ------------------------------------------------------------------- decode


@pytest.mark.parametrize("D,page", [(16, 16), (64, 64), (128, 32), (32, 128)])
@pytest.mark.parametrize("short", [0, 1, 15, 16, 127, 128, 32 * 128 + 1])
def test_decode_of_the_longest_sequences(D, page, short):
    """Tokens up to the largest number that a table may hold (the next to 2^31), almost all on pages that the table does
    not have; without those the sequence is a short one over the same pages."""
    max_pages = (2 ** 31 - 1) // page
    n = max_pages * page - short
    last = (n - 1) // page
    held = sorted({0, 5, last // 2, last - 32, last - 1, last})
    pool = Pool(1, 1, D, page, len(held), seed=D + short).clean()
    dense = pool.table
    q = torch.randn((1, 3, 1, D), generator=torch.Generator().manual_seed(short)).to(torch.bfloat16).cuda()
    tokens = (len(held) - 1) * page + (n - 1) % page + 1
    pool.table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    pool.table[0, held] = dense[0]
    args = pool.args()
    pool.table = dense
    idx = torch.tensor(held, dtype=torch.int32, device="cuda").view(1, 1, 1, -1)
    for length in (n, 2 ** 31 - 1) if short == 0 else (n,):
        lt = torch.tensor([length], dtype=torch.int32, device="cuda")
        for pick in (None, idx):
            out, lse = bsa.nsa_select_decode(q, *args, lt, block_idx=pick, return_lse=True)
            torch.cuda.synchronize()
            check_decode(out, lse, q, pool, [tokens], None)


def test_decode_of_the_least_lengths():
    pool = Pool(2, 1, 64, 32, 3, seed=1).clean()
    q = torch.randn((2, 2, 1, 64)).to(torch.bfloat16).cuda()
    lt = torch.tensor([-2 ** 31, -1], dtype=torch.int32, device="cuda")
    for pick in (None, torch.zeros((2, 1, 1, 2), dtype=torch.int32, device="cuda")):
        out, lse = bsa.nsa_select_decode(q, *pool.args(), lt, block_idx=pick, return_lse=True)
        assert not out.any() and (lse == -1.0e9).all()
