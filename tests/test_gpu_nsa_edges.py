"""GPU: the selection operators at the borders of their launch rules and of
their documented ranges, against the float64 oracle (tolerances as in
``test_gpu_nsa_cache.py``)."""

import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from test_gpu_nsa_cache import check_append

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
