"""Calls of the page operators that lie at the edges of what they take."""
import random

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from test_gpu_pages import CACHE_BIT, PAGES_BIT, Pool, dev, ints  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [3, 1500])
@pytest.mark.parametrize("starts", [[0, 2000000000, -2000000000, 9], [0, 2147483647, -2147483648, 9], [0, 2000000000, -2000000000, -2000000000]])
def test_packed_starts_whose_differences_wrap(dev, starts, B):  # noqa: F811
    """Differences of int32 that come out positive: such starts do not ascend, and the whole call is refused."""
    pool = Pool(dev, [3] * B, 8, 4, 10)
    slots = torch.full((12,), 55, dtype=torch.int64, device=dev)
    for at in {0, B - 3}:
        packed = [0] * at + starts + [starts[-1]] * (B - 3 - at)
        pool.errors.zero_()
        sv.spec_kv_reserve(*pool.args(), row_start=ints(packed, dev), slots=slots, errors=pool.errors)
        pool.same()
        assert (slots == -1).all() and pool.errors.item() == CACHE_BIT
