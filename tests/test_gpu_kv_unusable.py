"""Device data of the cache operators that cannot be used, one kind at a time:
what it reaches, and what it leaves as it was."""
import random

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from kv_helpers import Cache, parents_of  # noqa: E402

pytestmark = pytest.mark.gpu
CACHE_BIT = 4


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("what", [-0.01, -1e30, float("-inf")])
@pytest.mark.parametrize("ctx", [[250, 31], [0, 128], [40000, 1]])
def test_a_negative_value_scale_of_a_node_reaches_only_its_descendants(dev, ctx, what):
    """A negative value scale reads as NaN: the rows that see the node are NaN,
    the other rows of the tree keep every bit."""
    N, D = 7, 128
    rng = random.Random(14)
    cache = Cache([c + N for c in ctx], 2, D, 16, "e4m3", dev, 14)
    gen = torch.Generator(device=dev).manual_seed(15)
    q = torch.randn(2, N, 4, D, generator=gen, device=dev).to(torch.bfloat16)
    parents = ints([parents_of("binary", N, rng) for _ in ctx], dev)
    call = lambda: sv.spec_tree_attention(q, cache.k, cache.v, cache.table, ints(ctx, dev), parent=parents, **cache.scales())  # noqa: E731
    ref = call()
    for b, node in ((0, 1), (0, 6), (1, 5)):
        page, slot = cache.at(b, [ctx[b] + node])
        cache.v_scale[page, 0, slot] = what
    got = call()
    hit = torch.zeros(got.shape, dtype=torch.bool, device=dev)
    for b, n in ((0, 1), (0, 3), (0, 4), (0, 6), (1, 5)):
        hit[b, n, :2] = True
    assert got[hit].isnan().all()
    assert torch.equal(got[~hit], ref[~hit])


def test_a_negative_value_scale_in_the_context(dev):
    """All rows of the key head see it; the other key head's do not."""
    N, D, ctx = 3, 64, [200]
    cache = Cache([203], 2, D, 16, "e4m3", dev, 16)
    q = torch.randn(1, N, 4, D, generator=torch.Generator(device=dev).manual_seed(17), device=dev).to(torch.bfloat16)
    call = lambda: sv.spec_tree_attention(q, cache.k, cache.v, cache.table, ints(ctx, dev), **cache.scales())  # noqa: E731
    ref = call()
    page, slot = cache.at(0, [77])
    cache.v_scale[page, 1, slot] = -0.02
    got = call()
    assert got[:, :, 2:].isnan().all() and torch.equal(got[:, :, :2], ref[:, :, :2])
