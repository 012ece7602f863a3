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


# starts, rows -> the sequence and index of each usable row, the rows that are NaN; the rest are no sequence's
STARTS = {
    "first": ([3, 0, 5, 8], {5: (2, 0), 6: (2, 1), 7: (2, 2)}, [3, 4]),
    "middle": ([0, 5, 2, 8], {0: (0, 0), 1: (0, 1), 5: (2, 3), 6: (2, 4), 7: (2, 5)}, [2, 3, 4]),
    "last": ([0, 4, 9, 6], {0: (0, 0), 1: (0, 1), 2: (0, 2), 3: (0, 3)}, [4, 5]),
    "beyond": ([0, 9, 4], {}, [0, 1, 2, 3]),
    "where no row looks": ([0, 4, 9, 4], {0: (0, 0), 1: (0, 1), 2: (0, 2), 3: (0, 3)}, []),
    "negative": ([-2, 3, 6], {3: (1, 0), 4: (1, 1), 5: (1, 2)}, [0, 1, 2]),
}


@pytest.mark.parametrize("starts,usable,nan", STARTS.values(), ids=STARTS.keys())
def test_append_row_starts_that_do_not_ascend(dev, starts, usable, nan):
    rows, Hq, Hkv, D, page = 8, 4, 2, 64, 8
    B = len(starts) - 1
    ctx = [3 * b for b in range(B)]
    cache = Cache([c + 10 for c in ctx], Hkv, D, page, "bf16", dev, 18)
    gen = torch.Generator(device=dev).manual_seed(19)
    q, k, v = (torch.randn(rows, h, D, generator=gen, device=dev).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    before = cache.k.clone(), cache.v.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = sv.spec_kv_append(k, v, cache.k, cache.v, cache.table, ints(ctx, dev), q=q, row_start=ints(starts, dev), errors=err)
    assert err.item() == CACHE_BIT
    for t in range(rows):
        if t in usable:
            assert torch.equal(out[t], q[t]), t
        elif t in nan:
            assert out[t].isnan().all(), t
        else:
            assert (out[t] == 0).all(), t
    want = [x.clone() for x in before]
    for t, (b, i) in usable.items():
        p, s = cache.at(b, [ctx[b] + i])
        want[0][p, :, s], want[1][p, :, s] = k[t], v[t]
    for w, got in zip(want, (cache.k, cache.v)):
        assert torch.equal(w.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("starts,usable,nan", STARTS.values(), ids=STARTS.keys())
def test_read_row_starts_that_do_not_ascend(dev, starts, usable, nan):
    rows, Hkv, D = 8, 2, 64
    B = len(starts) - 1
    first = [2 * b for b in range(B)]
    cache = Cache([f + 10 for f in first], Hkv, D, 8, "e4m3", dev, 20)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    k, v = sv.spec_kv_read(cache.k, cache.v, cache.table, ints(first, dev), ints(starts, dev), rows, dtype=torch.float32,
                           errors=err, **cache.scales())
    assert err.item() == CACHE_BIT
    for t in range(rows):
        for got, name in ((k, "k"), (v, "v")):
            if t in usable:
                b, i = usable[t]
                assert torch.equal(got[t], cache.rows64(name, b, [first[b] + i])[0].float()), t
            elif t in nan:
                assert got[t].isnan().all(), t
            else:
                assert (got[t] == 0).all(), t


@pytest.mark.parametrize("Hkv,D", [(1, 64), (5, 128), (7, 256)])   # blocks of different shapes
def test_many_sequences_with_one_wrong_start(dev, Hkv, D):
    """More sequences than threads: the fault is reported wherever it lies."""
    B = 5000
    cache = Cache([1], Hkv, D, 8, "bf16", dev, 21)
    table = cache.table.expand(B, -1).contiguous()
    k = torch.zeros(4, Hkv, D, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    starts, zero = (torch.zeros(B + n, dtype=torch.int32, device=dev) for n in (1, 0))
    calls = (lambda: sv.spec_kv_append(k, k, cache.k, cache.v, table, zero, row_start=starts, errors=err),
             lambda: sv.spec_kv_read(cache.k, cache.v, table, zero, starts, 4, errors=err))
    for call in calls:
        call()
    assert err.item() == 0
    for at in (1, 190, 191, 192, 193, 223, 224, 255, 256, 257, 2500, B - 1):
        starts[at] = 1
        for call in calls:
            err.zero_()
            call()
            assert err.item() == CACHE_BIT, at
        starts[at] = 0
