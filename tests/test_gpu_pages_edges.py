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


def negative_pages(pool, new):
    """Whether a page below 0 is served, or gets new tokens."""
    held = pool.held[:]
    slots, _ = pool.reserve(new)
    bad = False
    for b, s in enumerate(slots):
        if s is not None:
            bad |= any(p < 0 for p in pool.table[b][held[b]:pool.held[b]])
            bad |= any(pool.table[b][p // pool.page] < 0 for p in range(pool.len[b], pool.len[b] + new[b]))
    return bad


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("with_slots", [True, False])
@pytest.mark.parametrize("B", [4, 1300])
@pytest.mark.parametrize("where", ["none", "served", "served, refused", "below the top", "last of the context", "held ahead", "context", "behind the tokens", "no new tokens"])
def test_pages_below_zero(dev, where, B, with_slots, packed):  # noqa: F811
    """Bit 2 for a page below 0 that is served or that new tokens go to, with slots and without."""
    b = B - 2                                          # this one's pages are looked at
    lengths = [11] * B                                 # two pages of 8, five new tokens go to these alone
    new = [5] * B
    lengths[1], new[1] = 8, 3                          # one page, another is asked for
    lengths[b], new[b] = 12, 30                        # two, and four of these that are held ahead
    if where == "no new tokens":
        new[b] = 0
    pool = Pool(dev, lengths, 8, 9, 3)
    pool.held[b] = 7
    pool.table[b][2:7] = range(5000, 5005)
    if where == "served":
        pool.stack[pool.free - 1] = -5
    elif where == "served, refused":
        pool.free, pool.stack[0] = 0, -5
    elif where == "below the top":
        pool.stack[0] = -5
    elif where != "none":
        pool.table[b][{"last of the context": 1, "held ahead": 4, "context": 0, "behind the tokens": 6, "no new tokens": 1}[where]] = -3
    pool.up()
    want = where in ("served", "last of the context", "held ahead")
    kw = dict(S=max(new), n_new=ints(new, dev))
    shape = (B, max(new))
    if packed:
        kw, shape = dict(row_start=ints([sum(new[:i]) for i in range(B + 1)], dev)), (sum(new),)
    slots = torch.full(shape, 55, dtype=torch.int64, device=dev) if with_slots else None
    sv.spec_kv_reserve(*pool.args(), slots=slots, errors=pool.errors, **kw)
    assert negative_pages(pool, new) == want
    pool.same()
    assert pool.errors.item() == (CACHE_BIT if want else 0) | (PAGES_BIT if where == "served, refused" else 0)
