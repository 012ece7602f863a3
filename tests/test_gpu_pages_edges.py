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


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("first", [0, 3])
@pytest.mark.parametrize("B,kind", [(5, "any"), (64, "any"), (1500, "short"), (2600, "empty"), (1025, "long last"), (2048, "mixed")])
def test_many_packed_rows(dev, B, kind, first, offset):  # noqa: F811
    """From 131072 rows on a thread writes four slots: groups that hold several sequences, start before the first row or
    end behind the last, lie across 1024 sequences, and slots that are not 16-byte aligned."""
    total, page = 140003, 16
    rng = random.Random(B)
    if kind == "short":      # most of one to three tokens
        new = [rng.randint(1, 3) for _ in range(B)]
    elif kind == "empty":
        new = [rng.choice([0, 0, 0, 1, 2, 70]) for _ in range(B)]
    elif kind == "mixed":
        new = [rng.choice([0, 1, 5, 60, 61, 62, 63]) for _ in range(B)]
    else:
        new = [rng.randint(0, 2 * total // B) if kind == "any" else 1 for _ in range(B)]
    new[B // 2] += 1
    big = B - 1 if kind == "long last" else 1023 if B > 1024 else 0     # the last of the first 1024, where there are more
    new[big] += max(0, total - sum(new))
    total = sum(new)
    lengths = [rng.choice([0, 0, rng.randint(0, 40)]) for _ in range(B)]
    ask = [-(-(a + n) // page) - -(-a // page) for a, n in zip(lengths, new)]
    stock = sum(ask) - ask[-1]                                          # the last that asks is refused
    pool = Pool(dev, lengths, page, -(-(40 + max(new)) // page), stock, seed=B)
    rows = total + first + 2
    starts = [first]
    for n in new:
        starts.append(starts[-1] + n)
    room = torch.full((rows + 4,), 55, dtype=torch.int64, device=dev)
    slots = room[offset:offset + rows]
    sv.spec_kv_reserve(*pool.args(), row_start=ints(starts, dev), slots=slots, errors=pool.errors)
    want, bits = pool.reserve(new)
    pool.same()
    assert pool.errors.item() == bits
    flat = [-1] * first
    for s, n in zip(want, new):
        flat += [-1] * n if s is None else s
    assert slots.tolist() == flat + [-1] * 2
    assert (room[:offset] == 55).all() and (room[offset + rows:] == 55).all()


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("B,S", [(1500, 101), (3, 50001), (1030, 131)])
def test_many_rows_a_sequence(dev, B, S, offset):  # noqa: F811
    """The same with S rows a sequence, not all of them real."""
    rng = random.Random(S)
    page = 8
    new = [rng.randint(0, S) for _ in range(B)]
    lengths = [rng.randint(0, 30) for _ in range(B)]
    pool = Pool(dev, lengths, page, -(-(30 + S) // page), sum(new) // page + B, seed=S)
    room = torch.full((B * S + 4,), 55, dtype=torch.int64, device=dev)
    slots = room[offset:offset + B * S].view(B, S)
    sv.spec_kv_reserve(*pool.args(), S=S, n_new=ints(new, dev), slots=slots, errors=pool.errors)
    want, bits = pool.reserve(new, S)
    pool.same()
    assert pool.errors.item() == bits
    assert slots.tolist() == [(s or []) + [-1] * (S - len(s or [])) for s in want]
    assert (room[:offset] == 55).all() and (room[offset + B * S:] == 55).all()
