"""Page tables and slots built on the GPU, against lists: whole numbers, equal."""
import random

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402

pytestmark = pytest.mark.gpu
CACHE_BIT, PAGES_BIT = 4, 8


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


class Pool:
    """Sequences with shuffled pages, and the stack of the others."""

    def __init__(self, dev, lengths, page, width, free, seed=0, extra=0, spare=0):
        rng = random.Random(seed)
        self.dev, self.page, self.width = dev, page, width
        self.len = list(lengths)
        self.held = [min(width, -(-n // page) + (rng.randint(0, extra) if extra else 0)) for n in lengths]
        ids = list(range(sum(self.held) + free))
        rng.shuffle(ids)
        self.table = []
        for h in self.held:
            self.table.append([ids.pop() for _ in range(h)] + [-7] * (width - h))
        self.stack = ids + [-9] * (spare + sum(self.held))
        self.free = free
        self.up()

    def up(self):
        d = self.dev
        self.t_table = ints(self.table, d).view(len(self.len), self.width)
        self.t_len, self.t_held = ints(self.len, d), ints(self.held, d)
        self.t_stack, self.t_free = ints(self.stack, d), ints([self.free], d)
        self.errors = torch.zeros(1, dtype=torch.int32, device=d)

    def args(self):
        return self.t_table, self.t_len, self.t_held, self.t_stack, self.t_free, self.page

    def reserve(self, new, most=None):
        """The definition; returns the slots of each sequence's new tokens (None: refused) and the error bits."""
        asked, bits, out, top = 0, 0, [], self.free
        for b, n in enumerate(new):
            length, held = self.len[b], self.held[b]
            if length < 0 or n < 0 or (most is not None and n > most) or not 0 <= held <= self.width or length + n > self.width * self.page:
                out.append(None)
                bits |= CACHE_BIT
                continue
            want = max(0, -(-(length + n) // self.page) - held)
            asked += want
            if want and asked > top:
                self.table[b][held:held + want] = [-1] * want
                out.append(None)
                bits |= PAGES_BIT
                continue
            for _ in range(want):
                self.free -= 1
                self.table[b][self.held[b]] = self.stack[self.free]
                self.held[b] += 1
            out.append([self.table[b][p // self.page] * self.page + p % self.page for p in range(length, length + n)])
        return out, bits

    def release(self):
        back, bits = [], 0
        for b, n in enumerate(self.len):
            keep = -(-n // self.page)
            if n < 0 or keep > self.held[b]:
                bits |= CACHE_BIT
                continue
            back += self.table[b][keep:self.held[b]]
            self.held[b] = keep
        self.stack[self.free:self.free + len(back)] = back[::-1]
        self.free += len(back)
        return bits

    def same(self, held=None, free=None):
        assert self.t_table.tolist() == self.table
        assert (self.t_held if held is None else held).tolist() == self.held
        assert self.t_stack.tolist() == self.stack
        assert (self.t_free if free is None else free).tolist() == [self.free]


def padded(slots, S):
    return [(s or []) + [-1] * (S - len(s or [])) for s in slots]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,S,page,stock", [(1, 1, 8, 1.0), (3, 9, 16, 0.5), (7, 32, 8, 2.0), (64, 15, 16, 0.9), (511, 3, 8, 0.7), (512, 5, 32, 1.0),
                                            (513, 9, 8, 0.99), (1500, 15, 8, 0.6), (3001, 17, 16, 1.1), (40, 1000, 8, 0.8), (700, 900, 64, 0.95)])
def test_reserve(dev, B, S, page, stock, in_place):
    rng = random.Random(B * S)
    lengths = [rng.randint(0, 90) for _ in range(B)]
    new = [rng.randint(0, S) for _ in range(B)]
    need = sum(-(-(a + n) // page) - -(-a // page) for a, n in zip(lengths, new))
    pool = Pool(dev, lengths, page, -(-(90 + S) // page) + 2, int(need * stock), seed=B, extra=1)
    slots = torch.full((B, S), 55, dtype=torch.int64, device=dev)
    held, free = (None, None) if in_place else (torch.empty_like(pool.t_held), torch.empty_like(pool.t_free))
    got = sv.spec_kv_reserve(*pool.args(), S=S, n_new=ints(new, dev), slots=slots, errors=pool.errors, held_out=held, free_count_out=free)
    before = pool.held[:], pool.free
    want, bits = pool.reserve(new, S)
    pool.same(got, free)
    assert slots.tolist() == padded(want, S)
    assert pool.errors.item() == bits
    if not in_place:   # the counts before it are as they were: the call can be made again
        assert (pool.t_held.tolist(), pool.t_free.item()) == before
        slots.fill_(3)
        sv.spec_kv_reserve(*pool.args(), S=S, n_new=ints(new, dev), slots=slots, held_out=held, free_count_out=free)
        pool.same(held, free)
        assert slots.tolist() == padded(want, S)


@pytest.mark.parametrize("B,total,page", [(1, 1, 8), (5, 300, 16), (64, 50000, 64), (515, 9000, 8), (1100, 200, 16)])
@pytest.mark.parametrize("with_slots", [True, False])
def test_reserve_packed(dev, B, total, page, with_slots):
    rng = random.Random(total)
    cut = sorted(rng.randint(0, total) for _ in range(B - 1))
    new = [b - a for a, b in zip([0] + cut, cut + [total])]
    lengths = [rng.choice([0, 0, rng.randint(0, 40)]) for _ in range(B)]
    pool = Pool(dev, lengths, page, -(-(40 + max(new)) // page), -(-total // page) + B, seed=B)
    first, rows = 3, total + 8
    starts = [first]
    for n in new:
        starts.append(starts[-1] + n)
    slots = torch.full((rows,), 55, dtype=torch.int64, device=dev) if with_slots else None
    sv.spec_kv_reserve(*pool.args(), row_start=ints(starts, dev), slots=slots, errors=pool.errors)
    want, bits = pool.reserve(new)
    pool.same()
    assert pool.errors.item() == bits == 0
    if with_slots:
        assert slots.tolist() == [-1] * first + sum(want, []) + [-1] * (rows - first - total)


@pytest.mark.parametrize("starts", [[0, 5, 4, 9], [-1, 3, 5, 9], [0, 3, 5, 13], [4, 3, 3, 3]])
def test_packed_starts_that_cannot_be_used(dev, starts):
    pool = Pool(dev, [3, 0, 9], 8, 4, 10)
    slots = torch.full((12,), 55, dtype=torch.int64, device=dev)
    sv.spec_kv_reserve(*pool.args(), row_start=ints(starts, dev), slots=slots, errors=pool.errors)
    pool.same()
    assert (slots == -1).all() and pool.errors.item() == CACHE_BIT


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,hi,page,ended", [(1, 50, 8, 0.0), (5, 400, 16, 0.4), (64, 100, 8, 1.0), (513, 200, 16, 0.1), (2100, 120, 8, 0.5), (30, 9000, 8, 0.5)])
def test_release(dev, B, hi, page, ended, in_place):
    rng = random.Random(B)
    lengths = [rng.randint(0, hi) for _ in range(B)]
    pool = Pool(dev, lengths, page, -(-hi // page) + 3, 11, seed=B, extra=3, spare=5)
    pool.len = [0 if rng.random() < ended else n for n in lengths]
    pool.t_len = ints(pool.len, dev)
    held, free = (None, None) if in_place else (torch.empty_like(pool.t_held), torch.empty_like(pool.t_free))
    got = sv.spec_kv_release(*pool.args(), errors=pool.errors, held_out=held, free_count_out=free)
    bits = pool.release()
    pool.same(got, free)
    assert pool.errors.item() == bits == 0


@pytest.mark.parametrize("B", [6, 1300])
def test_release_undoes_reserve(dev, B):
    rng = random.Random(3)
    pool = Pool(dev, [rng.randint(0, 200) for _ in range(B)], 8, 40, 4 * B, seed=1)
    before = pool.t_stack.clone(), pool.t_held.clone(), pool.t_free.clone()
    sv.spec_kv_reserve(*pool.args(), S=20, errors=pool.errors)
    assert not torch.equal(pool.t_held, before[1])
    sv.spec_kv_release(*pool.args(), errors=pool.errors)
    assert all(torch.equal(a, b) for a, b in zip((pool.t_stack, pool.t_held, pool.t_free), before))
    assert pool.errors.item() == 0


BAD = {"length": dict(len={1: -1}), "length past the table": dict(len={1: 8 * 6 + 1}), "held": dict(held={1: -2}), "held past the table": dict(held={1: 7}),
       "new": dict(new={1: -3}), "too many new": dict(new={1: 6})}


@pytest.mark.parametrize("B", [3, 600])
@pytest.mark.parametrize("what", BAD.values(), ids=BAD.keys())
def test_sequences_that_cannot_be_used(dev, what, B):
    """They are refused; the others are served as if they asked for nothing."""
    pool = Pool(dev, [10, 20] + [17] * (B - 2), 8, 6, 3 * B)
    new = [5] * B
    for b, v in what.get("len", {}).items():
        pool.len[b] = v
    for b, v in what.get("held", {}).items():
        pool.held[b] = v
    for b, v in what.get("new", {}).items():
        new[b] = v
    pool.up()
    slots = torch.full((B, 5), 55, dtype=torch.int64, device=dev)
    sv.spec_kv_reserve(*pool.args(), S=5, n_new=ints(new, dev), slots=slots, errors=pool.errors)
    want, bits = pool.reserve(new, 5)
    pool.same()
    assert want[1] is None and slots.tolist() == padded(want, 5) and pool.errors.item() == bits == CACHE_BIT


@pytest.mark.parametrize("what", [dict(len={1: -1}), dict(len={1: 41})])
def test_release_of_lengths_that_cannot_be_used(dev, what):
    pool = Pool(dev, [10, 20, 33], 8, 9, 3, extra=2)
    pool.len[0], pool.len[1] = 0, what["len"][1]
    pool.t_len = ints(pool.len, dev)
    sv.spec_kv_release(*pool.args(), errors=pool.errors)
    assert pool.release() == CACHE_BIT
    pool.same()
    assert pool.errors.item() == CACHE_BIT


@pytest.mark.parametrize("free", [-1, 1000])
def test_stack_heights_that_cannot_be_used(dev, free):
    pool = Pool(dev, [10, 20, 33], 8, 9, 30)
    pool.t_free.fill_(free)
    pool.free = free
    slots = torch.full((3, 4), 55, dtype=torch.int64, device=dev)
    sv.spec_kv_reserve(*pool.args(), S=4, slots=slots, errors=pool.errors)
    pool.same()
    assert (slots == -1).all() and pool.errors.item() == CACHE_BIT
    pool.errors.zero_()
    pool.t_len.zero_()
    sv.spec_kv_release(*pool.args(), errors=pool.errors)
    pool.same()
    assert pool.errors.item() == CACHE_BIT


def test_stack_that_would_grow_past_its_capacity(dev):
    pool = Pool(dev, [10, 20, 33], 8, 9, 30)
    pool.t_stack = pool.t_stack[:38].clone()
    pool.stack = pool.stack[:38]
    pool.t_len.zero_()
    sv.spec_kv_release(*pool.args(), errors=pool.errors)   # 10 pages onto 30
    pool.same()
    assert pool.errors.item() == CACHE_BIT


def test_pages_below_zero_are_reported(dev):
    pool = Pool(dev, [8, 8], 8, 3, 4)
    pool.t_stack[3] = -5
    slots = torch.empty((2, 1), dtype=torch.int64, device=dev)
    sv.spec_kv_reserve(*pool.args(), S=1, slots=slots, errors=pool.errors)
    assert slots[0].item() == -1 and slots[1].item() >= 0 and pool.errors.item() == CACHE_BIT


def test_slots_past_32_bits(dev):
    """Pages of 1024 positions with ids above 2^21."""
    pool = Pool(dev, [1000, 0], 1024, 3, 6)
    pool.t_stack += 1 << 22
    pool.t_table[0, 0] = 1 << 23
    slots = torch.empty((2, 30), dtype=torch.int64, device=dev)
    sv.spec_kv_reserve(*pool.args(), S=30, slots=slots, errors=pool.errors)
    assert slots[0].tolist() == [(1 << 33) + 1000 + i for i in range(24)] + [pool.t_table[0, 1].item() * 1024 + i for i in range(6)]
    assert slots[1].tolist() == [pool.t_table[1, 0].item() * 1024 + i for i in range(30)] and slots[1, 0].item() > 1 << 32


def test_refused_sequences_are_not_appended_to(dev):
    """The -1 that a refused request leaves is what spec_kv_append reports."""
    pool = Pool(dev, [8, 8], 8, 3, 1)
    sv.spec_kv_reserve(*pool.args(), S=2, errors=pool.errors)
    assert pool.errors.item() == PAGES_BIT
    n = 4
    k = torch.ones(2, 2, 1, 64, dtype=torch.bfloat16, device=dev)
    kc, vc = (torch.zeros(n, 1, 8, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    sv.spec_kv_append(k, k, kc, vc, pool.t_table, pool.t_len, errors=pool.errors)
    assert pool.errors.item() == PAGES_BIT | CACHE_BIT
    got = pool.t_table[0, 1].item()
    assert (kc[got, 0, :2] == 1).all() and kc.sum().item() == 2 * 64


def test_flags_are_read_and_cleared(dev):
    pool = Pool(dev, [8, 8], 8, 3, 1)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    sv.spec_kv_reserve(*pool.args(), S=2, errors=ws.view(torch.int32))
    W = type("W", (), {"ptr": ws.data_ptr()})
    assert sv.sv_workspace_errors(W) == PAGES_BIT
    assert sv.sv_workspace_errors(W) == 0


def test_capture_and_another_stream(dev):
    """Rounds of a captured reserve and release, in place, on changing lengths."""
    rng = random.Random(9)
    B, S = 50, 9
    pool = Pool(dev, [rng.randint(0, 100) for _ in range(B)], 8, 40, 300, seed=2)
    slots = torch.empty((B, S), dtype=torch.int64, device=dev)
    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        sv.spec_kv_reserve(*pool.args(), S=S, slots=slots, errors=pool.errors)
    h = torch.cuda.CUDAGraph()
    with torch.cuda.graph(h):
        sv.spec_kv_release(*pool.args(), errors=pool.errors)
    for _ in range(6):
        g.replay()
        torch.cuda.synchronize()
        want, _ = pool.reserve([S] * B)
        assert slots.tolist() == padded(want, S)
        pool.len = [0 if rng.random() < 0.2 else n + rng.randint(1, S) for n in pool.len]
        pool.t_len.copy_(ints(pool.len, dev))
        h.replay()
        torch.cuda.synchronize()
        pool.release()
        pool.same()
    assert pool.errors.item() == 0


def test_empty_calls(dev):
    pool = Pool(dev, [], 8, 4, 3)
    sv.spec_kv_reserve(*pool.args(), S=4)
    sv.spec_kv_release(*pool.args())
    pool = Pool(dev, [5, 9], 8, 4, 3)
    sv.spec_kv_reserve(*pool.args(), S=0, errors=pool.errors)
    pool.same()
    assert pool.errors.item() == 0
