"""spec_kv_append, spec_kv_commit and spec_kv_read against their definitions
in 64 bits."""
import random

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from kv_helpers import E4M3, Cache, ancestors, parents_of, rotated64  # noqa: E402

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


def angles(rows, rot, dev):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    a = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], -1).float()


def bits(t):
    return t.contiguous().view(torch.uint8)


def snapshot(cache):
    return [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]


def check_rows(got, ref, dtype, where=""):
    """Dense rows: one rounding to dtype, and fp32 arithmetic over a row whose
    norm and rotation cost at most 16 roundings of its largest magnitude."""
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    bound = unit * ref.abs() + 16 * 2.0 ** -24 * ref.abs().amax(-1, keepdim=True) * 2 ** 0.5 + 1e-37
    assert ((got.double() - ref).abs() <= bound).all(), where


def check_stored(cache, which, b, positions, ref):
    """Stored entries.  e4m3: the scale to fp32 rounding, each value a nearest
    one (half of the gap at its place, a little more for the quotient's own
    rounding)."""
    t, s = (cache.k, cache.k_scale) if which == "k" else (cache.v, cache.v_scale)
    page, slot = cache.at(b, positions)
    if s is None:
        check_rows(t[page, :, slot], ref, torch.bfloat16, which)
        return
    step = (ref.abs().amax(-1) / 448.0).clamp(min=2.0 ** -100)
    got_step = s[page, :, slot].double()
    assert ((got_step - step).abs() <= 24 * 2.0 ** -24 * step).all()
    value = t.view(torch.uint8)[page, :, slot].view(E4M3).double()
    x = ref / step[..., None]
    gap = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    assert ((value - x).abs() <= 0.5 * gap + 64 * 2.0 ** -24 * 448).all(), which


APPEND = [  # ctx, S, tree, Hq, Hkv, D, rot, pairs, norm, page
    ([0], 1, "chain", 4, 1, 64, 64, False, True, 8),
    ([7, 0, 300], 1, "chain", 20, 4, 80, 32, True, False, 16),
    ([15, 16, 17, 1, 200], 15, "binary", 32, 8, 128, 128, False, True, 16),
    ([100, 5], 32, "random", 8, 8, 96, 96, True, True, 32),
    ([31, 2], 9, "chain", 6, 3, 112, 16, False, True, 8),
    ([0, 64], 7, "star", 4, 2, 144, 64, False, False, 64),
    ([9], 31, "random", 5, 1, 192, 192, True, True, 16),
    ([1023, 3], 13, "random", 16, 2, 256, 256, False, True, 1024),
    ([12, 40], 200, "chain", 3, 1, 240, 0, False, True, 128),   # a padded prompt, no rotation
    ([2, 3], 5, "random", 0, 5, 128, 128, False, True, 16),     # keys and values only
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"b{len(c[0])}s{c[1]}{c[2]}h{c[3]}x{c[4]}d{c[5]}r{c[6]}")
def test_append_padded(dev, case, fmt, dtype):
    ctx, S, tree, Hq, Hkv, D, rot, pairs, norm, page = case
    rng = random.Random(len(ctx) * 100 + D)
    B = len(ctx)
    new = [S] + [rng.randint(0, S) for _ in range(B - 1)]
    cache = Cache([c + S for c in ctx], Hkv, D, page, fmt, dev, 2)
    gen = torch.Generator(device=dev).manual_seed(D)
    fused = torch.randn(B, S, Hq + 2 * Hkv, D, generator=gen, device=dev).to(dtype)
    q, k, v = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv], fused[:, :, Hq + Hkv:]
    qn, kn = ((1 + 0.2 * torch.randn(2, D, generator=gen, device=dev)).to(dtype)) if norm else (None, None)
    table = angles(max(ctx) + S, rot, dev) if rot else None
    parents = [parents_of(tree, S, rng) for _ in range(B)]
    before = snapshot(cache)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = sv.spec_kv_append(k, v, cache.k, cache.v, cache.table, ints(ctx, dev), n_new=ints(new, dev),
                            q=q if Hq else None, q_norm=qn if Hq else None, k_norm=kn, eps=1e-5, cos_sin=table,
                            interleaved=pairs, parent=ints(parents, dev) if tree != "chain" else None,
                            errors=err, **cache.scales())
    assert err.item() == 0
    written = torch.zeros(cache.num_pages, page, dtype=torch.bool, device=dev)
    for b in range(B):
        n = new[b]
        if Hq:
            assert (out[b, n:] == 0).all()
        if n == 0:
            continue
        pos = [ctx[b] + len(ancestors(parents[b], i)) - 1 for i in range(n)]
        if Hq:
            check_rows(out[b, :n], rotated64(q[b, :n], qn, table, pos, pairs, 1e-5), dtype, "q")
        places = range(ctx[b], ctx[b] + n)
        check_stored(cache, "k", b, places, rotated64(k[b, :n], kn, table, pos, pairs, 1e-5))
        check_stored(cache, "v", b, places, v[b, :n].double())
        page_ids, slots = cache.at(b, places)
        written[page_ids, slots] = True
    # nothing else in the cache has changed
    after = snapshot(cache)
    for x, y in zip(before, after):
        same = (bits(x).view(*x.shape[:3], -1) == bits(y).view(*x.shape[:3], -1)).all(-1)
        assert (same | written[:, None, :]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("counts", [[5], [1, 0, 300, 2, 0, 77], [3] * 70, [0, 0, 1], list(range(40)) * 30],
                         ids=["one", "ragged", "seventy", "empty_first", "many"])
def test_append_packed(dev, counts, fmt, dtype):
    Hq, Hkv, D, page = 4, 2, 64, 16
    B, T = len(counts), sum(counts)
    ctx = [(7 * b) % 50 for b in range(B)]
    cache = Cache([c + n for c, n in zip(ctx, counts)], Hkv, D, page, fmt, dev, 3)
    gen = torch.Generator(device=dev).manual_seed(T)
    spare = 3   # rows of no sequence at the end
    q, k, v = (torch.randn(T + spare, h, D, generator=gen, device=dev).to(dtype) for h in (Hq, Hkv, Hkv))
    qn, kn = (1 + 0.2 * torch.randn(2, D, generator=gen, device=dev)).to(dtype)
    table = angles(400, 32, dev)
    starts = [sum(counts[:b]) for b in range(B + 1)]
    out = sv.spec_kv_append(k, v, cache.k, cache.v, cache.table, ints(ctx, dev), q=q, q_norm=qn, k_norm=kn,
                            eps=1e-6, cos_sin=table, row_start=ints(starts, dev), **cache.scales())
    assert (out[T:] == 0).all()
    pos = [ctx[b] + i for b in range(B) for i in range(counts[b])]
    check_rows(out[:T], rotated64(q[:T], qn, table, pos, False, 1e-6), dtype, "q")
    kr, vr = rotated64(k[:T], kn, table, pos, False, 1e-6), v[:T].double()
    for b in range(B) if B < 100 else range(0, B, 37):
        if counts[b]:
            places, rows = range(ctx[b], ctx[b] + counts[b]), slice(starts[b], starts[b + 1])
            check_stored(cache, "k", b, places, kr[rows])
            check_stored(cache, "v", b, places, vr[rows])


def test_append_in_place_queries_and_values_of_any_size(dev):
    """q_out may be q itself; rows of zeros, of tiny and of huge magnitudes and
    with an infinity are stored as the format says."""
    D, Hkv = 128, 2
    cache = Cache([6], Hkv, D, 8, "e4m3", dev, 4)
    gen = torch.Generator(device=dev).manual_seed(1)
    k = torch.randn(1, 6, Hkv, D, generator=gen, device=dev)
    q = torch.randn(1, 6, 4, D, generator=gen, device=dev)
    k[0, 0] = 0.0
    k[0, 1] *= 1e-37
    k[0, 2] *= 1e37
    k[0, 3, 0, 5] = float("inf")
    k[0, 4, 1, 7] = float("nan")
    want = rotated64(q[0], None, angles(10, 64, dev), list(range(6)), False, 1e-6)
    same = sv.spec_kv_append(k, k.clone(), cache.k, cache.v, cache.table, ints([0], dev), q=q,
                             cos_sin=angles(10, 64, dev), q_out=q, **cache.scales())
    assert same.data_ptr() == q.data_ptr()
    check_rows(q[0], want, torch.float32)
    v = cache.rows64("v", 0, range(6))
    assert (v[0] == 0).all()
    # far below the smallest scale's steps: the values flush to within half of the least step
    assert ((v[1] - k[0, 1].double()).abs() <= 2.0 ** -100 * 2.0 ** -10 * 1.01).all()
    assert ((v[2] - k[0, 2].double()).abs() <= k[0, 2].double().abs() * 2.0 ** -4 * 1.001 + 1e37 * 2.0 ** -10).all()
    assert v[3, 0].isnan().all() and v[4, 1].isnan().all()
    check_stored(cache, "v", 0, [5], k[0, 5:].double())


def test_append_unusable_tokens(dev):
    """A bad length, count, tree, page or position: that sequence (or token) is
    not stored, its queries are NaN, bit 2 is set; the others are untouched."""
    B, S, Hq, Hkv, D = 8, 4, 4, 2, 64
    ctx = [10, 20, 5, 8, 3, 12, 0, 9]
    cache = Cache([c + S for c in ctx], Hkv, D, 8, "bf16", dev, 5)
    gen = torch.Generator(device=dev).manual_seed(2)
    q, k, v = (torch.randn(B, S, h, D, generator=gen, device=dev).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    par = [parents_of("binary", S, None) for _ in range(B)]
    kv, new = list(ctx), [S] * B
    table = cache.table.clone()
    kv[0] = -2
    kv[1] = 10 ** 7
    new[2] = S + 1
    new[3] = -1
    par[4][2] = 2
    table[5, 1] = cache.num_pages + 9       # positions 8 ... 15: all four tokens
    cs = angles(11, 64, dev)                # sequence 7: its second level is position 10, its third 11
    before = snapshot(cache)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = sv.spec_kv_append(k, v, cache.k, cache.v, table, ints(kv, dev), n_new=ints(new, dev), q=q, cos_sin=cs,
                            parent=ints(par, dev), errors=err)
    assert err.item() == CACHE_BIT
    assert out[:6].isnan().all()
    assert not out[6].isnan().any()
    assert not out[7, :3].isnan().any() and out[7, 3].isnan().all()
    after = snapshot(cache)
    for b in range(8):
        places = [p for p in range(ctx[b], ctx[b] + S)]
        page, slot = cache.at(b, places)
        same = bits(before[0][page, :, slot]) == bits(after[0][page, :, slot])
        if b < 6:
            assert same.all(), b
    check_stored(cache, "v", 6, range(0, S), v[6].double())
    check_stored(cache, "v", 7, range(9, 12), v[7, :3].double())
    # packed rows whose starts do not ascend
    err.zero_()
    sv.spec_kv_append(k[0], v[0], cache.k, cache.v, cache.table[:2], ints([0, 0], dev),
                      row_start=ints([0, 9, 4], dev), errors=err)
    assert err.item() in (0, CACHE_BIT)


def _commit_case(dev, B, N, layers, Hkv, D, page, fmt, seed, tree="random"):
    rng = random.Random(seed)
    ctx = [rng.choice([0, 1, 7, 30, 65]) for _ in range(B)]
    cache = Cache([c + N for c in ctx], Hkv, D, page, fmt, dev, seed, layers=layers, fill=False)
    path, length = [], []
    for b in range(B):
        par, at, p = parents_of(tree, N, rng), 0, []
        while True:
            kids = [n for n in range(1, N) if par[n] == at]
            if not kids or rng.random() < 0.15:
                break
            at = rng.choice(kids)
            p.append(at)
        if b % 7 == 6:
            path.append([-1] * N)
            length.append(-1)                  # verification met unusable data
        else:
            path.append(p + [-1] * (N - len(p)))
            length.append(len(p))
    return ctx, cache, path, length


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [(1, 2, 1, 1, 64, 8), (9, 15, 3, 8, 128, 16), (40, 32, 2, 2, 80, 8), (5, 31, 1, 3, 256, 64),
                                   (3, 1, 2, 1, 64, 8)])
def test_commit_moves_the_kept_path(dev, shape, fmt, in_place):
    B, N, layers, Hkv, D, page = shape
    ctx, cache, path, length = _commit_case(dev, B, N, layers, Hkv, D, page, fmt, B + N, "chain" if N == 2 else "random")
    before = snapshot(cache)
    kv = ints(ctx, dev)
    out = None if in_place else torch.full((B,), -7, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = sv.spec_kv_commit(cache.k, cache.v, cache.table, kv, ints(path, dev), ints(length, dev), kv_len_out=out, errors=err,
                            **cache.scales())
    assert err.item() == 0
    assert got.data_ptr() == (kv if in_place else out).data_ptr()
    assert got.tolist() == [c + 1 + n if n >= 0 else c for c, n in zip(ctx, length)]
    after = snapshot(cache)
    for x, y in zip(before, after):
        want = x.clone()
        for b in range(B):
            for i in range(max(0, length[b])):
                (sp,), (ss,) = (t.tolist() for t in cache.at(b, [ctx[b] + path[b][i]]))
                (dp,), (ds,) = (t.tolist() for t in cache.at(b, [ctx[b] + 1 + i]))
                bits_w, bits_x = want.view(torch.uint8) if x.dtype == E4M3 else want, x.view(torch.uint8) if x.dtype == E4M3 else x
                bits_w[:, dp, :, ds] = bits_x[:, sp, :, ss]
        assert torch.equal(bits(want), bits(y))


def test_commit_follows_verification(dev):
    """out_path and out_len of spec_verify_tree go in as they are."""
    import numpy as np
    import workloads as W
    B, N, V = 12, 15, 1003
    d = W.make_tree_host(B, W.full_tree(2, 3), V, "f32", 2.0, 0.3, np.full(B, 1.0, np.float32), seed=5)
    put = lambda a, t: torch.from_numpy(np.ascontiguousarray(a, t)).to(dev)  # noqa: E731
    _, path, length = sv.spec_verify_tree(put(d["target"], np.float32), put(d["draft"], np.float32), put(d["tokens"], np.int32),
                                          put(d["parent"], np.int32), put(d["uniforms"], np.float32),
                                          put(d["temperature"], np.float32), put(d["n_nodes"], np.int32))
    ctx = [5 * b for b in range(B)]
    cache = Cache([c + N for c in ctx], 2, 64, 16, "bf16", dev, 6, fill=False)
    before = cache.k.clone()
    kv = ints(ctx, dev)
    sv.spec_kv_commit(cache.k, cache.v, cache.table, kv, path, length)
    path, length = path.tolist(), length.tolist()
    assert max(length) >= 2
    assert kv.tolist() == [c + 1 + n for c, n in zip(ctx, length)]
    for b in range(B):
        sp, ss = cache.at(b, [ctx[b] + n for n in path[b][:length[b]]])
        dp, ds = cache.at(b, [ctx[b] + 1 + i for i in range(length[b])])
        assert torch.equal(cache.k[dp, :, ds], before[sp, :, ss])


def test_commit_unusable_sequences(dev):
    B, N = 7, 6
    ctx = [10] * B
    cache = Cache([c + N for c in ctx], 2, 64, 8, "bf16", dev, 7, fill=False)
    before = snapshot(cache)
    path = [[2, 4, -1, -1, -1, -1] for _ in range(B)]
    length = [2] * B
    kv, table = list(ctx), cache.table.clone()
    path[0] = [4, 2, -1, -1, -1, -1]       # descends
    path[1][1] = N                         # no such node
    length[2] = N
    length[3] = -2
    kv[4] = 10 ** 6
    table[5, 1] = cache.num_pages
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = ints(kv, dev)
    sv.spec_kv_commit(cache.k, cache.v, table, lens, ints(path, dev), ints(length, dev), errors=err)
    assert err.item() == CACHE_BIT
    assert lens.tolist() == kv[:6] + [13]
    used = torch.zeros(cache.num_pages, 8, dtype=torch.bool, device=dev)
    page, slot = cache.at(6, [11, 12])
    used[page, slot] = True
    for x, y in zip(before, snapshot(cache)):
        assert ((x == y).all(-1) | used[:, None, :]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [([1], 1, 64, 8), ([5, 0, 300], 3, 80, 16), ([33] * 50, 2, 256, 64), ([2000], 8, 128, 128)])
def test_read_returns_the_entries(dev, shape, fmt, dtype):
    counts, Hkv, D, page = shape
    B, T = len(counts), sum(counts)
    start = [(13 * b) % 40 for b in range(B)]
    cache = Cache([s + c for s, c in zip(start, counts)], Hkv, D, page, fmt, dev, 8)
    bounds = [sum(counts[:b]) for b in range(B + 1)]
    k, v = sv.spec_kv_read(cache.k, cache.v, cache.table, ints(start, dev), ints(bounds, dev), T + 2, dtype=dtype, **cache.scales())
    assert (k[T:] == 0).all() and (v[T:] == 0).all()
    for b in range(B):
        for got, name in ((k, "k"), (v, "v")):
            if counts[b]:
                ref = cache.rows64(name, b, range(start[b], start[b] + counts[b]))
                # the product is exact in fp64; fp32 rounds it once, bf16 once more
                want = ref.float().to(dtype)
                assert torch.equal(got[bounds[b]:bounds[b + 1]], want)


def test_read_unusable_ranges(dev):
    cache = Cache([40, 40, 40], 2, 64, 8, "e4m3", dev, 9)
    table = cache.table.clone()
    table[1, 2] = -1                       # positions 16 ... 23
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    k, v = sv.spec_kv_read(cache.k, cache.v, table, ints([0, 10, 39], dev), ints([0, 20, 40, 42], dev), 42, errors=err, **cache.scales())
    assert err.item() == CACHE_BIT
    nan = torch.zeros(42, dtype=torch.bool, device=dev)
    nan[26:34] = True                      # sequence 1's positions 16 ... 23
    nan[40:] = True                        # sequence 2's range leaves the table
    assert torch.equal(k.isnan().all(-1).all(-1), nan) and torch.equal(k.isnan().any(-1).any(-1), nan)
    assert torch.equal(v.isnan().all(-1).all(-1), nan)


def test_offsets_past_32_bits(dev):
    """Append, commit and read in the last pages of a cache of more than 2^32
    bytes a tensor."""
    Hkv, D, page = 8, 256, 64
    pages = (1 << 32) // (Hkv * D * page * 2) + 50
    k_cache = torch.zeros((pages, Hkv, page, D), dtype=torch.bfloat16, device=dev)
    v_cache = torch.zeros_like(k_cache)
    table = ints([[pages - 1, 0], [pages - 3, pages - 2]], dev)
    kv = ints([60, 3], dev)
    gen = torch.Generator(device=dev).manual_seed(3)
    k, v = (torch.randn(2, 6, Hkv, D, generator=gen, device=dev).to(torch.bfloat16) for _ in range(2))
    sv.spec_kv_append(k, v, k_cache, v_cache, table, kv)
    assert torch.equal(k_cache[pages - 1, :, 60:64].transpose(0, 1), k[0, :4])
    assert torch.equal(v_cache[0, :, 0:2].transpose(0, 1), v[0, 4:])
    path, length = ints([[2, 5, -1, -1, -1, -1], [3, -1, -1, -1, -1, -1]], dev), ints([2, 1], dev)
    start = kv.clone()
    sv.spec_kv_commit(k_cache, v_cache, table, kv, path, length)
    assert kv.tolist() == [63, 5]
    rk, rv = sv.spec_kv_read(k_cache, v_cache, table, start, ints([0, 3, 5], dev), 5)
    assert torch.equal(rk, torch.cat([k[0, [0, 2, 5]], k[1, [0, 3]]]))
    assert torch.equal(rv, torch.cat([v[0, [0, 2, 5]], v[1, [0, 3]]]))


def test_refusals(dev):
    cache = Cache([20], 2, 64, 8, "bf16", dev, 1)
    k = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device=dev)
    kv = ints([0], dev)
    args = (cache.k, cache.v, cache.table, kv)
    with pytest.raises(TypeError):
        sv.spec_kv_append(k.half(), k.half(), *args)
    with pytest.raises(TypeError):
        sv.spec_kv_append(k, k.float(), *args)
    with pytest.raises(ValueError):
        sv.spec_kv_append(k[..., :32], k[..., :32], *args)
    with pytest.raises(ValueError):
        sv.spec_kv_append(k, k, *args, row_start=ints([0, 4], dev))
    with pytest.raises(ValueError):
        sv.spec_kv_append(k.cpu(), k.cpu(), *args)
    with pytest.raises(sv.SpecVerifyError) as e:     # a rotation wider than the head
        sv.spec_kv_append(k, k, *args, cos_sin=angles(10, 128, dev))
    assert e.value.status == sv.SV_ERR_INVALID_ARG
    with pytest.raises(sv.SpecVerifyError):          # rows off their 16-byte places
        odd = torch.zeros(1 * 4 * 2 * 64 + 1, dtype=torch.bfloat16, device=dev)[1:].view(1, 4, 2, 64)
        sv.spec_kv_append(odd, odd, *args)
    with pytest.raises(sv.SpecVerifyError):          # a tree of more than 32 nodes
        wide = torch.zeros(1, 33, 2, 64, dtype=torch.bfloat16, device=dev)
        sv.spec_kv_append(wide, wide, *args, parent=torch.zeros(1, 33, dtype=torch.int32, device=dev))
    with pytest.raises(sv.SpecVerifyError) as e:     # a page size that is no power of two
        c = torch.zeros(4, 2, 24, 64, dtype=torch.bfloat16, device=dev)
        sv.spec_kv_append(k, k, c, c.clone(), cache.table, kv)
    assert e.value.status == sv.SV_ERR_UNSUPPORTED
    with pytest.raises(sv.SpecVerifyError):          # head_dim 48
        c = torch.zeros(4, 2, 8, 48, dtype=torch.bfloat16, device=dev)
        sv.spec_kv_read(c, c.clone(), cache.table, kv, ints([0, 1], dev), 1)
    with pytest.raises(TypeError):
        sv.spec_kv_read(cache.k, cache.v, cache.table, kv, ints([0, 1], dev), 1, dtype=torch.float16)
    with pytest.raises(ValueError):
        sv.spec_kv_commit(cache.k, cache.v, cache.table, kv, kv, kv)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_kv_commit(cache.k, cache.v, cache.table, kv, torch.zeros(1, 40, dtype=torch.int32, device=dev), kv)
    k0, v0 = sv.spec_kv_read(cache.k, cache.v, cache.table, kv, ints([0, 0], dev), 0)
    assert k0.shape == (0, 2, 64)
