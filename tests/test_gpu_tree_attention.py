"""spec_tree_attention against the definition in 64 bits: types, head layouts,
lengths, page sizes, trees, ragged and unusable batches.  Every cache entry
behind a sequence's nodes is NaN, so that using one anywhere shows."""
import random

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from kv_helpers import Cache, attention64, attention_bound, parents_of  # noqa: E402

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


def make(ctx, N, tree, Hq, Hkv, D, fmt, page, dev, seed=1, nodes=None, by=1.0):
    rng = random.Random(seed)
    B = len(ctx)
    nodes = [N] * B if nodes is None else nodes
    cache = Cache([c + n for c, n in zip(ctx, nodes)], Hkv, D, page, fmt, dev, seed)
    gen = torch.Generator(device=dev).manual_seed(seed + 1)
    q = (torch.randn(B, N, Hq, D, generator=gen, device=dev) * by).to(torch.bfloat16)
    parents = [parents_of(tree, N, rng) for _ in range(B)]
    return q, cache, nodes, parents


def call(q, cache, ctx, nodes, parents, dev, **kw):
    tree = kw.pop("tree", "random")
    return sv.spec_tree_attention(q, cache.k, cache.v, cache.table, ints(ctx, dev), ints(nodes, dev),
                                  parent=None if tree == "chain" else ints(parents, dev), **cache.scales(), **kw)


def check(got, q, cache, ctx, nodes, parents, scale=None):
    D = q.shape[-1]
    ref, spread, big = attention64(q, cache, ctx, nodes, parents, D ** -0.5 if scale is None else scale)
    off = (got.double() - ref).abs()
    bound = attention_bound(ref, spread, big, D)
    assert torch.isfinite(got).all()
    worst = (off / bound).max().item()
    print(f"worst error / bound: {worst:.3f}")
    assert worst <= 1.0
    for b, n in enumerate(nodes):
        assert (got[b, n:] == 0).all()


CASES = [  # ctx, N, tree, Hq, Hkv, D, page
    ([0], 1, "chain", 1, 1, 64, 8),
    ([1], 1, "chain", 8, 8, 128, 16),
    ([700], 1, "chain", 32, 8, 128, 16),
    ([0, 1, 5, 127, 128, 129, 255, 256], 7, "binary", 8, 2, 128, 16),
    ([126, 0, 383], 32, "random", 4, 4, 128, 32),
    ([300, 17], 32, "star", 16, 2, 128, 64),      # 256 rows to a key head
    ([640, 64, 1], 9, "chain", 6, 2, 64, 128),
    ([77, 1000], 15, "binary", 20, 4, 80, 8),
    ([500, 129], 31, "random", 5, 1, 96, 16),
    ([40, 260], 3, "star", 24, 2, 112, 256),
    ([10, 511], 5, "random", 6, 3, 144, 16),
    ([200, 513], 13, "random", 12, 2, 192, 64),
    ([1, 140, 1025], 32, "random", 16, 2, 256, 16),
    ([2000], 17, "random", 32, 1, 128, 1024),     # one key head, 544 rows
    ([90, 3000], 2, "chain", 71, 71, 64, 32),     # many heads of one row each
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"ctx{c[0][-1]}n{c[1]}{c[2]}h{c[3]}x{c[4]}d{c[5]}p{c[6]}")
def test_matches_definition(dev, case, fmt):
    ctx, N, tree, Hq, Hkv, D, page = case
    q, cache, nodes, parents = make(ctx, N, tree, Hq, Hkv, D, fmt, page, dev)
    check(call(q, cache, ctx, nodes, parents, dev, tree=tree), q, cache, ctx, nodes, parents)


WIDE = [  # row groups: several nodes, one node, part of a node's heads
    ([250, 3], 5, "random", 100, 2, 64, 16),      # 50 heads a node: two nodes a group
    ([140], 3, "chain", 129, 1, 128, 32),         # 129 heads to one key head: two blocks of heads
    ([70, 600], 2, "star", 200, 1, 64, 8),
    ([33], 4, "random", 70, 1, 256, 16),
    ([500], 32, "binary", 24, 8, 96, 8),          # three query heads a key head
    ([260], 17, "random", 48, 16, 160, 128),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", WIDE, ids=lambda c: f"n{c[1]}h{c[3]}x{c[4]}d{c[5]}")
def test_many_query_heads(dev, case, fmt):
    ctx, N, tree, Hq, Hkv, D, page = case
    q, cache, nodes, parents = make(ctx, N, tree, Hq, Hkv, D, fmt, page, dev, seed=21)
    check(call(q, cache, ctx, nodes, parents, dev, tree=tree), q, cache, ctx, nodes, parents)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_scores_far_from_zero(dev, fmt):
    """All scores of a row near +-several hundred: weights have to follow the
    row's own level."""
    ctx = [900, 130]
    q, cache, nodes, parents = make(ctx, 5, "random", 4, 2, 64, fmt, 16, dev, seed=22)
    q[:] = 4.0
    q[:, :, 1::2] = -4.0
    shift = torch.full((64,), 20.0, device=dev)
    for b in range(2):
        page, slot = cache.at(b, range(ctx[b] + 5))
        if fmt == "bf16":
            cache.k[page, :, slot] = (cache.k[page, :, slot].float() * 0.1 + shift).to(torch.bfloat16)
        else:
            cache.k.view(torch.uint8)[page, :, slot] = 0x38   # 1.0
            cache.k_scale[page, :, slot] = 20.0 + 0.01 * torch.arange(ctx[b] + 5, device=dev)[:, None]
    check(call(q, cache, ctx, nodes, parents, dev), q, cache, ctx, nodes, parents)


SPREAD = [([700, 0], 3, 8, 2, 64), ([9000], 32, 32, 8, 128), ([130, 1], 7, 20, 4, 80), ([1000], 5, 16, 2, 192), ([257], 1, 70, 1, 256)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", SPREAD, ids=lambda c: f"n{c[1]}h{c[2]}x{c[3]}d{c[4]}")
def test_rows_of_different_magnitudes(dev, case, fmt):
    """A row keeps its precision beside rows that are up to 2^46 larger, and
    beside rows of zeros."""
    ctx, N, Hq, Hkv, D = case
    q, cache, nodes, parents = make(ctx, N, "random", Hq, Hkv, D, fmt, 16, dev, seed=24)
    gen = torch.Generator(device=dev).manual_seed(25)
    e = torch.randint(-40, 7, q.shape[:3], generator=gen, device=dev)
    q = (q.float() * torch.exp2(e.float())[..., None] * (e % 5 != 0)[..., None]).to(torch.bfloat16)
    check(call(q, cache, ctx, nodes, parents, dev), q, cache, ctx, nodes, parents)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", SPREAD, ids=lambda c: f"n{c[1]}h{c[2]}x{c[3]}d{c[4]}")
def test_ordinary_rows_beside_huge_ones(dev, case, fmt):
    ctx, N, Hq, Hkv, D = case
    q, cache, nodes, parents = make(ctx, N, "random", Hq, Hkv, D, fmt, 16, dev, seed=26)
    gen = torch.Generator(device=dev).manual_seed(27)
    e = torch.tensor([-3, 0, 2, 30, 60], device=dev)[torch.randint(0, 5, q.shape[:3], generator=gen, device=dev)]
    q = (q.float() * torch.exp2(e.float())[..., None]).to(torch.bfloat16)
    check(call(q, cache, ctx, nodes, parents, dev), q, cache, ctx, nodes, parents)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx", [[0], [300], [40000]])
def test_a_row_of_infinite_scores_is_nan(dev, ctx, fmt):
    """All scores -inf: the softmax of that is NaN, whether one block has the
    row or several do; the other rows are as without it."""
    q, cache, nodes, parents = make(ctx, 3, "star", 4, 2, 64, fmt, 16, dev, seed=23)
    page, slot = cache.at(0, range(ctx[0] + 3))
    if fmt == "bf16":
        cache.k[page, :, slot, 0] = -1.0
    else:
        cache.k.view(torch.uint8)[page, :, slot, 0] = 0xb8   # -1.0
    q[0, 1, 2, 0] = float("inf")
    got = call(q, cache, ctx, nodes, parents, dev)
    assert torch.isnan(got[0, 1, 2]).all()
    q[0, 1, 2, 0] = 0.0
    want = call(q, cache, ctx, nodes, parents, dev)
    want[0, 1, 2] = got[0, 1, 2] = 0.0
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_every_length_around_a_tile(dev, fmt):
    """Lengths 0 ... 159 of one batch: the context ends at every slot of a page
    and of a 128-position tile, and the tree straddles tiles."""
    ctx = list(range(160))
    q, cache, nodes, parents = make(ctx, 12, "random", 4, 2, 64, fmt, 16, dev, seed=5)
    check(call(q, cache, ctx, nodes, parents, dev), q, cache, ctx, nodes, parents)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_ragged_batch_with_idle_sequences(dev, fmt):
    rng = random.Random(9)
    B, N = 300, 15
    ctx = [rng.choice([0, 3, 50, 128, 400, 900]) for _ in range(B)]
    nodes = [rng.choice([0, 1, 2, 7, 14, 15]) for _ in range(B)]
    q, cache, nodes, parents = make(ctx, N, "random", 8, 2, 128, fmt, 32, dev, seed=9, nodes=nodes)
    check(call(q, cache, ctx, nodes, parents, dev), q, cache, ctx, nodes, parents)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_long_context_and_sharp_weights(dev, fmt):
    """70001 positions split over the whole GPU, scores of several tens: the
    running maximum moves in every part, and the parts' maxima differ widely."""
    ctx = [70001, 3]
    q, cache, nodes, parents = make(ctx, 21, "random", 8, 2, 128, fmt, 16, dev, seed=3, by=12.0)
    check(call(q, cache, ctx, nodes, parents, dev), q, cache, ctx, nodes, parents)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_ascending_scores(dev, fmt):
    """Keys that grow with their position: every tile raises the maximum."""
    ctx = [3000]
    q, cache, nodes, parents = make(ctx, 6, "binary", 4, 1, 128, fmt, 16, dev, seed=4)
    q[:] = 1.0
    ramp = torch.arange(3008, device=dev, dtype=torch.float32)
    page, slot = cache.at(0, range(3006))
    if fmt == "bf16":
        cache.k[page, :, slot] = (ramp[:3006, None, None] / 100).expand(-1, 1, 128).to(torch.bfloat16)
    else:
        cache.k.view(torch.uint8)[page, :, slot] = 0x38   # 1.0
        cache.k_scale[page, :, slot] = (ramp[:3006, None] / 100)
    check(call(q, cache, ctx, nodes, parents, dev), q, cache, ctx, nodes, parents)


@pytest.mark.parametrize("scale", [1.0, 0.001, -0.3, 0.0])
def test_scale(dev, scale):
    ctx = [130, 20]
    q, cache, nodes, parents = make(ctx, 4, "random", 4, 2, 64, "bf16", 8, dev, seed=6)
    check(call(q, cache, ctx, nodes, parents, dev, scale=scale), q, cache, ctx, nodes, parents, scale)


def test_strided_queries_other_stream_and_repeatability(dev):
    """Queries as slices of a fused projection, on a stream of the caller's;
    the same call gives the same bits, whatever ran before in its workspace."""
    ctx, N = [900, 0, 333], 10
    q, cache, nodes, parents = make(ctx, N, "random", 8, 2, 128, "bf16", 16, dev, seed=7)
    wide = torch.full((3, N, 12, 128), float("nan"), device=dev, dtype=torch.bfloat16)
    wide[:, :, 2:10] = q
    ws = torch.full((sv.sv_attention_workspace_size(N, 8, 2, 128),), 255, dtype=torch.uint8, device=dev)
    ref = call(q, cache, ctx, nodes, parents, dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [call(wide[:, :, 2:10], cache, ctx, nodes, parents, dev, workspace=ws) for _ in range(3)]
    direct = call(wide[:, :, 2:10], cache, ctx, nodes, parents, dev, stream=s)
    s.synchronize()
    for g in got + [direct]:
        assert torch.equal(g, ref)
    check(ref, q, cache, ctx, nodes, parents)


def test_graph_replay_with_new_lengths(dev):
    """A captured call follows the device's lengths and trees at each replay."""
    N = 8
    ctx = [1000, 40]
    q, cache, nodes, parents = make(ctx, N, "random", 8, 2, 128, "e4m3", 16, dev, seed=8)
    kv, nn, par = ints(ctx, dev), ints(nodes, dev), ints(parents, dev)
    run = lambda: sv.spec_tree_attention(q, cache.k, cache.v, cache.table, kv, nn, parent=par, **cache.scales())  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for ctx2 in (ctx, [1, 39], [777, 0]):
        kv.copy_(ints(ctx2, dev))
        g.replay()
        torch.cuda.synchronize()
        check(out.clone(), q, cache, ctx2, nodes, parents)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_infinite_and_nan_entries_reach_only_their_rows(dev, fmt):
    """A NaN key of one node is seen by its descendants alone; a NaN in a
    sequence's context makes that key head's rows NaN and no other's."""
    ctx, N = [200, 200], 7
    q, cache, nodes, parents = make(ctx, N, "binary", 4, 2, 64, fmt, 16, dev, seed=11)
    ref = call(q, cache, ctx, nodes, parents, dev)
    page, slot = cache.at(0, [200 + 4])           # node 4: a leaf, seen by itself alone
    bad = lambda t: t.view(torch.uint8) if fmt == "e4m3" else t  # noqa: E731
    bad(cache.k)[page, 0, slot] = 0x7f if fmt == "e4m3" else float("nan")
    page, slot = cache.at(1, [57])
    bad(cache.v)[page, 1, slot] = 0x7f if fmt == "e4m3" else float("nan")
    got = call(q, cache, ctx, nodes, parents, dev)
    hit = torch.zeros(got.shape, dtype=torch.bool, device=dev)
    hit[0, 4, :2] = True
    hit[1, :, 2:] = True
    assert got[hit].isnan().all()
    assert torch.equal(got[~hit], ref[~hit])


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e4m3_scale"])
def test_values_of_a_node_reach_only_its_descendants(dev, fmt, what):
    """A node's values that are not finite make the rows that see it NaN; the
    other rows of the tree keep every bit."""
    ctx, N = [250, 31], 7          # the first tree straddles two tiles
    q, cache, nodes, parents = make(ctx, N, "binary", 4, 2, 128, fmt[:4], 16, dev, seed=14)
    ref = call(q, cache, ctx, nodes, parents, dev)
    for b, node in ((0, 1), (0, 6), (1, 5)):
        page, slot = cache.at(b, [ctx[b] + node])
        if fmt == "bf16":
            cache.v[page, 0, slot, 77] = what
        elif fmt == "e4m3":
            cache.v.view(torch.uint8)[page, 0, slot, 77] = 0xff
        else:
            cache.v_scale[page, 0, slot] = what
    got = call(q, cache, ctx, nodes, parents, dev)
    hit = torch.zeros(got.shape, dtype=torch.bool, device=dev)
    for b, n in ((0, 1), (0, 3), (0, 4), (0, 6), (1, 5)):
        hit[b, n, :2] = True
    assert got[hit].isnan().all()
    assert torch.equal(got[~hit], ref[~hit])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_unusable_sequences_are_reported_and_isolated(dev, fmt):
    ctx, N = [150, 300, 90, 40, 260, 33, 20], 6
    q, cache, nodes, parents = make(ctx, N, "random", 8, 2, 128, fmt, 16, dev, seed=12)
    ref = call(q, cache, ctx, nodes, parents, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    clean = call(q, cache, ctx, nodes, parents, dev, errors=err)
    assert torch.equal(clean, ref) and err.item() == 0
    table = cache.table.clone()
    bad_ctx, bad_nodes, bad_par = list(ctx), list(nodes), [list(p) for p in parents]
    table[0, 3] = cache.num_pages        # a page that does not exist
    table[1, 0] = -5
    bad_ctx[2] = -1
    bad_ctx[3] = 10 ** 6                 # past the table's width
    bad_nodes[4] = N + 1
    bad_par[5][3] = 3                    # its own parent
    got = sv.spec_tree_attention(q, cache.k, cache.v, table, ints(bad_ctx, dev), ints(bad_nodes, dev),
                                 parent=ints(bad_par, dev), errors=err, **cache.scales())
    assert err.item() == CACHE_BIT
    assert got[:6].isnan().all()
    assert torch.equal(got[6], ref[6])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_offsets_past_32_bits(dev, fmt):
    """A cache of more than 2^32 bytes a tensor, its last pages used."""
    Hkv, D, page = 8, 256, 64
    elem = 2 if fmt == "bf16" else 1
    pages = (1 << 32) // (Hkv * D * page * elem) + 600
    ctx, N = [1500, 200], 5
    small = Cache([c + N for c in ctx], Hkv, D, page, fmt, dev, 13)
    q, _, nodes, parents = make(ctx, N, "random", 8, Hkv, D, fmt, page, dev, seed=13)
    shift = pages - small.num_pages
    big = [torch.empty((pages, Hkv, page, D), dtype=small.k.dtype, device=dev) for _ in range(2)]
    big[0][shift:], big[1][shift:] = small.k, small.v
    scales = {}
    if fmt == "e4m3":
        for n, t in small.scales().items():
            scales[n] = torch.full((pages, Hkv, page), float("nan"), device=dev)
            scales[n][shift:] = t
    table = torch.where(small.table >= 0, small.table + shift, -1)
    got = sv.spec_tree_attention(q, big[0], big[1], table, ints(ctx, dev), ints(nodes, dev),
                                 parent=ints(parents, dev), **scales)
    check(got, q, small, ctx, nodes, parents)


def test_refusals(dev):
    q, cache, nodes, parents = make([30], 4, "chain", 4, 2, 64, "bf16", 8, dev)
    kv = ints([30], dev)
    args = (cache.k, cache.v, cache.table, kv)
    with pytest.raises(sv.SpecVerifyError):   # 4 heads over 3
        sv.spec_tree_attention(q[:, :, :3].contiguous(), *args)
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_tree_attention(q.float(), *args)
    assert e.value.status == sv.SV_ERR_UNSUPPORTED
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_tree_attention(q, *args, workspace=torch.empty(0, dtype=torch.uint8, device=dev))
    assert e.value.status == sv.SV_ERR_NO_MEMORY
    with pytest.raises(ValueError):
        sv.spec_tree_attention(q.transpose(2, 3), *args)
    with pytest.raises(TypeError):
        sv.spec_tree_attention(q, cache.k, cache.v, cache.table.long(), kv)
    with pytest.raises(ValueError):
        sv.spec_tree_attention(q, cache.k, cache.v, cache.table, kv, k_scale=kv, v_scale=kv)
    with pytest.raises(sv.SpecVerifyError):   # broadcast queries
        two = Cache([9, 9], 2, 64, 8, "bf16", dev)
        sv.spec_tree_attention(q[:, :1].expand(2, 1, 4, 64).as_strided((2, 1, 4, 64), (0, 256, 64, 1)), two.k, two.v, two.table, ints([3, 3], dev))
    with pytest.raises(sv.SpecVerifyError):   # more nodes than a tree may have
        sv.spec_tree_attention(torch.zeros(1, 33, 4, 64, device=dev, dtype=torch.bfloat16), *args)
    assert sv.spec_tree_attention(q[:0], cache.k, cache.v, cache.table[:0], kv[:0]).shape == (0, 4, 4, 64)
