"""Waits inside the attention kernel that give up: the call returns, its rows
are their values or NaN, and the next call is as if nothing had been.

A kind of wait is made to run out by the test-only argument expire_waits (the
barriers of that kind lack one arrival, and the limit is some milliseconds).
The copies and products under way are legitimate, land, and are waited for with
the normal bound before a block ends.  Nothing here traps, faults or hangs the GPU."""
import random

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from kv_helpers import Cache, parents_of  # noqa: E402

pytestmark = pytest.mark.gpu
KINDS = ["queries", "queries' place", "keys", "keys' slot", "values", "values' slot", "converted", "converted slot", "rows", "rows' place",
         "scores", "scores' place", "weights", "sums"]
CONVERTED = (6, 7)   # e4m3 caches only
SHAPES = [  # ctx, nodes, Hq, Hkv, D, page: whole items of one tile and of several, empty sequences; items cut between blocks
    ([5, 300, 0, 129, 700], [7, 7, 0, 3, 7], 8, 2, 128, 16),
    ([30000, 3], [7, 7], 32, 2, 64, 16),
    ([140, 2000], [6, 7], 12, 2, 256, 64),
    ([1], [1], 2, 1, 128, 8),
]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def make(dev, fmt, shape):
    ctx, nodes, Hq, Hkv, D, page = shape
    N, rng = max(nodes), random.Random(31)
    cache = Cache([c + n for c, n in zip(ctx, nodes)], Hkv, D, page, fmt, dev, 31)
    q = torch.randn(len(ctx), N, Hq, D, generator=torch.Generator(device=dev).manual_seed(32), device=dev).to(torch.bfloat16)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    parent, kv, n = ints([parents_of("random", N, rng) for _ in ctx]), ints(ctx), ints(nodes)
    ws = torch.zeros(sv.sv_attention_workspace_size(N, Hq, Hkv, D), dtype=torch.uint8, device=dev)
    return lambda **kw: sv.spec_tree_attention(q, cache.k, cache.v, cache.table, kv, n, parent=parent, workspace=ws, **cache.scales(), **kw)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", range(sv.SV_ATTENTION_WAITS), ids=lambda k: KINDS[k].replace(" ", "_"))
def test_the_next_call_is_unaffected(dev, kind, fmt):
    for shape in SHAPES:
        call = make(dev, fmt, shape)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        ref = call(errors=err)
        got = call(expire_waits=1 << kind)
        if fmt == "bf16" and kind in CONVERTED:
            assert torch.equal(got, ref)          # it has no such waits
        for _ in range(2):
            assert torch.equal(call(errors=err), ref)
        assert err.item() == 0


def test_all_waits_at_once(dev):
    for fmt in ("bf16", "e4m3"):
        for shape in SHAPES:
            call = make(dev, fmt, shape)
            ref = call()
            call(expire_waits=(1 << sv.SV_ATTENTION_WAITS) - 1)
            assert torch.equal(call(), ref)


MORE = [  # several items to a block; items of many tiles
    ([200] * 300, [3] * 300, 4, 2, 64, 16),
    ([3000] * 24, [9] * 24, 16, 8, 64, 64),
]
PLACES = (1, 3, 5, 7, 9, 11)   # waits for something to be free again: the first passes


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", range(sv.SV_ATTENTION_WAITS), ids=lambda k: KINDS[k].replace(" ", "_"))
def test_rows_are_right_or_nan_and_reported(dev, kind, fmt):
    """No row is anything but its value or NaN, and bit 0 says whether one is
    NaN.  Where a kind's first wait is needed for any result, all are."""
    some = False
    for shape in SHAPES + MORE:
        ctx, nodes, Hq, Hkv, D, page = shape
        call = make(dev, fmt, shape)
        ref = call()
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        # NaN where nothing is written would pass for a lost row: start from something else
        out = torch.full_like(ref, 7.0)
        got = call(expire_waits=1 << kind, errors=err, out=out)
        lost = got.isnan().all(-1)
        assert (lost | (got == ref).all(-1)).all()
        real = torch.arange(ref.shape[1], device=dev) < torch.tensor(nodes, device=dev)[:, None]
        assert not (lost & ~real[..., None]).any()
        assert err.item() == (1 if lost.any() else 0)
        some |= bool(lost.any())
        if kind not in PLACES and not (fmt == "bf16" and kind in CONVERTED):
            assert lost[real].all()
    assert some == (fmt == "e4m3" or kind not in CONVERTED)
