"""The cache operators at the longest lengths that they take."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from kv_helpers import E4M3  # noqa: E402

pytestmark = pytest.mark.gpu
LIMIT = (1 << 31) - (1 << 16)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


@pytest.mark.parametrize("page", [64, 1024])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_sequence_as_long_as_positions_go(dev, fmt, page):
    """A context of 2^31 - 2^16 - 40 positions whose table repeats one page; the
    last full page holds a key that outweighs all the rest together, so that
    the rows are its value; the nodes behind it are appended, moved and read."""
    D, N, pages = 64, 3, LIMIT // page
    ctx = LIMIT - 40
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    gen = torch.Generator(device=dev).manual_seed(41)
    rand = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    k, v = (0.1 * rand(4, 1, page, D) for _ in range(2))
    k[..., 0] = 0.0
    heavy, at = page - 7, 2          # position of the last full page, physical page 2
    k[at, 0, heavy, 0] = 40.0
    v[at, 0, heavy] = torch.arange(D, device=dev) / 64.0 + 0.5
    scales = {}
    if fmt == "e4m3":
        for n, x in (("k_scale", k), ("v_scale", v)):
            scales[n] = (x.abs().amax(-1) / 448.0).contiguous()
        k, v = (x / s[..., None] for x, s in ((k, scales["k_scale"]), (v, scales["v_scale"])))
    k, v = (x.to(torch.bfloat16 if fmt == "bf16" else E4M3).contiguous() for x in (k, v))
    want = v[at, 0, heavy].float() * (scales["v_scale"][at, 0, heavy] if scales else 1.0)
    table = torch.zeros(1, pages, dtype=torch.int32, device=dev)
    table[0, -2], table[0, -1] = at, 3
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kv = ints([ctx])
    new_k, new_v = (0.1 * rand(1, N, 1, D) for _ in range(2))
    new_k[..., 0] = 0.0
    sv.spec_kv_append(new_k, new_v, k, v, table, kv, errors=err, **scales)
    q = torch.zeros(1, N, 2, D, device=dev, dtype=torch.bfloat16)
    q[..., 0] = 8.0
    # the key's score is 40 (all others are 0): e^40 = 2^57.7 against 2^31 positions, less than 2^-26 of it
    out = sv.spec_tree_attention(q, k, v, table, kv, errors=err, **scales)
    # one rounding of the weight (bf16 or fp16), one of the result, and the sums' (8 k-steps of 2^17 / 2^3 tiles a block in fp32)
    assert ((out.float() - want).abs() <= 2.0 ** -7 * want.abs()).all()
    start = kv.clone()
    rows = sv.spec_kv_read(k, v, table, start, ints([0, N]), N, dtype=torch.float32, errors=err, **scales)
    sv.spec_kv_commit(k, v, table, kv, ints([[2, -1, -1]]), ints([1]), errors=err, **scales)
    assert kv.tolist() == [ctx + 2]
    moved = sv.spec_kv_read(k, v, table, start, ints([0, 2]), 2, dtype=torch.float32, errors=err, **scales)
    for a, b, x in zip(rows, moved, (new_k, new_v)):
        assert (a - x[0]).abs().max() <= 2.0 ** -4 * x.abs().max()
        assert torch.equal(b, a[[0, 2]])
    assert err.item() == 0
