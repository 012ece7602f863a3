"""spec_tree_attention in two calls at once, and inside the decoding example."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from kv_helpers import E4M3, Cache, attention64, attention_bound  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def test_two_calls_at_once(dev):
    """Calls that overlap on two streams, each with its workspace and error word."""
    made = []
    for seed, fmt, ctx in ((61, "bf16", [5000, 31, 1200]), (62, "e4m3", [9000, 2, 700])):
        N = 9
        cache = Cache([c + N for c in ctx], 4, 128, 16, fmt, dev, seed)
        q = torch.randn(3, N, 16, 128, generator=torch.Generator(device=dev).manual_seed(seed), device=dev).to(torch.bfloat16)
        ws = torch.empty(sv.sv_attention_workspace_size(N, 16, 4, 128), dtype=torch.uint8, device=dev)
        out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device=dev)
        args = (q, cache.k, cache.v, cache.table, ints(ctx, dev))
        ref = sv.spec_tree_attention(*args, **cache.scales())
        made.append((args, dict(cache.scales(), workspace=ws, out=out, errors=err, stream=torch.cuda.Stream()), ref))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, kw, _ in made:
            kw["out"].fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(3):
            for args, kw, _ in made:
                sv.spec_tree_attention(*args, **kw)
        torch.cuda.synchronize()
        for _, kw, ref in made:
            assert torch.equal(kw["out"], ref) and kw["errors"].item() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_of_the_decoding_example(dev, fmt, monkeypatch):
    """Every call that the example makes, against the definition."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")
    spec = importlib.util.spec_from_file_location("tree_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    real, count = sv.spec_tree_attention, []

    def checked(q, k, v, table, kv_len, parent=None, **kw):
        out = real(q, k, v, table, kv_len, parent=parent, **kw)
        c = Cache.__new__(Cache)
        c.k, c.v, c.k_scale, c.v_scale, c.page, c.Hkv = k, v, kw.get("k_scale"), kw.get("v_scale"), k.shape[-2], k.shape[-3]
        c.pages = table.tolist()
        ref, spread, big = attention64(q, c, kv_len.tolist(), [q.shape[1]] * q.shape[0], parent.tolist(), q.shape[-1] ** -0.5)
        assert ((out.double() - ref).abs() <= attention_bound(ref, spread, big, q.shape[-1])).all()
        count.append(k.dtype)
        return out

    monkeypatch.setattr(sv, "spec_tree_attention", checked, raising=False)
    example.run(rounds=4, B=3, fmt=fmt, seed=5)
    assert count == [torch.bfloat16 if fmt == "bf16" else E4M3] * 4
