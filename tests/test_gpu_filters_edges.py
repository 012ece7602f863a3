"""Rows at the edges of what the filters take, against the definitions in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from test_gpu_filters import DT, check_draw, check_filter, dev, rows, settings  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,B", [(9, 12), (1024, 12), (3001, 12), (128256, 12)])
def test_greedy_rows_use_no_filter(dev, V, B, dtype):  # noqa: F811
    """T = 0 is the argmax whatever the filters and the uniforms hold; an unusable row is one all the same, and a
    neighbour with T > 0 and such a filter too."""
    logits, u = rows(B, V, dtype, dev, V + 80)
    nan, inf = math.nan, math.inf
    T = [0.0] * B
    T[B - 1] = T[B - 2] = 0.8
    k = [-1, 0, 0, -2 ** 31, 3, 2 ** 31 - 1, 0, 0, 0, 0, -1, 5]
    p = [1.0, nan, 0.9, 0.9, -1.0, 2.0, inf, 1.0, 0.9, 0.5, 0.9, 0.9]
    m = [0.0, 0.0, nan, 0.1, 1.5, -0.5, -inf, inf, 0.0, 0.0, 0.0, 0.0]
    u[:] = torch.tensor([nan, 1.0, -1.0, inf, 0.5, 0.5, nan, 2.0, 0.1, 0.1, 0.5, 0.5])
    logits[8, V // 2] = nan
    logits[9, V // 3] = inf
    s = settings(dev, T, k, p, m)
    tok, prob, kept = sv.spec_sample_filtered(logits, u, **s)
    out, kept2 = sv.spec_filter_logits(logits, **s)
    top = logits[:8] == logits[:8].amax(-1, keepdim=True)
    first = torch.where(top, torch.arange(V, device=dev), V).amin(-1)   # the lowest of equal ones
    assert torch.equal(tok[:8].long(), first) and (prob[:8] == 1).all() and (kept[:8] == 1).all() and torch.equal(kept2, kept)
    assert torch.equal(out[:8].isinf().sum(-1), torch.full((8,), V - 1, device=dev))
    assert torch.equal(out.gather(1, tok.clamp(min=0).long()[:, None])[:8, 0], logits[:8].amax(-1))
    assert (tok[8:11] == -1).all() and prob[8:11].isnan().all() and (kept[8:11] == -1).all() and out[8:11].isnan().all()
    one = settings(dev, T[11:], k[11:], p[11:], m[11:])
    check_draw(logits[11:], u[11:], one, (tok[11:], prob[11:], kept[11:]))
    check_filter(logits[11:], one, (out[11:], kept2[11:]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("near", [0.0, -0.0, 3e-8, -5.9604644775390625e-08, 1e-12])
@pytest.mark.parametrize("n", [1, 5, 16, 40, 3000])
@pytest.mark.parametrize("reach", [14.0, 45.0])
def test_logits_at_zero(dev, reach, n, near, dtype):  # noqa: F811
    """Logits nearer to zero than 2^-24 at low temperatures, where 2^-24 is a thousandth of a percent of a weight: shares
    within the rounding of one quotient, draws and kept sets as they are defined."""
    V, B = 9001, 60
    rng = np.random.default_rng(n)
    T = rng.choice([0.006, 0.0072, 0.01, 0.03, 0.8], B)
    top = (T * rng.uniform(0.0, reach, B)).astype(np.float32)
    x = torch.full((B, V), -2.0, device=dev) - torch.rand(B, V, generator=torch.Generator(device=dev).manual_seed(n), device=dev)
    for b in range(B):
        at = rng.permutation(V)
        x[b, torch.from_numpy(at[:n]).to(dev)] = near
        x[b, at[n]] = float(top[b])
        x[b, at[n + 1]] = float(top[b]) * 0.75
    x = x.to(DT[dtype])
    u = torch.from_numpy(rng.uniform(0, 1, B).astype(np.float32)).to(dev)
    for k, p in ((None, None), (None, rng.uniform(0.3, 0.9999, B)), ([n // 2 + 400] * B, None)):
        s = settings(dev, T, k, p)
        check_draw(x, u, s)
        check_filter(x, s)


NAN_BITS = {"bf16": (torch.int16, [0x7fc1, 0xffc1 - 0x10000, 0x7f81, 0xff81 - 0x10000, 0x7fff, -1]),
            "f32": (torch.int32, [0x7fc00001, 0xffc00001 - 2 ** 32, 0x7f800001, 0xff800001 - 2 ** 32, 0x7fffffff, -1])}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [7, 1000, 2049, 30011, 128256])
@pytest.mark.parametrize("one", [dict(), dict(p=0.9), dict(k=700), dict(k=20), dict(m=0.1), dict(k=3, p=0.5), dict(greedy=True)], ids=str)
def test_every_nan_makes_a_row_unusable(dev, one, V, dtype):  # noqa: F811
    """Both signs, quiet and signalling, at the row's ends and inside; the rows between are as without it."""
    view, bits = NAN_BITS[dtype]
    at = [0, V - 1, V // 2]
    B = 2 * len(bits) * len(at)
    if B * V > 2000000:                      # a few rows, each over several CTAs
        at, B = [V // 3], 2 * len(bits)
    logits, u = rows(B, V, dtype, dev, V + 3)
    raw = logits.view(view)
    for i, b in enumerate(bits):
        for j, a in enumerate(at):
            raw[2 * (i * len(at) + j), a] = b
    assert logits[::2].isnan().any(-1).all()
    s = settings(dev, [0.0 if "greedy" in one else 0.8] * B, *([one[n]] * B if n in one else None for n in "kpm"))
    tok, prob, kept = sv.spec_sample_filtered(logits, u, **s)
    out, n = sv.spec_filter_logits(logits, **s)
    assert (tok[::2] == -1).all() and prob[::2].isnan().all() and (kept[::2] == -1).all() and (n[::2] == -1).all() and out[::2].isnan().all()
    few = slice(1, 8, 2)
    half = {k: None if t is None else t[few].contiguous() for k, t in s.items()}
    check_draw(logits[few], u[few], half, (tok[few], prob[few], kept[few]))
    check_filter(logits[few], half, (out[few], n[few]))
    assert (kept[1::2] > 0).all() and (n[1::2] == kept[1::2]).all()
