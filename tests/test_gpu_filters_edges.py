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
