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
