"""Filtered sampling and filtered logits against the definitions in 64 bits.

Tokens, kept counts and kept sets have to be equal.  A token's share is a
quotient of sums that are good to 2^-29 and is rounded to fp32 once: within
2^-24 + 2^-28 of itself.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from filter_helpers import draw_of, filtered  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SHARE = 2.0 ** -24 + 2.0 ** -28


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def settings(dev, T, k=None, p=None, m=None):
    put = lambda x, t: None if x is None else torch.tensor(x, dtype=t, device=dev)  # noqa: E731
    return dict(temperature=put(T, torch.float32), top_k=put(k, torch.int32), top_p=put(p, torch.float32), min_p=put(m, torch.float32))


def host(logits, s):
    x = logits.double().cpu().numpy()
    B = x.shape[0]
    get = lambda n, d: [d] * B if s[n] is None else s[n].cpu().tolist()  # noqa: E731
    return x, get("temperature", 1.0), get("top_k", 0), get("top_p", 1.0), get("min_p", 0.0)


def check_draw(logits, u, s, got=None):
    tok, prob, kept = (t.cpu().tolist() for t in (got or sv.spec_sample_filtered(logits, u, **s)))
    x, T, k, p, m = host(logits, s)
    for b in range(len(x)):
        want = draw_of(x[b], u[b].item(), T[b], k[b], p[b], m[b])
        assert (tok[b], kept[b]) == (want[0], want[2]), (b, T[b], k[b], p[b], m[b], (tok[b], prob[b], kept[b]), want)
        assert (np.isnan(prob[b]) and want[0] == -1) or abs(prob[b] - want[1]) <= SHARE * want[1], (b, prob[b], want)


def check_filter(logits, s, got=None):
    out, kept = got or sv.spec_filter_logits(logits, **s)
    flat = logits if logits.dim() == 3 else logits[:, None]
    out, kept = out.reshape(flat.shape).double().cpu().numpy(), kept.reshape(flat.shape[:2]).cpu().tolist()
    x, T, k, p, m = host(flat, s)
    for b in range(len(x)):
        for i in range(x.shape[1]):
            want, n = filtered(x[b, i], T[b], k[b], p[b], m[b])
            assert kept[b][i] == n, (b, i, T[b], k[b], p[b], m[b], kept[b][i], n)
            assert np.array_equal(out[b, i], want, equal_nan=True), (b, i, T[b], k[b], p[b], m[b])


def rows(B, V, dtype, dev, seed, sigma=2.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(B, V, generator=g, device=dev) * sigma
    if V > 40:   # a few that stand out
        x[:, ::V // 7] += torch.rand(B, 1, generator=g, device=dev) * 8
    return x.to(DT[dtype]), torch.rand(B, generator=g, device=dev)


MIXED = dict(T=[1.0, 0.7, 0.0, 1.3, 0.9, 0.6, 1.0, 0.8, 2.5, 1.0], k=[0, 50, 3, 0, 1, 7, 0, 1000, 0, 200], p=[0.9, 0.95, 0.5, 1.0, 1.0, 0.8, 1.0, 0.999, 0.7, 0.9],
             m=[0.0, 0.0, 0.0, 0.05, 0.0, 0.01, 0.0, 0.0, 0.001, 0.1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 15, 31, 33, 100, 511, 1000, 1024, 1025, 4099, 8191, 32000, 50257])
def test_settings_of_their_own(dev, V, dtype):
    logits, u = rows(10, V, dtype, dev, V)
    s = settings(dev, **MIXED)
    check_draw(logits, u, s)
    check_filter(logits, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 100, 129, 300, 511, 513, 1000, 1024, 1025, 2048])
def test_many_short_rows(dev, V, dtype):
    """More of them than fill the device, around the sizes where rows change their blocks and their sort."""
    logits, u = rows(530, V, dtype, dev, V)
    logits[7, V // 2] = float("nan")
    logits[8] = -float("inf")
    s = settings(dev, **{n: v * 53 for n, v in MIXED.items()})
    check_draw(logits, u, s)
    check_filter(logits, s)
    out = logits.reshape(53, 10, V).clone()
    few = {n: t[:53].contiguous() for n, t in s.items()}
    check_filter(logits.reshape(53, 10, V), few, sv.spec_filter_logits(out, out=out, **few))


@pytest.mark.parametrize("dtype,V,B", [("bf16", 128256, 10), ("f32", 151936, 10), ("bf16", 200003, 10)])
def test_large_vocabularies(dev, dtype, V, B):
    logits, u = rows(B, V, dtype, dev, V)
    s = settings(dev, **MIXED)
    check_draw(logits, u, s)
    check_filter(logits, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_vocabulary(dev, dtype):
    V = sv.sv_max_vocab(sv.SV_DTYPE_BF16 if dtype == "bf16" else sv.SV_DTYPE_F32)
    logits, u = rows(3, V, dtype, dev, 5)
    s = settings(dev, [1.0, 0.7, 1.1], [0, 40, 0], [0.9, 1.0, 1.0], [0.0, 0.0, 0.02])
    check_draw(logits, u, s)
    check_filter(logits, s)


@pytest.mark.parametrize("which", ["none", "k", "p", "min"])
@pytest.mark.parametrize("B", [1, 2, 5, 40, 160, 400])
def test_batches(dev, B, which):
    logits, u = rows(B, 5003, "bf16" if B % 2 else "f32", dev, B)
    rng = np.random.default_rng(B)
    s = settings(dev, rng.uniform(0.4, 1.5, B), k=rng.integers(1, 600, B) if which == "k" else None, p=rng.uniform(0.1, 0.999, B) if which in ("k", "p") else None,
                 m=rng.uniform(0.0005, 0.5, B) if which == "min" else None)
    check_draw(logits, u, s)
    check_filter(logits, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 1000, 6007, 70001])
def test_equal_logits(dev, V, dtype):
    """Borders that fall exactly on a token: masses of equal weights are whole numbers."""
    g = torch.Generator(device=dev).manual_seed(V)
    level = torch.tensor([-3.0, 0.0, -0.0, 0.0], device=dev)
    x = torch.stack([torch.full((V,), 2.5, device=dev), torch.zeros(V, device=dev), level[torch.randint(4, (V,), generator=g, device=dev)],
                     torch.full((V,), -7e4, device=dev), torch.randint(2, (V,), generator=g, device=dev) * 0.125, torch.full((V,), 1.0, device=dev)])
    x[3, V // 2:] = float("-inf")
    s = settings(dev, [1.0, 0.5, 1e3, 1.0, 0.25, 30.0], [0, V // 2, 0, 0, 3, 0], [0.5, 0.25, 0.75, 0.5, 1.0, 0.375], [0.0, 1.0, 0.0, 0.0, 0.0, 0.9])
    for u in (0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24):
        check_draw(x.to(DT[dtype]), torch.full((6,), u, device=dev), s)
    check_filter(x.to(DT[dtype]), s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 20011])
def test_orders_and_runs(dev, V, dtype):
    """Rows in ascending and descending order, and rows whose largest values sit together."""
    up = torch.linspace(-20, 12, V, device=dev)
    x = torch.stack([up, up.flip(0), up.abs().neg(), torch.where(torch.arange(V, device=dev) < V // 3, up + 20, up), up * 0.01, up * 0.01])
    s = settings(dev, [1.0, 0.8, 0.3, 1.0, 1.0, 0.05], [40, 40, 0, 300, 0, 0], [0.9, 1.0, 0.9, 1.0, 0.3, 0.5], [0.0, 0.0, 0.0, 0.0, 0.0, 0.2])
    u = torch.tensor([0.3, 0.999, 0.0, 0.5, 0.77, 0.1], device=dev)
    check_draw(x.to(DT[dtype]), u, s)
    check_filter(x.to(DT[dtype]), s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [33, 3001, 40009])
def test_masked_tokens(dev, V, dtype):
    """-inf for most or all but one; a filter's border among what is left."""
    logits, u = rows(6, V, dtype, dev, V + 1)
    keep = torch.rand(6, V, device=dev, generator=torch.Generator(device=dev).manual_seed(3)) < torch.tensor([0.5, 0.1, 0.02, 0.5, 0.0, 0.9], device=dev)[:, None]
    keep[:, V // 2] = True
    logits = logits.masked_fill(~keep, float("-inf"))
    s = settings(dev, [1.0, 0.7, 1.0, 0.0, 1.0, 1.0], [0, V, 5, 0, 50, 20], [0.9, 1.0, 1.0, 1.0, 0.9, 0.0], [0.0, 0.0, 0.0, 0.0, 0.0, 0.0])
    check_draw(logits, u, s)
    check_filter(logits, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_temperatures(dev, dtype):
    """From the smallest normal number to beyond 1e37, and logits from tiny to huge."""
    T = [1.1754944e-38, 1e-30, 1e-10, 1e-4, 1e-3, 0.01, 0.1, 10.0, 100.0, 1e4, 1e10, 1e30, 3e37]
    for scale in (1e-30, 1e-3, 1.0, 300.0, 1e30):
        logits, u = rows(len(T), 2003, "f32", dev, 7)
        logits = (logits * scale).to(DT[dtype])
        s = settings(dev, T, None, [0.9] * len(T), None)
        check_draw(logits, u, s)
        check_filter(logits, s)
        check_draw(logits, u, settings(dev, T, [17] * len(T), None, [0.25] * len(T)))


UNUSABLE = [dict(value=float("nan")), dict(value=float("inf")), dict(T=float("nan")), dict(T=-1.0), dict(T=float("inf")), dict(T=1e-40), dict(k=-1), dict(p=-0.1),
            dict(p=1.5), dict(p=float("nan")), dict(m=-0.1), dict(m=1.1), dict(m=float("nan")), dict(u=1.0), dict(u=-0.5), dict(u=float("nan")), dict(empty=True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [9, 2049, 30011])
@pytest.mark.parametrize("bad", UNUSABLE, ids=lambda b: "-".join(f"{k}{v}" for k, v in b.items()))
def test_unusable_rows(dev, bad, V, dtype):
    """Such a row has no token; its neighbours are as without it."""
    logits, u = rows(3, V, dtype, dev, 11)
    s = settings(dev, [0.9] * 3, [20] * 3, [0.9] * 3, [0.001] * 3)
    if "value" in bad:
        logits[1, V - 2] = bad["value"]
    if "empty" in bad:
        logits[1] = float("-inf")
    for n, key in (("T", "temperature"), ("k", "top_k"), ("p", "top_p"), ("m", "min_p")):
        if n in bad:
            s[key][1] = bad[n]
    if "u" in bad:
        u[1] = bad["u"]
    tok, prob, kept = sv.spec_sample_filtered(logits, u, **s)
    assert tok[1].item() == -1 and prob[1].isnan().item() and kept[1].item() == -1
    check_draw(logits, u, s, (tok, prob, kept))
    if "u" not in bad:
        out, kept = sv.spec_filter_logits(logits, **s)
        assert out[1].isnan().all() and kept[1].item() == -1
        check_filter(logits, s, (out, kept))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,B", [(2049, 3), (30011, 3), (60000, 1)])
@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf"), None])
def test_unusable_rows_whatever_the_filters(dev, bad, V, B, dtype):
    logits, u = rows(B, V, dtype, dev, 15)
    if bad is None:
        logits[B - 1] = float("-inf")
    else:
        logits[B - 1, V // 3] = bad
        if bad != bad and dtype == "bf16":   # both signs of a NaN
            logits.view(torch.int16)[B - 1, V // 3] = 0x7fc1 if str(bad)[0] != "-" else -0x3f
    for one in (dict(), dict(k=[0] * B, p=[0.9] * B), dict(k=[700] * B), dict(k=[V] * B), dict(m=[0.1] * B), dict(k=[3] * B, p=[0.5] * B)):
        s = settings(dev, [0.8] * B, **one)
        check_draw(logits, u, s)
        check_filter(logits, s)
    s = settings(dev, [0.0] * B)
    check_draw(logits, u, s)
    check_filter(logits, s)


@pytest.mark.parametrize("V", [2500, 40000, 128256])
def test_top_k_of_every_size(dev, V):
    for dtype in ("bf16", "f32"):
        ks = [1, 2, 127, 128, 129, 1000, 1025, 2048, 2049, V - 1, V, V + 1, 2 ** 31 - 1]
        logits, u = rows(len(ks), V, dtype, dev, V + 2)
        for p in (None, [0.7] * len(ks)):
            s = settings(dev, [0.9] * len(ks), ks, p)
            check_draw(logits, u, s)
            check_filter(logits, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2049, 4096, 30011])
@pytest.mark.parametrize("sigma", [6.0, 40.0, -40.0])
def test_logits_far_apart(dev, sigma, V, dtype):
    """Neighbouring bf16 values of these weigh 2^-10 of one another and less; the largest logit is a large one, or
    (sigma below 0) below zero."""
    logits, u = rows(40, V, dtype, dev, V, abs(sigma))
    if sigma < 0:
        logits = -logits.abs() - 3
    rng = np.random.default_rng(V)
    T = rng.uniform(0.05, 2.0, 40)
    check_draw(logits, u, settings(dev, T))
    check_filter(logits, settings(dev, T, p=rng.uniform(0.1, 1.0, 40)))
    s = settings(dev, T, k=rng.integers(1, V, 40), p=rng.uniform(0.5, 1.0, 40))
    check_draw(logits, u, s)
    check_filter(logits, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_beyond_the_usual_range(dev, dtype):
    """Near zero, far below, and around 256: what the counted levels of bf16 rows do not cover."""
    V = 9000
    base, u = rows(8, V, dtype, dev, 60)
    x = base.float()
    x[0, ::2] *= 1e-9                       # half of the row next to zero
    x[1] *= 1e-9
    x[2, ::3] = 0.0
    x[2, 1::3] = -0.0
    x[3, ::2] = -1e4                        # a finite mask
    x[4] += 300
    x[5] -= 300
    x[6, 5:] = -300 - x[6, 5:].abs()        # five tokens and a far tail
    x[7, :10] = torch.arange(10, device=dev) * 1e-8
    x = x.to(DT[dtype])
    for T, k, p in ((1.0, None, [0.9] * 8), (20.0, None, [0.5] * 8), (0.7, [600] * 8, [0.99] * 8), (1.0, None, None), (300.0, None, [0.999] * 8)):
        s = settings(dev, [T] * 8, k, p)
        check_draw(x, u, s)
        check_filter(x, s)


def test_a_large_batch_against_a_plain_sort(dev):
    """Whole numbers over many rows: nothing that happens once in a few hundred."""
    B, V = 700, 20011
    for dtype in ("bf16", "f32"):
        logits, u = rows(B, V, dtype, dev, 70, sigma=2.5)
        T = torch.rand(B, device=dev) + 0.4
        p = torch.rand(B, device=dev) * 0.9 + 0.05
        tok, _, kept = sv.spec_sample_filtered(logits, u, T, top_p=p)
        value, order = torch.sort(logits.double(), dim=-1, descending=True, stable=True)
        w = torch.exp((value - value[:, :1]) / T.double()[:, None])
        mass = torch.cumsum(w, -1)
        n = (mass - w < p.double()[:, None] * mass[:, -1:]).sum(-1)
        end = mass.gather(1, n[:, None] - 1)
        r = (mass <= u.double()[:, None] * end).sum(-1)
        assert torch.equal(kept.long(), n) and torch.equal(tok.long(), order.gather(1, r[:, None])[:, 0])


def test_a_capture_may_be_the_first_call():
    code = ("import torch, speculative_decoding_verification_04_gb300 as sv\n"
            "x = torch.randn(2, 9000, device='cuda'); T = torch.ones(2, device='cuda'); u = torch.full((2,), 0.5, device='cuda')\n"
            "p = torch.full((2,), 0.9, device='cuda')\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g):\n    a = sv.spec_sample_filtered(x, u, T, top_p=p)\n"
            "g.replay(); torch.cuda.synchronize()\n"
            "b = sv.spec_sample_filtered(x, u, T, top_p=p)\n"
            "assert all(torch.equal(i, j) for i, j in zip(a, b))\n")
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=120)


def test_greedy_rows_read_no_uniform_and_no_filter_value(dev):
    logits, u = rows(2, 3001, "bf16", dev, 12)
    u[:] = float("nan")
    s = settings(dev, [0.0, 0.0], [1, 0], [0.5, 1.0], None)
    check_draw(logits, u, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [13, 4096, 9001])
def test_rows_that_are_not_real_stay(dev, V, dtype):
    B, S = 5, 4
    logits, _ = rows(B * S, V, dtype, dev, 13)
    logits = logits.view(B, S, V)
    n = torch.tensor([4, 0, 1, 3, 2], dtype=torch.int32, device=dev)
    for b in range(B):
        logits[b, n[b].item():] = float("nan")
    s = settings(dev, [0.7, 1.0, 0.9, 0.0, 1.2], [5, 0, 0, 0, 1], [1.0, 0.9, 0.9, 1.0, 1.0], None)
    out = torch.full_like(logits, 77.0)
    got, kept = sv.spec_filter_logits(logits, **s, n_rows=n, out=out)
    assert got.data_ptr() == out.data_ptr()
    for b in range(B):
        r = n[b].item()
        assert (out[b, r:] == 77).all() and (kept[b, r:] == 0).all()
        one = {k: None if v is None else v[b:b + 1] for k, v in s.items()}
        if r:
            check_filter(logits[b:b + 1, :r].contiguous(), one, (out[b:b + 1, :r], kept[b:b + 1, :r]))
    same = logits.clone()
    again, kept2 = sv.spec_filter_logits(same, **s, n_rows=n, out=same)
    real = (torch.arange(S, device=dev) < n[:, None])[:, :, None].expand_as(out)
    assert torch.equal(again[real], out[real]) and torch.equal(kept, kept2) and again[~real].isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [64, 5001, 131072])
@pytest.mark.parametrize("at,to", [(0, 1), (1, 0), (1, 1), (3, 2), (5, 5)])
def test_addresses_that_are_not_aligned(dev, at, to, V, dtype):
    B = 3
    x, u = rows(B, V, dtype, dev, 14)
    space = torch.zeros(B * V + 16, dtype=DT[dtype], device=dev)
    room = torch.full((B * V + 16,), 5.0, dtype=DT[dtype], device=dev)
    logits = space[at:at + B * V].view(B, V)
    logits.copy_(x)
    out = room[to:to + B * V].view(B, V)
    s = settings(dev, [0.8, 1.0, 1.0], [30, 0, 0], [1.0, 0.9, 1.0], [0.0, 0.0, 0.01])
    check_draw(logits, u, s)
    check_filter(logits, s, sv.spec_filter_logits(logits, **s, out=out))
    assert (room[:to] == 5).all() and (room[to + B * V:] == 5).all()


def test_other_stream_and_overlapping_calls(dev):
    sets = [rows(64, 20001, "bf16", dev, 20 + i) for i in range(4)]
    s = settings(dev, [0.9] * 64, [40] * 32 + [0] * 32, [0.9] * 64, None)
    want = [[t.clone() for t in sv.spec_sample_filtered(x, u, **s)] for x, u in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(3):
        for i, (x, u) in enumerate(sets):
            got[i].append(sv.spec_sample_filtered(x, u, **s, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(4):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_graph_replays_on_new_inputs(dev):
    x, u = rows(6, 12007, "f32", dev, 30)
    s = settings(dev, [0.9] * 6, [40, 0, 0, 5, 600, 0], [0.9] * 6, [0.0, 0.0, 0.03, 0.0, 0.0, 0.0])
    out = torch.empty_like(x)
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    sv.spec_sample_filtered(x, u, **s)
    sv.spec_filter_logits(x, **s, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        drawn = sv.spec_sample_filtered(x, u, **s)
    with torch.cuda.graph(h):
        kept = sv.spec_filter_logits(x, **s, out=out)[1]
    for seed in (31, 32):
        y, v = rows(6, 12007, "f32", dev, seed)
        x.copy_(y)
        u.copy_(v)
        s["top_p"].uniform_(0.3, 0.95)
        g.replay()
        h.replay()
        torch.cuda.synchronize()
        check_draw(x, u, s, drawn)
        check_filter(x, s, (out, kept))


def test_empty_batches(dev):
    x = torch.empty(0, 50, dtype=torch.bfloat16, device=dev)
    e = torch.empty(0, device=dev)
    assert [t.shape for t in sv.spec_sample_filtered(x, e, e)] == [(0,)] * 3
    assert sv.spec_filter_logits(x, e)[0].shape == (0, 50)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 9007])
def test_draws_follow_the_shares(dev, V, dtype):
    """Every u: the tokens that come out, one u after the other, hold their shares of [0, 1)."""
    n = 512
    x, _ = rows(1, V, dtype, dev, 40)
    u = (torch.arange(n, device=dev) + 0.5) / n
    s = settings(dev, [0.9] * n, [30] * n, [0.95] * n, None)
    tok, prob, _ = sv.spec_sample_filtered(x.expand(n, V).contiguous(), u, **s)
    seen = dict(zip(tok.tolist(), prob.tolist()))
    count = torch.bincount(tok.long(), minlength=V)
    for t, share in seen.items():
        assert abs(count[t].item() - share * n) <= 1.001
    assert (prob[1:] <= prob[:-1]).all()   # the order of the draw
