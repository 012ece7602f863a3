"""Rounds of speculative decoding with the filters and the page operators where
a serving loop has them: pages are reserved, tokens drafted with filters,
written, attended to, verified against filtered rows, committed, and pages past
the new lengths go back."""
import random

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
from filter_helpers import kept_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def floats(v, dev):
    return torch.tensor(v, dtype=torch.float32, device=dev)


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_filtered_verification_is_lossless(dev, dtype):
    """Whatever the draft, the first committed token follows the target's filtered
    distribution: over n rounds a share p of it within 5 standard deviations."""
    n, V = 40000, 61
    gen = torch.Generator(device=dev).manual_seed(5)
    target, draft = (torch.randn(V, generator=gen, device=dev).mul(1.5).to(dtype) for _ in range(2))
    T, k, p = 0.8, 20, 0.9
    one = dict(top_k=ints([k] * n, dev), top_p=floats([p] * n, dev))
    Tn = floats([T] * n, dev)
    q_rows = draft.expand(n, 1, V).contiguous()
    p_rows = target.expand(n, 2, V).contiguous()
    x, share, kept = sv.spec_sample_filtered(q_rows.view(n, V), torch.rand(n, generator=gen, device=dev), Tn, **one)
    sv.spec_filter_logits(q_rows, Tn, out=q_rows, **one)
    sv.spec_filter_logits(p_rows, Tn, out=p_rows, **one)
    u = torch.rand(n, 2, generator=gen, device=dev) * 0.9999999
    tokens, accepted = sv.spec_verify(p_rows, q_rows, x.view(n, 1), u, Tn, [1] * n)
    assert (accepted >= 0).all() and 0 < accepted.float().mean().item() < 1
    order, w = kept_of(target.double().cpu().numpy(), T, k, p)
    assert kept.unique().numel() == 1 and share.min() > 0
    first = torch.bincount(tokens[:, 0].long(), minlength=V).cpu().double() / n
    want = torch.zeros(V, dtype=torch.float64)
    want[torch.from_numpy(order.copy())] = torch.from_numpy(w / w.sum())
    assert (first[want == 0] == 0).all()
    assert ((first - want).abs() <= 5 * (want * (1 - want) / n).sqrt() + 1e-12).all()


def test_rounds_over_a_shared_pool(dev):
    """The pool serves sequences that grow, shrink to what was verified, end and
    start again; every round the cache holds what was committed, no page is held
    twice, and none is lost."""
    rng = random.Random(4)
    gen = torch.Generator(device=dev).manual_seed(6)
    B, N, V, Hq, Hkv, D, page, width = 9, 7, 900, 4, 2, 64, 8, 12
    pages = 40                                       # too few for all to grow at once
    kc, vc = (torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    kv_len, held = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(2))
    stack, count = torch.arange(pages, dtype=torch.int32, device=dev), ints([pages], dev)
    errors = torch.zeros(1, dtype=torch.int32, device=dev)
    parent = ints([[-1, 0, 0, 1, 1, 2, 2]] * B, dev)
    nodes = ints([N] * B, dev)
    settings = dict(temperature=floats([0.9, 0.0, 1.2] * 3, dev), top_k=ints([30, 0, 0] * 3, dev), top_p=floats([0.95, 1.0, 0.9] * 3, dev))
    embed = torch.randn(V, Hkv, D, generator=gen, device=dev).to(torch.bfloat16)
    bigram = torch.randn(V, V, generator=gen, device=dev).mul(2).to(torch.bfloat16)
    history = [[] for _ in range(B)]
    starved = 0
    for _ in range(25):
        errors.zero_()
        slots = torch.empty(B, N, dtype=torch.int64, device=dev)
        sv.spec_kv_reserve(table, kv_len, held, stack, count, page, S=N, slots=slots, errors=errors)
        ok = (slots[:, 0] >= 0).tolist()
        assert bool(errors.item() & 8) == (not all(ok)) and errors.item() & ~8 == 0
        starved += ok.count(False)
        # the drafts: children drawn from their parent's filtered row
        tokens = torch.randint(V, (B, N), generator=gen, device=dev)
        for n in range(1, N):
            row = bigram[tokens[:, parent[0, n].item()]]
            tokens[:, n] = sv.spec_sample_filtered(row, torch.rand(B, generator=gen, device=dev), **settings)[0]
        draft = bigram[tokens]
        k = embed[tokens]
        v = k.flip(-1).contiguous()
        before = errors.item()
        sv.spec_kv_append(k, v, kc, vc, table, kv_len, parent=parent, errors=errors)
        assert errors.item() == (before if all(ok) else before | 4)   # what was refused is not written, and reported
        # the slot map is where the keys are
        flat = kc.permute(0, 2, 1, 3).reshape(-1, Hkv, D)
        for b in range(B):
            if ok[b]:
                assert torch.equal(flat[slots[b]], k[b])
        o = sv.spec_tree_attention(torch.randn(B, N, Hq, D, generator=gen, device=dev).to(torch.bfloat16), kc, vc, table, kv_len, parent=parent)
        assert not o[ok].isnan().any()
        target = draft + torch.randn(B, N, V, generator=gen, device=dev).to(torch.bfloat16)
        kept_t = sv.spec_filter_logits(target, **settings, n_rows=nodes, out=target)[1]
        sv.spec_filter_logits(draft, **settings, n_rows=nodes, out=draft)
        assert (kept_t[1::3] == 1).all() and (kept_t[0::3] <= 30).all()
        u = torch.rand(B, N, generator=gen, device=dev) * 0.9999999
        out, path, length = sv.spec_verify_tree(target, draft, tokens.int(), parent, u, settings["temperature"], nodes)
        assert (length >= 0).all()
        for b in range(B):
            n = length[b].item()
            at = path[b, n - 1].item() if n else 0
            assert target[b, at, out[b, n]].item() > float("-inf")    # the last token is one that the filters keep
        length = torch.where(torch.tensor(ok, device=dev), length, -1)    # a refused sequence waits for the next round
        sv.spec_kv_commit(kc, vc, table, kv_len, path, length, errors=errors)
        for b in range(B):
            if ok[b]:
                history[b] += [tokens[b, 0].item()] + out[b, :length[b]].tolist()
            if len(history[b]) > width * page - 2 * N or (not all(ok) and rng.random() < 0.3):   # it ends, another starts in its place
                history[b] = []
                kv_len[b] = 0
        errors.zero_()
        sv.spec_kv_release(table, kv_len, held, stack, count, page, errors=errors)
        assert errors.item() == 0 and kv_len.tolist() == [len(h) for h in history]
        assert held.tolist() == [-(-len(h) // page) for h in history]
        mine = [p for b in range(B) for p in table[b, :held[b]].tolist()]
        assert sorted(mine + stack[:count.item()].tolist()) == list(range(pages))
        rows = [len(h) for h in history]
        starts = ints([sum(rows[:b]) for b in range(B + 1)], dev)
        got, _ = sv.spec_kv_read(kc, vc, table, torch.zeros_like(kv_len), starts, sum(rows))
        assert torch.equal(got, embed[torch.tensor(sum(history, []), dtype=torch.long, device=dev)])
    assert starved > 0
