"""Performance cases of the operators around verification: filtered sampling, filtered logits, and the cache's pages.

A serving loop that decodes speculatively does four more things on the device between the model's forward passes:

  sample     a token per row from softmax(logits / T) after min-p, top-k and top-p (the draft model's step)
  filter     the same filters on rows of logits, kept tokens as they are and the rest -inf (what verification then reads)
  reserve    pages for the new tokens of each sequence from a stack of free ones into its page table, and each token's slot
  release    pages past each sequence's length go back onto the stack

The filters: tokens are ordered by logit, the largest first, equal ones by index.  min-p drops those whose weight
exp((l - max) / T) is below min_p, top-k keeps the first k of the rest, top-p the shortest prefix of these that holds
the share p of their mass.  A draw takes the first token whose cumulative mass is above u times the kept mass.
T = 0 is the argmax.

``own`` selects the library's kernels; otherwise the same results are computed with elementary torch operations.
``exact`` computes them in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user's next token: latency
        dict(name="sample_1_bf16", kind="sample", B=1, V=128256, dtype="bf16", filters="k"),
        # a batch of drafts, every user with settings of their own, some of them greedy
        dict(name="sample_1024_bf16", kind="sample", B=1024, V=128256, dtype="bf16", filters="mixed"),
        # nucleus sampling alone: every token of the row counts
        dict(name="sample_256_f32", kind="sample", B=256, V=151936, dtype="f32", filters="p"),
        # an odd vocabulary, rows that start anywhere
        dict(name="sample_odd_bf16", kind="sample", B=37, V=50257, dtype="bf16", filters="p"),
        # one user's target rows before verification: 8 drafts and the bonus row
        dict(name="filter_1x9_bf16", kind="filter", B=1, S=9, V=128256, dtype="bf16", filters="k"),
        # trees of 15 nodes, ragged, settings of their own
        dict(name="filter_64x15_bf16", kind="filter", B=64, S=15, V=128256, dtype="bf16", filters="mixed"),
        # an odd vocabulary in 32 bits
        dict(name="filter_odd_f32", kind="filter", B=29, S=5, V=32003, dtype="f32", filters="p"),
        # a few users, a chain of 8 drafts and the root
        dict(name="reserve_8x9", kind="reserve", B=8, N=9, packed=False, lo=0, hi=2000, page=16, stock=1.5),
        # a large batch of trees, and a pool that runs out
        dict(name="reserve_1024x15", kind="reserve", B=1024, N=15, packed=False, lo=100, hi=1500, page=16, stock=0.9),
        # prompts that arrive together
        dict(name="reserve_prompts", kind="reserve", B=64, N=2000003, packed=True, lo=0, hi=0, page=64, stock=1.1),
        # the large batch of trees after verification
        dict(name="release_1024x15", kind="release", B=1024, N=15, lo=100, hi=1500, page=16, done=0.02),
        # long conversations, half of which have ended
        dict(name="release_ended", kind="release", B=2048, N=32, lo=1, hi=32000, page=16, done=0.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["sample", "sample", "filter", "filter", "reserve", "release"])
    if kind in ("sample", "filter"):
        V = rng.choice([_log_int(rng, 2, 1024), _log_int(rng, 1025, 40000), _log_int(rng, 32000, 200000), 32000, 128256, 151936])
        c = dict(kind=kind, B=_log_int(rng, 1, 512), V=V, dtype=rng.choice(["bf16", "bf16", "f32"]), filters=rng.choice(["k", "p", "min", "mixed", "none"]))
        if kind == "filter":
            c["S"] = rng.randint(1, 15)
        most = max(1, 40000000 // (V * c.get("S", 1)))
        c["B"] = min(c["B"], most)
        return c
    B, page = _log_int(rng, 1, 2048), rng.choice([8, 16, 32, 64, 128])
    hi = _log_int(rng, 16, max(17, min(60000, 20000000 // B)))
    if kind == "reserve":
        packed = rng.random() < 0.4
        N = _log_int(rng, B, 1000000) if packed else rng.randint(1, 32)
        return dict(kind=kind, B=B, N=max(N, B) if packed else N, packed=packed, lo=0, hi=hi, page=page, stock=rng.choice([0.3, 0.9, 1.2, 2.0]))
    return dict(kind=kind, B=B, N=rng.randint(1, 32), lo=0, hi=hi, page=page, done=rng.choice([0.0, 0.05, 0.5, 1.0]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _split(rng, total, B):
    """B lengths of at least one that add up to total."""
    w = [rng.expovariate(1.0) + 0.05 for _ in range(B)]
    n = [1 + int((total - B) * x / sum(w)) for x in w]
    n[-1] += total - sum(n)
    return n


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _floats(v):
    return torch.tensor(v, dtype=torch.float32, device=DEV)


def _settings(rng, filters, B, V):
    """Temperature, top-k, top-p and min-p of each sequence (None: the filter is off for all)."""
    T, k, p, m = [], [], [], []
    for _ in range(B):
        f = rng.choice(["k", "p", "min", "none", "greedy", "k"]) if filters == "mixed" else filters
        T.append(0.0 if f == "greedy" else rng.uniform(0.5, 1.2))
        k.append(min(V, rng.choice([20, 40, 50, 64, 100, 500])) if f == "k" else 0)
        p.append(rng.uniform(0.8, 0.98) if f in ("k", "p") else 1.0)
        m.append(rng.uniform(0.02, 0.2) if f == "min" else 0.0)
    return dict(temperature=_floats(T), top_k=_ints(k) if any(k) else None, top_p=_floats(p) if min(p) < 1.0 else None,
                min_p=_floats(m) if any(m) else None)


def _logits(rng, gen, rows, V, dtype):
    """Rows of a language model's logits: a bulk of unlikely tokens and a few that stand out, by more in some rows than in others."""
    x = torch.randn(rows, V, generator=gen, device=DEV).mul_(2.0)
    n = min(V, 24)
    at = torch.randint(V, (rows, n), generator=gen, device=DEV)
    lead = torch.rand(rows, 1, generator=gen, device=DEV) * 6.0 + 3.0
    x.scatter_reduce_(1, at, lead * (0.6 + 0.6 * torch.rand(rows, n, generator=gen, device=DEV)), "amax")   # (an index drawn twice: the larger)
    return x.to(dtype)


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind, B = case["kind"], case["B"]
    s = dict(kind=kind)
    if kind == "sample":
        s.update(_settings(rng, case["filters"], B, case["V"]), logits=_logits(rng, gen, B, case["V"], DTYPES[case["dtype"]]),
                 uniforms=torch.rand(B, generator=gen, device=DEV))
        return s
    if kind == "filter":
        S, V = case["S"], case["V"]
        logits = _logits(rng, gen, B * S, V, DTYPES[case["dtype"]]).view(B, S, V)
        # ragged, the first sequence's rows all real
        s.update(_settings(rng, case["filters"], B, V), logits=logits, n_rows=_ints([S] + [rng.randint(max(1, S - 3), S) for _ in range(B - 1)]),
                 out=torch.zeros_like(logits))
        return s
    page = case["page"]
    s["page"] = page
    if kind == "reserve":
        ctx = [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(B - 1)]
        if case["packed"]:
            new = _split(rng, case["N"], B)
            s["row_start"] = _ints([sum(new[:i]) for i in range(B + 1)])
            s["slots"] = torch.empty(case["N"], dtype=torch.int64, device=DEV)
        else:
            new = [case["N"]] + [rng.randint(max(1, case["N"] - 3), case["N"]) for _ in range(B - 1)]
            s["n_new"], s["S"] = _ints(new), case["N"]
            s["slots"] = torch.empty(B, case["N"], dtype=torch.int64, device=DEV)
        held = [-(-c // page) for c in ctx]
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        free = max(1, int(sum(n - h for n, h in zip(need, held)) * case["stock"]))
        width = -(-(case["hi"] + case["N"]) // page)
        count, at = max(free, B * width), ctx
    else:
        # after verification: pages for N drafted tokens are held, a few of them were kept, some sequences have ended
        ctx = [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(B - 1)]
        held = [-(-(c + case["N"]) // page) for c in ctx]
        at = [0 if rng.random() < case["done"] else c + rng.randint(0, min(3, case["N"])) for c in ctx]
        width, free = held[0], 64
        count = free + B * width
    held_at = torch.tensor(held, device=DEV)
    ids = torch.randperm(sum(held) + free, generator=gen, device=DEV, dtype=torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV) < held_at[:, None]] = ids[:sum(held)]
    stack = torch.full((count,), -1, dtype=torch.int32, device=DEV)
    stack[:free] = ids[sum(held):sum(held) + free]
    s.update(page_table=table, kv_len=_ints(at), held=_ints(held), free_pages=stack, free_count=_ints([free]),
             held_out=_ints(held), free_count_out=_ints([0]))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    kind = s["kind"]
    if own:
        import speculative_decoding_verification_04_gb300 as sv
        if kind == "sample":
            return list(sv.spec_sample_filtered(s["logits"], s["uniforms"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"]))
        if kind == "filter":
            return list(sv.spec_filter_logits(s["logits"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                                              n_rows=s["n_rows"], out=s["out"]))
        pool = (s["page_table"], s["kv_len"], s["held"], s["free_pages"], s["free_count"], s["page"])
        outs = dict(held_out=s["held_out"], free_count_out=s["free_count_out"])
        if kind == "reserve":
            sv.spec_kv_reserve(*pool, S=s.get("S"), n_new=s.get("n_new"), row_start=s.get("row_start"), slots=s["slots"], **outs)
            return [s["page_table"], s["held_out"], s["free_count_out"], s["slots"]]
        sv.spec_kv_release(*pool, **outs)
        return [s["free_pages"], s["held_out"], s["free_count_out"]]
    return {"sample": _plain_sample, "filter": _plain_filter, "reserve": _plain_reserve, "release": _plain_release}[kind](s)


def _kept(x, T, top_k, top_p, min_p):
    """Rows x [R, V] sorted: their order, weights, cumulative kept mass and the length of the kept prefix."""
    V = x.shape[1]
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    greedy = (T == 0)[:, None]
    value = value.double()
    w = torch.exp((value - value[:, :1]) / torch.where(greedy, 1.0, T.double()[:, None]))
    rank = torch.arange(V, device=DEV)
    keep = (value > -math.inf) & (~greedy | (rank == 0))
    if min_p is not None:
        keep &= greedy | (w >= min_p.double()[:, None])
    if top_k is not None:
        k = top_k[:, None]
        keep &= (k == 0) | (rank < k)
    if top_p is not None:
        p = top_p.double()[:, None]
        mass = torch.cumsum(w * keep, -1)
        before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], -1)
        keep &= (p >= 1.0) | (rank == 0) | (before < p * mass[:, -1:])
    return order, w, torch.cumsum(w * keep, -1), keep.sum(-1)


def _plain_sample(s):
    order, w, mass, kept = _kept(s["logits"].float(), s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    point = s["uniforms"].double()[:, None] * mass[:, -1:]
    r = torch.minimum((mass <= point).sum(-1), kept - 1)[:, None]
    r = torch.where((s["temperature"] == 0)[:, None], 0, r)
    prob = w.gather(1, r) / mass[:, -1:]
    return [order.gather(1, r)[:, 0].int(), prob[:, 0].float(), kept.int()]


def _plain_filter(s):
    B, S, V = s["logits"].shape
    of_row = lambda t: None if t is None else t.repeat_interleave(S)  # noqa: E731
    x = s["logits"].view(B * S, V)
    order, _, _, kept = _kept(x.float(), of_row(s["temperature"]), of_row(s["top_k"]), of_row(s["top_p"]), of_row(s["min_p"]))
    keep = torch.zeros(B * S, V, dtype=torch.bool, device=DEV)
    keep.scatter_(1, order, torch.arange(V, device=DEV) < kept[:, None])
    real = torch.arange(S, device=DEV) < s["n_rows"][:, None]
    new = torch.where(keep, x, torch.full((), -math.inf, dtype=x.dtype, device=DEV)).view(B, S, V)
    s["out"].copy_(torch.where(real[:, :, None], new, s["out"]))
    return [s["out"], torch.where(real, kept.view(B, S), 0).int()]


def _plain_reserve(s):
    page, table, ctx, held, stack = s["page"], s["page_table"], s["kv_len"].long(), s["held"].long(), s["free_pages"]
    free = s["free_count"].long()
    starts = s.get("row_start")
    new = s["n_new"].long() if starts is None else (starts[1:] - starts[:-1]).long()
    want = ((ctx + new + page - 1) // page - held).clamp(min=0)
    upto = torch.cumsum(want, 0)
    granted = (want == 0) | (upto <= free)
    took = want * granted
    b = torch.repeat_interleave(torch.arange(len(want), device=DEV), want)
    j = torch.arange(b.shape[0], device=DEV)
    at = held[b] + j - (upto - want)[b]
    table[b, at] = torch.where(granted[b], stack[(free - 1 - j).clamp(min=0)], -1)
    s["held_out"].copy_(held + took)
    s["free_count_out"].copy_(free - took.sum())
    if starts is None:
        i = torch.arange(s["S"], device=DEV)
        real = (i < new[:, None]) & granted[:, None]
        place = torch.where(real, ctx[:, None] + i, 0)
        slot = table.gather(1, place // page).long() * page + place % page
    else:
        t = torch.arange(s["slots"].shape[0], device=DEV)
        b = torch.searchsorted(starts.long(), t, right=True) - 1
        real = granted[b]
        place = torch.where(real, ctx[b] + t - starts.long()[b], 0)
        slot = table[b, place // page].long() * page + place % page
    s["slots"].copy_(torch.where(real, slot, -1))
    return [table, s["held_out"], s["free_count_out"], s["slots"]]


def _plain_release(s):
    page, held, stack = s["page"], s["held"].long(), s["free_pages"]
    keep = torch.minimum(held, (s["kv_len"].long() + page - 1) // page)
    count = held - keep
    upto = torch.cumsum(count, 0)
    b = torch.repeat_interleave(torch.arange(len(count), device=DEV), count)
    j = torch.arange(b.shape[0], device=DEV)
    stack[s["free_count"].long() + b.shape[0] - 1 - j] = s["page_table"][b, keep[b] + j - (upto - count)[b]]
    s["held_out"].copy_(keep)
    s["free_count_out"].copy_(s["free_count"] + upto[-1])
    return [stack, s["held_out"], s["free_count_out"]]


# ---------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------
def work(case):
    """Bytes read and written once, and operations, of one pass."""
    kind, B = case["kind"], case["B"]
    if kind in ("sample", "filter"):
        rows, size = B * case.get("S", 1), 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * case["V"] * size * (2 if kind == "filter" else 1) + rows * 12 + B * 16, "flops": rows * case["V"] * 4}
    if kind == "reserve":
        tokens = case["N"] if case["packed"] else B * case["N"]
        pages = tokens // case["page"] + 1
        return {"bytes": tokens * 8 + pages * 8 + B * 16, "flops": 0}
    ended = case["done"] * (case["lo"] + case["hi"]) / 2 / case["page"]
    return {"bytes": int(B * ((ended + case["N"] / case["page"]) * 8 + 12)), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "filter": _exact_filter, "reserve": _exact_reserve, "release": _exact_release}[s["kind"]](s)


def _host(t):
    return None if t is None else t.cpu().tolist()


class _Levels:
    """A row's kept tokens, level by level: the distinct logits in descending order, how many tokens of each are kept, and their weights."""

    def __init__(self, row, T, k, p, m):
        level, count = torch.unique(row[row > -math.inf], sorted=True, return_counts=True)
        level, count = level.flip(0), count.flip(0)
        if T == 0:
            level, count, k, p, m = level[:1], torch.ones_like(count[:1]), 0, 1.0, 0.0
        w = torch.exp((level - level[0]) / (T or 1.0))
        if m > 0:
            n = int((w >= m).sum())
            level, count, w = level[:n], count[:n], w[:n]
        if k > 0:
            before = torch.cumsum(count, 0) - count
            count = torch.minimum(count, (k - before).clamp(min=0))
        if p < 1:
            mass = torch.cumsum(count * w, 0)
            goal = p * mass[-1]
            g = int((mass < goal).sum())
            above = mass[g] - count[g] * w[g]
            count = count.clone()
            count[g] = min(int(count[g]), max(1, math.ceil(float((goal - above) / w[g]))))
            count[g + 1:] = 0
        self.level, self.count, self.w = level, count, w
        self.kept = int(count.sum())


def _exact_rows(s):
    T, k, p, m = (_host(s[n]) for n in ("temperature", "top_k", "top_p", "min_p"))
    return lambda row, b: _Levels(row.double(), T[b], k[b] if k else 0, p[b] if p else 1.0, m[b] if m else 0.0)


def _exact_sample(s):
    rows, u = _exact_rows(s), _host(s["uniforms"])
    tokens, probs, kept = [], [], []
    for b, row in enumerate(s["logits"]):
        q = rows(row, b)
        mass = torch.cumsum(q.count * q.w, 0)
        point = u[b] * float(mass[-1]) if q.kept > 1 else 0.0
        g = min(int((mass <= point).sum()), int((q.count > 0).sum()) - 1)
        above = float(mass[g] - q.count[g] * q.w[g])
        i = min(int(q.count[g]) - 1, max(0, math.floor((point - above) / float(q.w[g]))))
        tokens.append(int((row.double() == q.level[g]).nonzero()[i]))
        probs.append(float(q.w[g] / mass[-1]))
        kept.append(q.kept)
    return [_ints(tokens), torch.tensor(probs, dtype=torch.float64, device=DEV), _ints(kept)]


def _exact_filter(s):
    rows, real = _exact_rows(s), _host(s["n_rows"])
    out, kept = s["out"].double(), torch.zeros(s["logits"].shape[:2], dtype=torch.int32, device=DEV)
    for b, n in enumerate(real):
        for i in range(n):
            row = s["logits"][b, i].double()
            q = rows(row, b)
            some = int((q.count > 0).sum()) - 1
            keep = row > q.level[some]
            keep[(row == q.level[some]).nonzero()[:int(q.count[some]), 0]] = True
            out[b, i] = torch.where(keep, row, -math.inf)
            kept[b, i] = q.kept
    return [out, kept]


def _exact_reserve(s):
    page, table, ctx, held, stack = s["page"], s["page_table"].cpu(), _host(s["kv_len"]), _host(s["held"]), s["free_pages"].cpu()
    free, starts = _host(s["free_count"])[0], _host(s.get("row_start"))
    new = _host(s["n_new"]) if starts is None else [e - a for a, e in zip(starts, starts[1:])]
    slots = torch.full(s["slots"].shape, -1, dtype=torch.int64)
    asked, out = 0, []
    for b, c in enumerate(ctx):
        want = max(0, -(-(c + new[b]) // page) - held[b])
        fits = want == 0 or asked + want <= free
        table[b, held[b]:held[b] + want] = stack[free - asked - want:free - asked].flip(0) if fits else -1
        out.append(held[b] + (want if fits else 0))
        asked += want
        if fits:
            place = torch.arange(c, c + new[b])
            line = slots[b, :new[b]] if starts is None else slots[starts[b]:starts[b + 1]]
            line.copy_(table[b][place // page].long() * page + place % page)
    return [table.to(DEV), _ints(out), _ints([free - sum(out) + sum(held)]), slots.to(DEV)]


def _exact_release(s):
    page, table, ctx, held = s["page"], s["page_table"].cpu(), _host(s["kv_len"]), _host(s["held"])
    free = _host(s["free_count"])[0]
    keep = [min(h, -(-c // page)) for c, h in zip(ctx, held)]
    back = torch.cat([table[b, k:h] for b, (k, h) in enumerate(zip(keep, held))]).flip(0)
    stack = s["free_pages"].cpu()
    stack[free:free + len(back)] = back
    return [stack.to(DEV), _ints(keep), _ints([free + len(back)])]
