"""Performance cases of the tree-decode operators: the paged key/value cache around token-tree verification.

A speculative decoding step that drafts a tree of tokens does four things with
its key/value cache besides verifying the tree:

  append     per-head norms of queries and keys, the position rotation, and the write of keys and values into the paged
             cache (bf16, or e4m3 with one scale per token and head)
  attention  every tree node attends to the cached context and to its own ancestors
  commit     after verification the kept path's keys and values move to consecutive positions
  read       a range of the cache comes back as dense rows (cache migration, prefix reuse)

``own`` selects the library's kernels; otherwise the same results are computed
with elementary torch operations in 32 bits.  ``exact`` computes them in 64
bits from the definitions.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100   # a row of zeros (or nearly) still gets a usable scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user, one token: the latency of a plain decode step
        dict(name="attention_1x1", kind="attention", B=1, N=1, tree="chain", lo=700, hi=700, Hq=32, Hkv=8, D=128, fmt="bf16", page=16),
        # chains of 8 drafts (the K = 8 workload) for 64 users over an 8-bit cache
        dict(name="attention_chain_e4m3", kind="attention", B=64, N=9, tree="chain", lo=200, hi=3000, Hq=32, Hkv=8, D=128, fmt="e4m3", page=64),
        # the tree benchmark's batch: 256 binary trees of 15 nodes
        dict(name="attention_trees_bf16", kind="attention", B=256, N=15, tree="binary", lo=100, hi=1500, Hq=32, Hkv=8, D=128, fmt="bf16", page=16),
        # two long conversations, trees as large as verification takes (32 nodes)
        dict(name="attention_long_e4m3", kind="attention", B=2, N=32, tree="random", lo=100001, hi=120007, Hq=32, Hkv=8, D=128, fmt="e4m3", page=128),
        # odd sizes throughout: 80-wide heads, 5 query heads to a key head, pages of 8
        dict(name="attention_odd_bf16", kind="attention", B=13, N=31, tree="random", lo=1, hi=9001, Hq=20, Hkv=4, D=80, fmt="bf16", page=8),
        # one token for each of 8 users, fp32 activations, part of the head rotated in adjacent pairs
        dict(name="append_tokens_f32", kind="append", B=8, N=1, tree="chain", packed=False, lo=0, hi=2000, Hq=20, Hkv=4, D=80, rot=32, pairs=True, norm=False,
             dtype="f32", fmt="bf16", page=16),
        # the tree benchmark's batch written to an 8-bit cache
        dict(name="append_trees_e4m3", kind="append", B=256, N=15, tree="binary", packed=False, lo=100, hi=1500, Hq=32, Hkv=8, D=128, rot=128, pairs=False, norm=True,
             dtype="bf16", fmt="e4m3", page=16),
        # ragged prompts, packed one after the other
        dict(name="append_prompts_bf16", kind="append", B=12, N=16411, tree="chain", packed=True, lo=0, hi=0, Hq=32, Hkv=8, D=128, rot=128, pairs=False, norm=True,
             dtype="bf16", fmt="bf16", page=32),
        # a few users, two layers (a draft model's cache)
        dict(name="commit_4x2", kind="commit", B=4, N=15, tree="binary", layers=2, lo=0, hi=500, Hkv=8, D=128, fmt="bf16", page=16),
        # the tree benchmark's batch, 32 layers
        dict(name="commit_256x32_e4m3", kind="commit", B=256, N=15, tree="binary", layers=32, lo=20, hi=100, Hkv=8, D=128, fmt="e4m3", page=16),
        # short odd ranges to fp32
        dict(name="read_odd_f32", kind="read", B=5, N=777, lo=0, hi=300, Hkv=4, D=80, fmt="e4m3", page=8, dtype="f32"),
        # a batch's whole 8-bit cache back to bf16
        dict(name="read_batch_bf16", kind="read", B=64, N=100003, lo=0, hi=700, Hkv=8, D=128, fmt="e4m3", page=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "append", "commit", "read"])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 80, 96, 112, 128, 128, 192, 256])
    fmt = rng.choice(["bf16", "e4m3"])
    page = rng.choice([8, 16, 32, 64, 128])
    tree = rng.choice(["chain", "binary", "random"])
    N = 1 if rng.random() < 0.2 else rng.randint(2, 32)
    G = rng.choice([1, 2, 3, 4, 5, 6, 8])
    B = _log_int(rng, 1, 256)
    if kind == "attention":
        hi = _log_int(rng, 64, max(65, min(120000, 180000 * 8 * 128 // (B * Hkv * D), 200000 // B)))
        return dict(kind=kind, B=B, N=N, tree=tree, lo=rng.randint(0, hi), hi=hi, Hq=G * Hkv, Hkv=Hkv, D=D, fmt=fmt, page=page)
    if kind == "append":
        packed = rng.random() < 0.4
        if packed:
            B = min(B, 64)
            N, tree = _log_int(rng, B, 8000), "chain"
        return dict(kind=kind, B=B, N=N, tree=tree, packed=packed, lo=0, hi=0 if packed else rng.randint(1, 1000), Hq=min(G, 4) * Hkv, Hkv=Hkv, D=D,
                    rot=rng.choice([0, 32, 64, D]), pairs=rng.random() < 0.3, norm=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "f32"]), fmt=fmt, page=page)
    if kind == "commit":
        layers = _log_int(rng, 1, 32)
        return dict(kind=kind, B=min(B, 128), N=max(2, N), tree=tree, layers=layers, lo=0, hi=rng.randint(1, 100), Hkv=Hkv, D=D, fmt=fmt, page=page)
    return dict(kind=kind, B=min(B, 64), N=_log_int(rng, 64, 60000), lo=0, hi=rng.randint(1, 1000), Hkv=Hkv, D=D, fmt=fmt, page=page, dtype=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _parents(rng, tree, N):
    if tree == "binary":
        return [-1] + [(n - 1) // 2 for n in range(1, N)]
    if tree == "random":
        return [-1] + [rng.randrange(max(0, n - 6), n) for n in range(1, N)]
    return [-1] + list(range(N - 1))


def _lengths(rng, case):
    """Context lengths, spread over lo..hi; the first is hi itself."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi] + [rng.randint(lo, hi) for _ in range(B - 1)]


def _split(rng, total, B):
    """B lengths of at least one that add up to total."""
    w = [rng.expovariate(1.0) + 0.05 for _ in range(B)]
    n = [1 + int((total - B) * x / sum(w)) for x in w]
    n[-1] += total - sum(n)
    return n


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(rng, need, page, pool):
    """A page table whose sequences own shuffled pages of a pool that holds `pool` tokens; entries past a sequence's last page are -1."""
    count = [max(1, -(-n // page)) for n in need]
    num = -(-pool // page) + len(need)
    ids = rng.sample(range(num), sum(count))
    width, rows, at = max(count), [], 0
    for c in count:
        rows.append(ids[at:at + c] + [-1] * (width - c))
        at += c
    return _ints(rows), num


def _cache(gen, case, num_pages, layers=None):
    shape = ([layers] if layers else []) + [num_pages, case["Hkv"], case["page"], case["D"]]
    made = {}
    for n in ("k", "v"):
        if case["fmt"] == "bf16":
            made[n + "_cache"] = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
            made[n + "_scale"] = None
        else:
            x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX)
            made[n + "_cache"] = x.to(torch.float8_e4m3fn)
            made[n + "_scale"] = torch.rand(shape[:-1], generator=gen, device=DEV).mul_(0.01).add_(0.005)
    return made


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind, page, D, Hkv = case["kind"], case["page"], case["D"], case["Hkv"]
    s = dict(kind=kind, page=page)

    def normal(*shape, dtype, by=1.0):
        return torch.randn(shape, generator=gen, device=DEV).mul_(by).to(dtype)

    if kind == "read":
        count = _split(rng, case["N"], case["B"])
        start = _lengths(rng, case)
        s["page_table"], pages = _pages(rng, [a + c for a, c in zip(start, count)], page, case["N"] + case["B"] * case["hi"])
        s.update(_cache(gen, case, pages), start=_ints(start), rows=case["N"], dtype=DTYPES[case["dtype"]],
                 row_start=_ints([sum(count[:i]) for i in range(len(count) + 1)]))
        return s
    B, N = case["B"], case["N"]
    ctx = _lengths(rng, case)
    s["kv_len"] = _ints(ctx)
    if kind == "append" and case["packed"]:
        count = _split(rng, N, B)
        s["row_start"] = _ints([sum(count[:i]) for i in range(B + 1)])
        tokens, need, longest = (N,), [a + c for a, c in zip(ctx, count)], max(count)
    else:
        # ragged node counts, the first sequence's whole
        nodes = [N] + [rng.randint(max(1, N - 3), N) for _ in range(B - 1)]
        s["n_nodes"] = _ints(nodes)
        s["parent"] = None if case["tree"] == "chain" else _ints([_parents(rng, case["tree"], N) for _ in range(B)])
        tokens, need, longest = (B, N), [a + N for a in ctx], N
    s["page_table"], pages = _pages(rng, need, page, B * case["hi"] + (N if "row_start" in s else B * N))
    s.update(_cache(gen, case, pages, case.get("layers")))
    if kind == "attention":
        s["q"] = normal(B, N, case["Hq"], D, dtype=torch.bfloat16, by=2.0)
    elif kind == "append":
        dtype, Hq = DTYPES[case["dtype"]], case["Hq"]
        # one fused projection, as the model's product leaves it: q, k and v are slices of its rows
        qkv = normal(*tokens, (Hq + 2 * Hkv) * D, dtype=dtype)
        heads = qkv.view(*tokens, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = heads[..., :Hq, :], heads[..., Hq:Hq + Hkv, :], heads[..., Hq + Hkv:, :]
        s["q_norm"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(dtype) if case["norm"] else None
        s["k_norm"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(dtype) if case["norm"] else None
        s["cos_sin"], s["pairs"] = None, case["pairs"]
        if case["rot"]:
            inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
            angle = torch.arange(case["hi"] + longest + 1, device=DEV, dtype=torch.float64)[:, None] * inv
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
    else:
        # a walk from the root through random children, as verification leaves it
        path, length = [], []
        for b in range(B):
            par, at, p = _parents(rng, case["tree"], N), 0, []
            while rng.random() < 0.75 and any(par[n] == at for n in range(1, nodes[b])):
                at = rng.choice([n for n in range(1, nodes[b]) if par[n] == at])
                p.append(at)
            path.append(p + [-1] * (N - len(p)))
            length.append(len(p))
        s["out_path"], s["out_len"] = _ints(path), _ints(length)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    kind = s["kind"]
    if own:
        import speculative_decoding_verification_04_gb300 as sv
        scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
        if kind == "attention":
            return sv.spec_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["n_nodes"], parent=s["parent"], **scales)
        if kind == "append":
            q = sv.spec_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], n_new=s.get("n_nodes"), q=s["q"], q_norm=s["q_norm"],
                                  k_norm=s["k_norm"], eps=1e-6, cos_sin=s["cos_sin"], interleaved=s["pairs"], parent=s.get("parent"),
                                  row_start=s.get("row_start"), **scales)
            return [q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
        if kind == "commit":
            new = sv.spec_kv_commit(s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["out_path"], s["out_len"], kv_len_out=torch.empty_like(s["kv_len"]), **scales)
            return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], new]
        return list(sv.spec_kv_read(s["k_cache"], s["v_cache"], s["page_table"], s["start"], s["row_start"], s["rows"], dtype=s["dtype"], **scales))
    if kind == "attention":
        return _plain_attention(s)
    if kind == "append":
        return _plain_append(s)
    if kind == "commit":
        return _plain_commit(s)
    return _plain_read(s)


def _ancestors(parent, B, N):
    """[B, N, N] truth: column m is an ancestor of row n, or n itself."""
    n = torch.arange(N, device=DEV)
    if parent is None:
        return (n[None, :] <= n[:, None]).expand(B, N, N)
    step = ((parent[:, :, None] == n) | (n[:, None] == n)).float()   # a node to itself and its parent
    two = (step @ step > 0).float()
    four = (two @ two > 0).float()
    eight = (four @ four > 0).float()
    sixteen = (eight @ eight > 0).float()
    return sixteen @ sixteen > 0                                      # N <= 32


def _gathered(cache, scale, pages):
    """[B, Hkv, L, D] in 32 bits: each sequence's pages one after the other."""
    x = cache[pages].float()
    x = x if scale is None else x * scale[pages][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    q = s["q"].float()
    B, N, Hq, D = q.shape
    Hkv = s["k_cache"].shape[1]
    pages = s["page_table"].clamp(min=0).long()
    k, v = _gathered(s["k_cache"], s["k_scale"], pages), _gathered(s["v_cache"], s["v_scale"], pages)
    L, ctx = k.shape[2], s["kv_len"].long()[:, None]
    j = torch.arange(L, device=DEV)
    node = j - ctx                                                     # [B, L]: the key's node, negative in the context
    tree = _ancestors(s["parent"], B, N).gather(2, node.clamp(0, N - 1)[:, None, :].expand(B, N, L))
    seen = (node < 0)[:, None] | ((node < s["n_nodes"][:, None])[:, None] & tree)
    seen = seen & (torch.arange(N, device=DEV) < s["n_nodes"][:, None])[:, :, None]
    qh = q.view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = (qh @ k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, N, Hq // Hkv, L)
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp_(min=1e-30))
    valid = (node < s["n_nodes"][:, None])[:, None, :, None]
    o = p.view(B, Hkv, -1, L) @ torch.where(valid, v, torch.zeros((), device=DEV))
    return o.view(B, Hkv, N, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype)


def _normed(x, w, eps=1e-6):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotated(x, cs, pairs):
    """x [T, H, D] rotated by each token's angles: cs [T, rot] holds the cosines, then the sines."""
    if cs is None:
        return x
    h = cs.shape[-1] // 2
    c, z = cs[:, None, :h], cs[:, None, h:]
    if pairs:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        turned = torch.stack([a * c - b * z, b * c + a * z], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        turned = torch.cat([a * c - b * z, b * c + a * z], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _token_places(s, table, first, T):
    """For packed rows: each token's sequence and position."""
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["row_start"].long(), t, right=True) - 1
    return b, first.long()[b] + t - s["row_start"].long()[b]


def _page_slots(s, b, position):
    page = s["page"]
    return s["page_table"][b, position // page].long(), position % page


def _put(cache, scale, at, x):
    """Rows x [T, Hkv, D] into the cache, in its format."""
    page, slot = at
    if scale is None:
        cache[page, :, slot] = x.to(cache.dtype)
        return
    step = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_FLOOR)
    scale[page, :, slot] = step
    cache.view(torch.uint8)[page, :, slot] = (x / step[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    q, k, v = s["q"], s["k"], s["v"]
    if "row_start" in s:
        b, position = _token_places(s, s["page_table"], s["kv_len"], q.shape[0])
        place, source, live = position, slice(None), None
    else:
        B, N = q.shape[:2]
        n = torch.arange(N, device=DEV)
        live = n < s["n_nodes"][:, None]
        depth = _ancestors(s["parent"], B, N).sum(-1) - 1
        b = torch.arange(B, device=DEV)[:, None].expand(B, N).reshape(-1)
        position = (s["kv_len"].long()[:, None] + depth).reshape(-1)
        # a row past the sequence's nodes writes its first node once more
        first = torch.where(live, n, 0)
        place = (s["kv_len"].long()[:, None] + first).reshape(-1)
        source = (torch.arange(B, device=DEV)[:, None] * N + first).reshape(-1)
    cs = None if s["cos_sin"] is None else s["cos_sin"][position]
    flat = lambda x: x.reshape(-1, *x.shape[-2:])  # noqa: E731
    qo = _rotated(_normed(flat(q), s["q_norm"]), cs, s["pairs"])
    ko = _rotated(_normed(flat(k), s["k_norm"]), cs, s["pairs"])
    at = _page_slots(s, b, place)
    _put(s["k_cache"], s["k_scale"], at, ko[source])
    _put(s["v_cache"], s["v_scale"], at, flat(v).float()[source])
    if live is not None:
        qo = qo * live.reshape(-1, 1, 1)
    return [qo.view(q.shape).to(q.dtype), s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _plain_commit(s):
    path, length, ctx = s["out_path"].long(), s["out_len"].long(), s["kv_len"].long()[:, None]
    B, N = path.shape
    i = torch.arange(N, device=DEV)
    kept = i < length[:, None]
    # what is not kept moves the root onto itself
    b = torch.arange(B, device=DEV)[:, None].expand(B, N).reshape(-1)
    src = _page_slots(s, b, (ctx + torch.where(kept, path, 0)).reshape(-1))
    dst = _page_slots(s, b, (ctx + torch.where(kept, i + 1, 0)).reshape(-1))
    as_bytes = lambda x: x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x  # noqa: E731
    kc, vc = as_bytes(s["k_cache"]), as_bytes(s["v_cache"])
    kc[:, dst[0], :, dst[1]] = kc[:, src[0], :, src[1]]
    vc[:, dst[0], :, dst[1]] = vc[:, src[0], :, src[1]]
    if s["k_scale"] is not None:
        s["k_scale"][:, dst[0], :, dst[1]] = s["k_scale"][:, src[0], :, src[1]]
        s["v_scale"][:, dst[0], :, dst[1]] = s["v_scale"][:, src[0], :, src[1]]
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], (s["kv_len"] + 1 + s["out_len"])]


def _plain_read(s):
    b, position = _token_places(s, s["page_table"], s["start"], s["rows"])
    page, slot = _page_slots(s, b, position)

    def rows(cache, scale):
        # an 8-bit float has no gather of its own: its bytes are gathered
        x = cache[page, :, slot].float() if scale is None else cache.view(torch.uint8)[page, :, slot].view(cache.dtype).float() * scale[page, :, slot][..., None]
        return x.to(s["dtype"])

    return [rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])]


# ---------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------
def work(case):
    """Bytes read and written once, and operations, of one pass (lengths as the seed 0 gives them)."""
    kind, D, Hkv = case["kind"], case["D"], case["Hkv"]
    per = (D * 2 if case["fmt"] == "bf16" else D + 4) * Hkv * 2     # a token's keys and values
    rng = random.Random(0)
    if kind == "read":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["N"] * (per + 2 * Hkv * D * size), "flops": case["N"] * 2 * Hkv * D}
    ctx = _lengths(rng, case)
    if kind == "append":
        size, Hq = 2 if case["dtype"] == "bf16" else 4, case["Hq"]
        tokens = case["N"] if case["packed"] else case["B"] * case["N"]
        return {"bytes": tokens * (size * D * (2 * Hq + 2 * Hkv) + per + 4 * case["rot"]), "flops": tokens * D * (Hq + Hkv) * 8}
    if kind == "commit":
        kept = max(1, case["B"] * min(2, case["N"] - 1))           # about two nodes a walk
        return {"bytes": kept * case["layers"] * per * 2 + case["B"] * 12, "flops": 0}
    keys = sum(ctx) + case["B"] * case["N"]
    return {"bytes": keys * per + 4 * case["B"] * case["N"] * case["Hq"] * D, "flops": 4 * keys * case["N"] * case["Hq"] * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "commit": _exact_commit, "read": _exact_read}[s["kind"]](s)


def _host(t):
    return t.cpu().tolist()


def _spots(s, row, positions):
    """Page and slot of each position of one sequence (its page table row on the host)."""
    page = s["page"]
    return (torch.tensor([row[p // page] for p in positions], device=DEV, dtype=torch.long), torch.tensor([p % page for p in positions], device=DEV, dtype=torch.long))


def _value64(cache, scale, spots):
    page, slot = spots
    raw = cache if scale is None else cache.view(torch.uint8)
    x = raw[page, :, slot]
    return x.double() if scale is None else x.view(cache.dtype).double() * scale[page, :, slot].double()[..., None]


def _exact_attention(s):
    q = s["q"].double()
    B, N, Hq, D = q.shape
    out = torch.zeros_like(q)
    Hkv = s["k_cache"].shape[1]
    ctx, nodes, table = _host(s["kv_len"]), _host(s["n_nodes"]), _host(s["page_table"])
    parents = None if s["parent"] is None else _host(s["parent"])
    for b in range(B):
        n = nodes[b]
        if n == 0:
            continue
        at = _spots(s, table[b], range(ctx[b] + n))
        k, v = _value64(s["k_cache"], s["k_scale"], at), _value64(s["v_cache"], s["v_scale"], at)
        hidden = torch.ones(n, ctx[b] + n, dtype=torch.bool)
        hidden[:, :ctx[b]] = False
        for i in range(n):
            m = i
            while m >= 0:
                hidden[i, ctx[b] + m] = False
                m = (m - 1 if parents is None else parents[b][m]) if m > 0 else -1
        hidden = hidden.to(DEV)
        for h in range(Hq):
            x = (q[b, :n, h] @ k[:, h * Hkv // Hq].T) / math.sqrt(D)
            out[b, :n, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[:, h * Hkv // Hq]
    return out


def _exact_rows(x, w, table, position, pairs):
    """Norm and rotation of rows x [T, H, D] in 64 bits, pair by pair."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
    if table is None:
        return x
    half = table.shape[1] // 2
    out = x.clone()
    at = torch.tensor(position, device=DEV)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        c, z = table[at, i].double()[:, None], table[at, half + i].double()[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * z
        out[..., b] = x[..., b] * c + x[..., a] * z
    return out


def _nearest_e4m3(x):
    """The nearest of the values an e4m3 can hold, ties to the even one: steps of 2^-9 below 2^-6, of an eighth of the power of two above."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6)
    step = torch.exp2(exponent - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(s):
    q, k, v = s["q"], s["k"], s["v"]
    packed = "row_start" in s
    D = q.shape[-1]
    ctx, table = _host(s["kv_len"]), _host(s["page_table"])
    qf, kf, vf = (x.reshape(-1, x.shape[-2], D) for x in (q, k, v))
    parents = None if packed or s["parent"] is None else _host(s["parent"])
    rows, position, place = [], [], []
    bounds = _host(s["row_start"]) if packed else [b * q.shape[1] for b in range(len(ctx) + 1)]
    nodes = [bounds[b + 1] - bounds[b] for b in range(len(ctx))] if packed else _host(s["n_nodes"])
    for b, c in enumerate(ctx):
        depth = []
        for i in range(nodes[b]):
            depth.append(i if parents is None else (depth[parents[b][i]] + 1 if i else 0))
            rows.append(bounds[b] + i)
            position.append(c + depth[i])
            place.append((table[b][(c + i) // s["page"]], (c + i) % s["page"]))
    rows = torch.tensor(rows, device=DEV)
    qo = torch.zeros(qf.shape, dtype=torch.float64, device=DEV)
    qo[rows] = _exact_rows(qf[rows], s["q_norm"], s["cos_sin"], position, s["pairs"])
    page, slot = (torch.tensor(x, device=DEV) for x in zip(*place))
    out = [qo.view(q.shape)]
    scales = []
    for name, x in (("k", _exact_rows(kf[rows], s["k_norm"], s["cos_sin"], position, s["pairs"])), ("v", vf[rows].double())):
        cache = s[name + "_cache"].double()
        if s[name + "_scale"] is None:
            cache[page, :, slot] = x
            scales.append(None)
        else:
            scale = s[name + "_scale"].double()
            step = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_FLOOR)
            cache[page, :, slot] = _nearest_e4m3(x / step[..., None])
            scale[page, :, slot] = step
            scales.append(scale)
        out.append(cache)
    return out + scales


def _exact_commit(s):
    ctx, table, length, path = _host(s["kv_len"]), _host(s["page_table"]), _host(s["out_len"]), _host(s["out_path"])
    src, dst = [], []
    for b, c in enumerate(ctx):
        for i in range(length[b]):
            for to, p in ((src, c + path[b][i]), (dst, c + 1 + i)):
                to.append((table[b][p // s["page"]], p % s["page"]))
    out = []
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if s[name] is None:
            out.append(None)
            continue
        x = s[name].float()                                            # copies: 32 bits hold them exactly
        if src:
            (sp, ss), (dp, ds) = ((torch.tensor(y, device=DEV) for y in zip(*x_)) for x_ in (src, dst))
            x[:, dp, :, ds] = x[:, sp, :, ss]
        out.append(x)
    return out + [None]


def _exact_read(s):
    start, bounds, table = _host(s["start"]), _host(s["row_start"]), _host(s["page_table"])
    parts = {"k": [], "v": []}
    for b, a in enumerate(start):
        at = _spots(s, table[b], range(a, a + bounds[b + 1] - bounds[b]))
        for n in parts:
            parts[n].append(_value64(s[n + "_cache"], s[n + "_scale"], at))
    return [torch.cat(parts["k"]), torch.cat(parts["v"])]
