"""Decoding with token trees, end to end on the library's operators.

Every round, for each sequence: a tree of tokens is drafted behind the last
committed token; spec_kv_append writes the nodes' keys and values into the
paged cache (norms, rotation and, for an 8-bit cache, quantisation in the same
pass); spec_tree_attention attends from every node to the context and its
ancestors; spec_verify_tree keeps a path; spec_kv_commit moves that path's
entries behind the root and advances the lengths on the device.

The model is a toy: one attention layer with random weights on top of a bigram
table, and the bigram table alone as the draft.  The calls are those of a real
one.

  python examples/tree_decode.py [--rounds 8] [--cache e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_04_gb300 as sv  # noqa: E402
import workloads as W  # noqa: E402


class Model:
    """One layer: embedding, q/k/v projection, head norms and rotation, attention, output."""

    def __init__(self, dev, vocab=1003, width=256, n_heads=8, n_kv_heads=2, head_dim=64, positions=512, seed=0):
        gen = torch.Generator(device=dev).manual_seed(seed)

        def weights(*shape, by):
            return (torch.randn(*shape, generator=gen, device=dev) * by).to(torch.bfloat16)

        self.heads, self.kv_heads, self.head_dim, self.vocab = n_heads, n_kv_heads, head_dim, vocab
        self.embed = weights(vocab, width, by=1.0)
        self.qkv = weights(width, (n_heads + 2 * n_kv_heads) * head_dim, by=width ** -0.5)
        self.out = weights(n_heads * head_dim, vocab, by=2.0 * (n_heads * head_dim) ** -0.5)
        self.q_norm, self.k_norm = (1 + weights(head_dim, by=0.1) for _ in range(2))
        self.draft = weights(vocab, vocab, by=2.0)
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device=dev, dtype=torch.float64) / head_dim)
        angle = torch.arange(positions, device=dev, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], -1).float()

    def project(self, tokens):
        """q, k and v of tokens [...]: slices of one product."""
        x = (self.embed[tokens] @ self.qkv).view(*tokens.shape, -1, self.head_dim)
        return x[..., :self.heads, :], x[..., self.heads:-self.kv_heads, :], x[..., -self.kv_heads:, :]


class Cache:
    """A paged cache of one layer with a fixed page table."""

    def __init__(self, model, B, positions, fmt, dev, page=16):
        pages = -(-positions // page)
        shape = (B * pages, model.kv_heads, page, model.head_dim)
        dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
        self.k, self.v = (torch.empty(shape, dtype=dtype, device=dev) for _ in range(2))
        self.scales = {}
        if fmt != "bf16":
            self.scales = {n: torch.empty(shape[:-1], device=dev) for n in ("k_scale", "v_scale")}
        self.table = torch.randperm(B * pages, device=dev).to(torch.int32).view(B, pages)


def run(rounds=8, B=6, fmt="bf16", dev="cuda:0", seed=0):
    """Decode; returns (model, cache, kv_len, histories): each sequence's committed tokens."""
    dev = torch.device(dev)
    torch.cuda.set_device(dev)
    torch.manual_seed(seed)
    model = Model(dev, seed=seed)
    tree = W.full_tree(2, 3)
    N = len(tree)
    cache = Cache(model, B, positions=rounds * N + N, fmt=fmt, dev=dev)
    parent = torch.from_numpy(tree).to(dev).expand(B, N).contiguous()
    nodes = torch.full((B,), N, dtype=torch.int32, device=dev)
    temperature = torch.full((B,), 0.8, device=dev)
    kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
    root = torch.randint(model.vocab, (B,), device=dev)
    errors = torch.zeros(1, dtype=torch.int32, device=dev)
    histories = [[] for _ in range(B)]
    for _ in range(rounds):
        # draft: children drawn from the bigram row of their parent
        tokens = torch.empty(B, N, dtype=torch.int64, device=dev)
        tokens[:, 0] = root
        for n in range(1, N):
            p = torch.softmax(model.draft[tokens[:, tree[n]]].float() / 0.8, -1)
            tokens[:, n] = torch.multinomial(p, 1)[:, 0]
        draft = model.draft[tokens]
        # target: one pass over all nodes
        q, k, v = model.project(tokens)
        q = sv.spec_kv_append(k, v, cache.k, cache.v, cache.table, kv_len, q=q, q_norm=model.q_norm, k_norm=model.k_norm,
                              cos_sin=model.cos_sin, parent=parent, errors=errors, **cache.scales)
        o = sv.spec_tree_attention(q, cache.k, cache.v, cache.table, kv_len, parent=parent, errors=errors, **cache.scales)
        target = draft + o.flatten(2) @ model.out
        # verify and commit
        out, path, length = sv.spec_verify_tree(target, draft, tokens.int(), parent, torch.rand(B, N, device=dev) * 0.999999,
                                                temperature, nodes)
        sv.spec_kv_commit(cache.k, cache.v, cache.table, kv_len, path, length, errors=errors, **cache.scales)
        root_now, out, length = tokens[:, 0].tolist(), out.tolist(), length.tolist()
        for b in range(B):
            histories[b] += [root_now[b]] + out[b][:length[b]]
        root = torch.tensor([out[b][length[b]] for b in range(B)], device=dev)
    if errors.item():
        raise RuntimeError(f"device errors {errors.item()}")
    return model, cache, kv_len, histories


def check(model, cache, kv_len, histories):
    """The cache holds exactly the committed tokens' keys and values: read it
    back and compare with a plain computation.  Returns the largest error
    relative to the largest entry."""
    dev = kv_len.device
    counts = [len(h) for h in histories]
    assert kv_len.tolist() == counts
    bounds = torch.tensor([sum(counts[:b]) for b in range(len(counts) + 1)], dtype=torch.int32, device=dev)
    k, v = sv.spec_kv_read(cache.k, cache.v, cache.table, torch.zeros_like(kv_len), bounds, sum(counts), dtype=torch.float32, **cache.scales)
    tokens = torch.tensor(sum(histories, []), device=dev)
    position = torch.cat([torch.arange(c, device=dev) for c in counts])
    _, rk, rv = (x.float() for x in model.project(tokens))
    rk = rk * torch.rsqrt((rk * rk).mean(-1, keepdim=True) + 1e-6) * model.k_norm.float()
    half = model.head_dim // 2
    c, s = (model.cos_sin[position][:, None, i * half:(i + 1) * half] for i in (0, 1))
    rk = torch.cat([rk[..., :half] * c - rk[..., half:] * s, rk[..., half:] * c + rk[..., :half] * s], -1)
    return max(((x - y).abs().max() / y.abs().max()).item() for x, y in ((k, rk), (v, rv)))


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    state = run(a.rounds, fmt=a.cache)
    per = sum(len(h) for h in state[3]) / (a.rounds * len(state[3]))
    print(f"{a.rounds} rounds, {per:.2f} tokens a round and sequence, cache error {check(*state):.4f}")
