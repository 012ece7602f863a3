"""Plain 64-bit definitions of the cache operators, and their inputs, for the
tests.  A sequence at a time, a head at a time, on whatever device the tensors
are on; nothing here uses the library."""
from __future__ import annotations

import math
import random

import torch

E4M3 = torch.float8_e4m3fn


def parents_of(kind, N, rng):
    if kind == "binary":
        return [-1] + [(n - 1) // 2 for n in range(1, N)]
    if kind == "star":
        return [-1] + [0] * (N - 1)
    if kind == "random":
        return [-1] + [rng.randrange(0, n) for n in range(1, N)]
    return [-1] + list(range(N - 1))


def ancestors(parent, n):
    """Node n and its ancestors."""
    out = [n]
    while n > 0:
        n = parent[n]
        out.append(n)
    return out


class Cache:
    """A paged cache with shuffled pages.  What no sequence has written is NaN
    (and so are the scales there): using it anywhere shows."""

    def __init__(self, lengths, Hkv, D, page, fmt, dev, seed=0, layers=None, spare=3, fill=True):
        rng = random.Random(seed)
        gen = torch.Generator(device=dev).manual_seed(seed)
        count = [-(-n // page) for n in lengths]
        self.num_pages = sum(count) + spare
        ids = list(range(self.num_pages))
        rng.shuffle(ids)
        width, at, rows = max(1, max(count)), 0, []
        for c in count:
            rows.append(ids[at:at + c] + [-1] * (width - c))
            at += c
        self.page, self.Hkv, self.D, self.fmt, self.layers = page, Hkv, D, fmt, layers
        self.pages = rows
        self.table = torch.tensor(rows, dtype=torch.int32, device=dev)
        lead = [] if layers is None else [layers]
        shape = lead + [self.num_pages, Hkv, page, D]
        self.k_scale = self.v_scale = None
        made = []
        for _ in range(2):
            if fmt == "bf16":
                made.append(torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16))
            else:
                made.append((torch.randn(shape, generator=gen, device=dev) * 100).clamp(-448, 448).to(E4M3))
        self.k, self.v = made
        if fmt != "bf16":
            self.k_scale = torch.rand(shape[:-1], generator=gen, device=dev) * 0.01 + 0.005
            self.v_scale = torch.rand(shape[:-1], generator=gen, device=dev) * 0.01 + 0.005
        if fill:
            used = torch.zeros(self.num_pages, page, dtype=torch.bool, device=dev)
            for b, n in enumerate(lengths):
                for i, p in enumerate(rows[b]):
                    if p >= 0:
                        used[p, :min(page, n - i * page)] = True
            self.poison(~used)

    def poison(self, where):
        """NaN at every head of the (page, slot) pairs where `where` is true."""
        w = where[:, None, :]
        for t, bad in ((self.k, 0x7f), (self.v, 0x7f)):
            if self.fmt == "bf16":
                t.masked_fill_(w[..., None], float("nan"))
            else:
                t.view(torch.uint8).masked_fill_(w[..., None], bad)
        if self.fmt != "bf16":
            self.k_scale.masked_fill_(w, float("nan"))
            self.v_scale.masked_fill_(w, float("nan"))

    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)

    def at(self, b, positions):
        dev = self.k.device
        return (torch.tensor([self.pages[b][p // self.page] for p in positions], dtype=torch.long, device=dev),
                torch.tensor([p % self.page for p in positions], dtype=torch.long, device=dev))

    def rows64(self, which, b, positions, layer=None):
        """[len(positions), Hkv, D] in 64 bits."""
        t, s = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        if layer is not None:
            t, s = t[layer], None if s is None else s[layer]
        page, slot = self.at(b, positions)
        if s is None:
            return t[page, :, slot].double()
        return t.view(torch.uint8)[page, :, slot].view(E4M3).double() * s[page, :, slot].double()[..., None]


def attention64(q, cache, kv_len, n_nodes, parents, scale):
    """(out, bound): the definition in 64 bits and, per element, sum_j p_j |v_j|
    and the largest sum_d |q_d k_d| of a key (both set the rounding's size)."""
    B, N, Hq, D = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    spread, big = torch.zeros_like(out), torch.zeros_like(out)
    G = Hq // cache.Hkv
    for b in range(B):
        if n_nodes[b] == 0:
            continue
        L = kv_len[b] + n_nodes[b]
        k, v = cache.rows64("k", b, range(L)), cache.rows64("v", b, range(L))
        seen = torch.zeros(n_nodes[b], L, dtype=torch.bool)
        seen[:, :kv_len[b]] = True
        for n in range(n_nodes[b]):
            for m in ancestors(parents[b], n):
                seen[n, kv_len[b] + m] = True
        seen = seen.to(q.device)
        for h in range(Hq):
            x = q[b, :n_nodes[b], h].double()
            s = (x @ k[:, h // G].T * scale).masked_fill(~seen, -math.inf)
            p = torch.softmax(s, -1)
            out[b, :n_nodes[b], h] = p @ v[:, h // G]
            spread[b, :n_nodes[b], h] = p @ v[:, h // G].abs()
            worst = (x.abs() @ k[:, h // G].abs().T * abs(scale)).masked_fill(~seen, 0.0).amax(-1)
            big[b, :n_nodes[b], h] = worst[:, None]
    return out, spread, big


def attention_bound(out, spread, big, D):
    """What bf16 weights, a bf16 result and fp32 sums may differ by: half a
    bf16 unit (2^-9) of the result and of every weight, doubled; the score's
    rounding ((D + 8) 2^-24 of its magnitudes) moves a weight by as much, both
    in the numerator and in the denominator; 2^-16 covers the exponential and
    the sums of up to 2^17 positive terms in blocks."""
    return 2.0 ** -8 * (out.abs() + spread) + (2.0 * (D + 8) * 2.0 ** -24 * big + 2.0 ** -16) * spread + 1e-30


def rotated64(x, w, table, position, pairs, eps):
    """Norm and rotation of rows x [T, H, D] in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if table is None:
        return x
    half = table.shape[1] // 2
    out = x.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        c, s = table[position, i].double()[:, None], table[position, half + i].double()[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out
