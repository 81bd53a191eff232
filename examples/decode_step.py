"""One attention layer of a speculative decoding step under adapters.

Every token carries its own adapter; the base projections hold 4-bit weights;
keys and values live in a paged cache; each sequence drafts a tree of tokens, of
which one path is accepted.  A step of the layer is

    qkv   = x Wqkv                     lora_q4_matmul
    qkv  += (x A_l) B_l                lora_shrink_expand: q, k and v are its slices
    cache <- k, v                      lora_pages_resize, lora_pages_append
    o     = attention(q, cache)        lora_tree_attention
    y     = o Wo                       lora_q4_matmul
    y    += (o A_l) B_l                lora_shrink_expand
    cache <- accepted path             lora_pages_accept, lora_pages_resize

Run it on an MI355X:  python examples/decode_step.py
"""
import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lora_serving_build_amd as lsb  # noqa: E402


def quantise(w: torch.Tensor, group: int):
    """Codes, scales and zeros of a [n][k] weight, rounded to 4 bits by groups."""
    n, k = w.shape
    g = w.float().view(n, k // group, group)
    low, high = g.amin(-1), g.amax(-1)
    scale = ((high - low) / 15).clamp(min=1e-8).to(w.dtype)
    zero = (-low / scale.float()).round().clamp(0, 15)
    q = (g / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8).view(n, k)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), scale, zero.to(torch.uint8)


class Layer:
    """An attention layer's weights: 4-bit base projections and its adapters."""

    def __init__(self, hidden, heads, kv_heads, dim, adapters, rank, group=128, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s: torch.empty(*s, device="cuda").normal_(0, 1 / math.sqrt(s[-1]), generator=g).to(dtype)  # noqa: E731
        self.heads, self.kv_heads, self.dim, self.dtype, self.rank = heads, kv_heads, dim, dtype, rank
        self.widths = [heads * dim, kv_heads * dim, kv_heads * dim]
        self.raw_qkv = quantise(rnd(sum(self.widths), hidden), group)
        self.raw_o = quantise(rnd(hidden, heads * dim), group)
        self.w_qkv = lsb.lora_q4_pack(*self.raw_qkv, hidden, group)
        self.w_o = lsb.lora_q4_pack(*self.raw_o, heads * dim, group)
        self.a_qkv, self.a_o = rnd(adapters, rank, hidden), rnd(adapters, rank, heads * dim)
        self.b_qkv = [rnd(adapters, n, rank) for n in self.widths]
        self.b_o = [rnd(adapters, hidden, rank)]
        self.offsets = [0, heads * dim, (heads + kv_heads) * dim]

    def project(self, x, weight, a, bs, offsets, seg):
        """x W of the base weight plus each token's own adapter."""
        y = torch.empty(x.shape[0], weight.n, dtype=self.dtype, device=x.device)
        lsb.lora_q4_matmul(x, weight, y)
        v = torch.empty(x.shape[0], self.rank, dtype=torch.float32, device=x.device)
        lsb.lora_shrink_expand(x, a, bs, offsets, seg, v, y, add_inputs=True)
        return y

    def step(self, x, seg, cache, layer, seqs, start, table, ctx_len, mask):
        """The layer's output for the drafted tokens x, whose keys and values
        are left in the cache behind each sequence's context."""
        T, h, kv, d = x.shape[0], self.heads, self.kv_heads, self.dim
        qkv = self.project(x, self.w_qkv, self.a_qkv, self.b_qkv, self.offsets, seg)
        q = qkv[:, :h * d].view(T, h, d)
        k = qkv[:, h * d:(h + kv) * d].view(T, kv, d)
        v = qkv[:, (h + kv) * d:].view(T, kv, d)
        lsb.lora_pages_append(cache, layer, k, v, seqs, start)
        o = torch.empty(T, h, d, dtype=self.dtype, device=x.device)
        lsb.lora_tree_attention(q, *cache.layer(layer), table, ctx_len, start, o, 1 / math.sqrt(d), mask=mask)
        return self.project(o.view(T, h * d), self.w_o, self.a_o, self.b_o, [0], seg), o


def new_cache(layers, pages, page_size, kv_heads, dim, seqs, max_pages, dtype=torch.bfloat16):
    i32 = dict(dtype=torch.int32, device="cuda")
    return lsb.PageCache(torch.zeros(2 * layers, pages, page_size, kv_heads, dim, dtype=dtype, device="cuda"),
                         torch.zeros(pages, **i32), torch.full((seqs, max_pages), -1, **i32), torch.zeros(seqs, **i32))


def draft_trees(rs, counts):
    """A parent (-1: the context) for each drafted node, and the mask rows of
    one word: a node sees itself and its ancestors."""
    parents, rows = [], []
    for n in counts:
        first = len(rows)
        for i in range(n):
            p = int(rs.randint(max(0, i - 4), i)) if i else -1
            rows.append((rows[first + p] if p >= 0 else 0) | (1 << i))
            parents.append(p)
    return parents, torch.tensor(np.array(rows, np.uint64).view(np.int64)[:, None], device="cuda")


def path_to(parents, first, node):
    path = []
    while node >= 0:
        path.append(node)
        node = parents[first + node]
    return path[::-1]


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


def run(steps=3, seed=0, verbose=True, inspect=None):
    """A few steps over three sequences that share a prompt.  inspect, if given,
    is called with every step's tensors before the path is accepted."""
    rs = np.random.RandomState(seed)
    hidden, heads, kv, dim, adapters, rank, page = 1024, 8, 2, 128, 4, 16, 16
    layer = Layer(hidden, heads, kv, dim, adapters, rank, seed=seed)
    cache = new_cache(1, 64, page, kv, dim, seqs=4, max_pages=16)
    prompt = 37
    rnd = lambda *s: torch.from_numpy(rs.standard_normal(s).astype(np.float32)).cuda().to(layer.dtype)  # noqa: E731

    # The prompt's keys and values, and two more sequences that start from it:
    # they share its full pages and own a copy of the last one.
    lsb.lora_pages_resize(cache, ints([0]), extra=ints([prompt]))
    lsb.lora_pages_append(cache, 0, rnd(prompt, kv, dim), rnd(prompt, kv, dim), ints([0]), ints([0, prompt]))
    lsb.lora_pages_resize(cache, ints([0]), lens=ints([prompt]))
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    lsb.lora_pages_fork(cache, ints([0, 0]), ints([1, 2]), status)
    assert status.tolist() == [lsb.PAGES_OK] * 2

    seqs, ids = ints([0, 1, 2]), [3, 0, -1]  # the third sequence has no adapter
    for step in range(steps):
        counts = [5, 9, 1 + step]
        start = np.concatenate([[0], np.cumsum(counts)])
        parents, mask = draft_trees(rs, counts)
        seg = lsb.lora_build_segments(ints(np.repeat(ids, counts)), adapters)
        x = rnd(sum(counts), hidden)
        drafted = ints(counts)
        lsb.lora_pages_resize(cache, seqs, extra=drafted)
        table, ctx = cache.table[:3], cache.seq_len[:3]
        y, o = layer.step(x, seg, cache, 0, seqs, ints(start), table, ctx, mask)
        if inspect is not None:
            inspect(layer=layer, cache=cache, x=x, y=y, o=o, ids=np.repeat(ids, counts), start=start, parents=parents)
        # Verification would pick each sequence's path; here a random node's.
        paths = [path_to(parents, s, int(rs.randint(n))) for s, n in zip(start, counts)]
        accepted = ints([len(p) for p in paths])
        new_len = torch.empty(3, dtype=torch.int32, device="cuda")
        width = max(len(p) for p in paths)
        lsb.lora_pages_accept(cache, seqs, drafted, ints([p + [0] * (width - len(p)) for p in paths]), accepted, new_len)
        lsb.lora_pages_resize(cache, seqs, lens=new_len)
        if verbose:
            print(f"step {step}: drafted {counts}, accepted {accepted.tolist()}, cached {cache.seq_len.tolist()[:3]}, "
                  f"pages in use {int((cache.refs != 0).sum())}")
    lsb.lora_pages_free(cache, seqs)
    if verbose:
        print(f"freed: pages in use {int((cache.refs != 0).sum())}")
    return cache


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    run(a.steps, a.seed)
