"""Tree attention over a paged cache (lora_tree_attention) against the
definition in 64 bits.

Tolerance of o: half a step of its type; the weights' rounding to the cache's
type (half a step of each term w v); the scores' fp32 sums, dim roundings of at
most 2^-23 of the sum of |q k| that act on a weight as a factor (their share of
both sums), and the fp32 exponential and sums over the positions."""
import math

import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """Random sequences in a shuffled paged cache.  Slots that hold no token are
    NaN, as are the pages that no sequence owns."""

    def __init__(self, nodes, ctx, heads, kv, dim, page, dtype, mask="tree", head_major=False, seed=0, words=None,
                 spare=3):
        rs = np.random.RandomState(seed)
        self.nodes, self.ctx, self.heads, self.kv, self.dim, self.page, self.dtype = nodes, ctx, heads, kv, dim, page, dtype
        B, T = len(nodes), sum(nodes)
        held = [-(-(a + b) // page) for a, b in zip(ctx, nodes)]
        num = sum(held) + spare
        order = rs.permutation(num)
        self.table = np.full((B, max(max(held), 1) + 1), -1, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order[at:at + h]
            at += h
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s: torch.empty(*s, device="cuda").normal_(generator=g).to(DT[dtype])  # noqa: E731
        self.q = rnd(T, heads, dim)
        self.k = torch.full((num, page, kv, dim), float("nan"), dtype=DT[dtype], device="cuda")
        self.v = self.k.clone()
        for b in range(B):
            for p in range(held[b]):
                n = min(page, ctx[b] + nodes[b] - p * page)
                self.k[self.table[b, p], :n] = rnd(n, kv, dim)
                self.v[self.table[b, p], :n] = rnd(n, kv, dim)
        if head_major:
            self.k, self.v = (t.transpose(1, 2).contiguous() for t in (self.k, self.v))
        self.head_major = head_major
        # seen[b][i, j]: node i sees node j
        self.seen = []
        for n in nodes:
            m = np.zeros((n, n), bool)
            for i in range(n):
                if mask == "tree":
                    if i:
                        m[i] = m[rs.randint(max(0, i - 5), i)]
                    m[i, i] = True
                elif mask == "chain":
                    m[i, :i + 1] = True
                elif mask == "random":
                    m[i] = rs.rand(n) < 0.4
                # "none": sees no node
            self.seen.append(m)
        self.words = words or max(1, -(-max(nodes + [1]) // 64))
        bits = np.zeros((T, self.words), np.uint64)
        row = 0
        for n, m in zip(nodes, self.seen):
            for i in range(n):
                for j in range(n):
                    if m[i, j] and j < 64 * self.words:
                        bits[row, j // 64] |= np.uint64(1) << np.uint64(j % 64)
                for j in range(n, 64 * self.words):  # bits beyond the nodes mean nothing
                    if rs.rand() < 0.5:
                        bits[row, j // 64] |= np.uint64(1) << np.uint64(j % 64)
                row += 1
        self.mask = None if mask == "chain" else torch.from_numpy(bits.view(np.int64)).cuda()
        self.scale = 1.0 / math.sqrt(dim)

    def ints(self, v):
        return torch.tensor(np.asarray(v, np.int32), device="cuda")

    def run(self, out=None, lse=None, **change):
        a = dict(q=self.q, k=self.k, v=self.v, table=torch.from_numpy(self.table).cuda(), ctx=self.ints(self.ctx),
                 start=self.ints(np.concatenate([[0], np.cumsum(self.nodes)])), mask=self.mask)
        a.update(change)
        if out is None:
            out = torch.full(a["q"].shape, float("nan"), dtype=a["q"].dtype, device="cuda")
        lsb.lora_tree_attention(a["q"], a["k"], a["v"], a["table"], a["ctx"], a["start"], out, self.scale,
                                mask=a["mask"], lse=lse, head_major=self.head_major)
        return out

    def expect(self, pages=None):
        """(o, lse, magnitude of the terms, spread of the scores) in 64 bits.
        pages: number of page ids that are in range."""
        T = sum(self.nodes)
        o, mag = np.zeros((T, self.heads, self.dim)), np.zeros((T, self.heads, self.dim))
        lse, spread = np.full((T, self.heads), -np.inf), np.zeros((T, self.heads))
        G, row = self.heads // self.kv, 0
        k, v = ((t.transpose(1, 2) if self.head_major else t).double().cpu().numpy() for t in (self.k, self.v))
        q = self.q.double().cpu().numpy()
        num = k.shape[0]
        for b, n in enumerate(self.nodes):
            length = self.ctx[b] + n
            pos = np.arange(length)
            ids = self.table[b, pos // self.page] if length else np.zeros(0, int)
            there = (ids >= 0) & (ids < num)
            kk, vv = (np.where(there[:, None, None], t[np.where(there, ids, 0), pos % self.page], 0.0) for t in (k, v))
            for i in range(n):
                sees = there.copy()
                sees[self.ctx[b]:] &= self.seen[b][i]
                sees[self.ctx[b] + 64 * self.words:] = sees[self.ctx[b] + 64 * self.words:] & (self.mask is None)
                for h in range(self.heads):
                    if sees.any():
                        z = kk[sees, h // G] @ q[row, h] * self.scale
                        spread[row, h] = np.max(np.abs(kk[sees, h // G]) @ np.abs(q[row, h])) * self.scale
                        w = np.exp(z - z.max())
                        lse[row, h] = z.max() + np.log(w.sum())
                        w /= w.sum()
                        o[row, h] = w @ vv[sees, h // G]
                        mag[row, h] = w @ np.abs(vv[sees, h // G])
                row += 1
        return o, lse, mag, spread

    def check(self, got, lse=None, rows=slice(None)):
        o, want_lse, mag, spread = self.expect()
        longest = max(a + b for a, b in zip(self.ctx, self.nodes))
        half = torch.finfo(DT[self.dtype]).eps / 2
        score = spread * (self.dim + 8) * 2.0 ** -23
        sums = (64 + longest / 128) * 2.0 ** -23
        tol = np.abs(o) * half * 1.001 + mag * (half + 2 * score[..., None] + 2 * sums + 2.0 ** -20) + 2.0 ** -24
        worst = np.max((np.abs(got.double().cpu().numpy() - o) / tol)[rows])
        assert worst <= 1, worst
        if lse is not None:
            g = lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(g), np.isneginf(want_lse))
            fine = np.isfinite(want_lse)
            off = np.abs(g[fine] - want_lse[fine]) - (score + sums + 2.0 ** -18 + np.abs(np.where(fine, want_lse, 0)) * 2.0 ** -22)[fine]
            assert off.size == 0 or off.max() <= 0, off.max()


CASES = [
    # nodes, ctx, heads, kv_heads, dim, page, dtype, mask, head_major
    ([1], [0], 1, 1, 64, 16, "f16", "chain", False),
    ([1], [1], 4, 4, 128, 16, "bf16", "tree", False),
    ([1], [509], 32, 8, 128, 16, "f16", "tree", False),
    ([1, 1, 1], [31, 32, 33], 8, 2, 64, 16, "bf16", "chain", True),
    ([3, 0, 5, 1], [17, 40, 0, 127], 6, 2, 80, 24, "f16", "tree", False),
    ([16], [128], 8, 8, 128, 32, "bf16", "tree", False),
    ([17, 2], [100, 300], 12, 4, 96, 16, "f16", "random", True),
    ([8, 24, 9], [1000, 3, 250], 16, 2, 128, 64, "bf16", "tree", False),
    ([64], [65], 4, 1, 64, 1, "f16", "tree", False),
    ([70, 130], [200, 5], 4, 2, 128, 16, "bf16", "random", False),
    ([5, 6], [400, 77], 8, 1, 256, 16, "f16", "tree", False),
    ([40], [90], 6, 2, 200, 7, "bf16", "chain", True),
    ([2, 3], [5000, 40], 8, 2, 128, 16, "f16", "tree", False),
    ([4], [20000], 16, 1, 64, 100, "bf16", "tree", False),
    ([1] * 70, list(range(0, 700, 10)), 4, 2, 128, 16, "f16", "tree", False),
    ([33], [700], 24, 8, 8, 16, "bf16", "tree", False),
    ([2], [33000], 4, 2, 256, 32, "bf16", "tree", False),
    ([4, 3], [10, 64], 8, 2, 128, 16, "f16", "none", False),
    ([2, 1], [0, 0], 4, 2, 64, 16, "bf16", "none", True),
    # many rows over lines that are cut
    ([40, 24], [3000, 500], 64, 8, 128, 16, "bf16", "tree", False),
    ([20, 20], [1700, 90], 64, 8, 64, 16, "f16", "random", False),
    ([1] * 300, list(range(0, 1500, 5)), 8, 8, 64, 16, "f16", "tree", False),
    ([9] * 16, list(range(100, 1700, 100)), 16, 2, 256, 16, "bf16", "tree", False),
    ([100, 90], [1500, 40], 16, 4, 80, 24, "f16", "tree", True),
]


@pytest.mark.parametrize("nodes,ctx,heads,kv,dim,page,dtype,mask,head_major", CASES)
def test_attention(nodes, ctx, heads, kv, dim, page, dtype, mask, head_major):
    b = Batch(nodes, ctx, heads, kv, dim, page, dtype, mask, head_major, seed=sum(nodes) + dim)
    lse = torch.full((sum(nodes), heads), 7.0, device="cuda")
    out = b.run(lse=lse)
    b.check(out, lse)
    assert torch.equal(out, b.run())                   # same inputs, same bits


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_strides(dtype):
    """Rows of a wider projection as q, out and the cache."""
    b = Batch([3, 20], [50, 7], 8, 2, 64, 16, dtype, seed=3)
    T = 23
    wide = torch.full((T, 12 * 64), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, 64:9 * 64] = b.q.view(T, -1)
    q = wide.view(T, 12, 64)[:, 1:9]
    out = torch.full((T, 10, 72), -5.0, dtype=DT[dtype], device="cuda")
    kv = torch.stack((b.k, b.v), 2).contiguous()       # k and v of a slot side by side
    lsb.lora_tree_attention(q, kv[:, :, 0], kv[:, :, 1], torch.from_numpy(b.table).cuda(), b.ints(b.ctx),
                            b.ints([0, 3, 23]), out[:, 1:9, :64], b.scale, mask=b.mask)
    b.check(out[:, 1:9, :64])
    assert bool((out[:, 0] == -5).all()) and bool((out[:, 9] == -5).all()) and bool((out[:, :, 64:] == -5).all())


def test_pages_that_are_not_there():
    """Positions whose page id is out of range, or beyond the table, are not
    seen; lengths out of range are cut."""
    b = Batch([2, 4, 1], [100, 64, 40], 4, 2, 128, 16, "bf16", seed=4)
    b.table[0, 2] = -1
    b.table[1, 0] = 10 ** 6
    b.table[1, 4] = -2 ** 31
    b.table[2, :] = -1
    b.check(b.run())
    # A context longer than the table holds, a negative one.
    c = Batch([1, 1], [47, 0], 4, 2, 64, 16, "f16", mask="none", seed=5)
    table = torch.from_numpy(c.table[:, :3].copy()).cuda()
    c.ctx = [48, 0]
    got = c.run(table=table, ctx=c.ints([2 ** 31 - 1, -5]))
    # The mask sees no node and the table ends with position 47.  Its last slot
    # holds the first sequence's node; the second sequence sees nothing.
    c.nodes, c.seen = [1, 1], [np.zeros((1, 1), bool)] * 2
    c.table = np.concatenate((c.table, np.full((2, 1), -1, np.int32)), 1)
    c.check(got)


def test_empty_cache():
    b = Batch([2], [16], 4, 2, 64, 16, "f16", seed=6)
    out = b.run(k=b.k[:0], v=b.v[:0])
    assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_seen_does_not_reach_a_row(dtype, value):
    """A drafted node whose key and value are not finite spoils the rows that
    see it and no others."""
    b = Batch([12], [40], 8, 2, 128, 16, dtype, seed=7)
    clean = b.run().clone()
    bad = 5
    sees = b.seen[0][:, bad].copy()
    assert sees.any() and not sees.all()
    p = 40 + bad
    b.v[b.table[0, p // 16], p % 16, 1, 3] = value
    out = b.run()
    assert torch.equal(out[~sees], clean[~sees])
    hit = torch.from_numpy(sees).cuda()
    assert not bool(torch.isfinite(out[hit][:, 4:, 3]).any())          # the heads of key head 1, that column
    same = out.clone()
    same[:, 4:, 3] = clean[:, 4:, 3]
    assert np.allclose(same.double().cpu(), clean.double().cpu(), rtol=0, atol=2 * torch.finfo(DT[dtype]).eps)
    b.k[b.table[0, p // 16], p % 16] = float("nan")
    assert torch.equal(b.run()[~sees], clean[~sees])


def test_extreme_scores():
    """Scores far apart: one position takes all the weight; and scale 0."""
    b = Batch([3], [200], 4, 1, 64, 16, "bf16", seed=8)
    b.q *= 100
    b.check(b.run())
    b.scale = 0.0
    b.check(b.run())
    b.scale = -0.25
    b.check(b.run())


def test_no_rows():
    b = Batch([1], [5], 4, 2, 64, 16, "f16", seed=9)
    out = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    lsb.lora_tree_attention(b.q[:0], b.k, b.v, torch.from_numpy(b.table).cuda(), b.ints([5]), b.ints([0, 0]), out, 1.0)


def test_cache_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^31 (and byte offsets 2^32)."""
    pages, page, kv, dim = 70000, 16, 16, 128
    assert pages * page * kv * dim > 2 ** 31
    k = torch.empty(pages, page, kv, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    b = Batch([2], [90], 32, kv, dim, page, "bf16", seed=10)
    where = [69999, 3, 66000, 65537, 40000, 69000]
    for i, p in enumerate(where):
        k[p], v[p] = b.k[b.table[0, i]], b.v[b.table[0, i]]
    table = b.ints([where])
    assert torch.equal(b.run(k=k, v=v, table=table), b.run())


def test_stream_and_graph():
    b = Batch([5, 9], [800, 100], 8, 2, 128, 16, "bf16", seed=12)
    want = b.run().clone()
    table, ctx, start = torch.from_numpy(b.table).cuda(), b.ints(b.ctx), b.ints([0, 5, 14])
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.run(out=out, table=table, ctx=ctx, start=start)
    side.synchronize()
    assert torch.equal(out, want)
    need = lsb.lora_tree_attention_workspace_bytes(2, 14, 8, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lsb.lora_tree_attention(b.q, b.k, b.v, table, ctx, start, out, b.scale, mask=b.mask, workspace=ws)
    for lengths in ([800, 100], [3, 100], [500, 0], [790, 95]):   # lengths are data: the graph follows them
        ctx.copy_(b.ints(lengths))
        ws.fill_(255)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, b.run(ctx=b.ints(lengths)))


def test_workspace_argument():
    b = Batch([2], [600], 4, 2, 64, 16, "f16", seed=13)
    need = lsb.lora_tree_attention_workspace_bytes(1, 2, 4, 2, 64)
    args = (b.q, b.k, b.v, torch.from_numpy(b.table).cuda(), b.ints(b.ctx), b.ints([0, 2]))
    out = torch.empty_like(b.q)
    with pytest.raises(lsb.LoraError, match="workspace"):
        lsb.lora_tree_attention(*args, out, b.scale, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    lsb.lora_tree_attention(*args, out, b.scale, mask=b.mask, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    b.check(out)
