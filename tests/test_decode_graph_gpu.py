"""Captured calls without an explicit workspace: every graph has its own."""
import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb
from test_decode_attention_gpu import Batch
from test_decode_pages_gpu import Model, grow, ints, status_of
from test_decode_q4_gpu import make

pytestmark = pytest.mark.gpu


def spy(monkeypatch, name, at):
    """Notes the workspace address of every call of a C entry point (argument
    `at`; its size follows)."""
    seen, real = [], getattr(lsb.lib(), name)

    def call(*args):
        seen.append((args[at], args[at + 1]))
        return real(*args)

    monkeypatch.setattr(lsb.lib(), name, call)
    return seen


def capture(fn):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    return graph


def apart(spans):
    spans = sorted(spans)
    return all(a + n <= b for (a, n), (b, _) in zip(spans, spans[1:]))


def test_attention_graphs(monkeypatch):
    """Two graphs, the second with the larger workspace: their buffers are
    apart, from each other and from the eager calls', and replays side by side
    with eager work are right."""
    small = Batch([3], [900], 8, 2, 128, 16, "f16", seed=1)
    large = Batch([30, 20], [2000, 700], 32, 4, 128, 16, "bf16", seed=2)
    seen = spy(monkeypatch, "lora_tree_attention", 13)
    args, want, out = [], [], []
    for b in (small, large):
        args.append((b.q, b.k, b.v, torch.from_numpy(b.table).cuda(), b.ints(b.ctx),
                     b.ints(np.concatenate([[0], np.cumsum(b.nodes)]))))
        want.append(b.run().clone())
        out.append(torch.zeros_like(b.q))
    eager = seen[:]
    run = lambda i, b: lsb.lora_tree_attention(*args[i], out[i], b.scale, mask=b.mask)  # noqa: E731
    graphs = [capture(lambda i=i, b=b: run(i, b)) for i, b in enumerate((small, large))]
    assert len(seen) == 4 and apart([seen[2], seen[3], max(eager)])
    big = Batch([64] * 4, [3000] * 4, 16, 2, 256, 16, "bf16", seed=3)   # the stream's buffer grows
    big.run()
    filler = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 20, 1 << 22)]
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        again = [b.run() for b in (small, large)]
        torch.cuda.synchronize()
        for o, a, w in zip(out, again, want):
            assert torch.equal(o, w) and torch.equal(a, w)
    assert all(bool(torch.isnan(f).all()) for f in filler)


def test_a_step_of_calls_in_one_graph(monkeypatch):
    """Products with splits, a fork and a compaction in one graph."""
    x, codes, scales, z = make(12, 512, 10752, 32, False, "bf16", seed=3)
    w = lsb.lora_q4_pack(codes, scales, z, 10752, 32)
    assert lsb.lora_q4_matmul_workspace_bytes(12, 512, 10752, 32) > 0
    y, y2 = (torch.zeros(12, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = lsb.lora_q4_matmul(x, w, torch.empty_like(y)).clone()
    m = Model(pages=60, seed=4)
    c = m.device()
    grow(m, c, [0, 1], [6, 9])
    src, dst, gone, live = ints([0, 1, 0]), ints([2, 3, 4]), ints([0]), status_of(1)
    cached = dict(lsb._ws_cache)

    def step():
        lsb.lora_q4_matmul(x, w, y)
        lsb.lora_pages_fork(c, src, dst)
        lsb.lora_q4_matmul(x, w, y2)
        lsb.lora_pages_compact(c, live)

    graph = capture(step)
    assert lsb._ws_cache == cached
    for _ in range(3):
        y.zero_()
        y2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(y2, want)
        m.fork([0, 1, 0], [2, 3, 4])
        assert live.tolist() == [m.compact()]
        m.same(c)
        lsb.lora_pages_free(c, gone)
        m.free([0])
        grow(m, c, [0], [11])


def test_shrink_in_a_graph():
    """The adapters' shrink splits H over a workspace too."""
    T, H, r, L = 64, 8192, 16, 4
    ids = torch.arange(T, dtype=torch.int32, device="cuda") % L
    seg = lsb.lora_build_segments(ids, L)
    assert lsb.lora_shrink_workspace_bytes(T, L, H, r) > 0
    g = torch.Generator(device="cuda").manual_seed(5)
    x, A = (torch.randn(*s, device="cuda", generator=g).half() for s in ((T, H), (L, r, H)))
    want = lsb.lora_shrink(x, A, seg, torch.zeros(T, r, device="cuda")).clone()
    cached = dict(lsb._ws_cache)
    v = torch.zeros(T, r, device="cuda")
    graph = capture(lambda: lsb.lora_shrink(x, A, seg, v))
    assert lsb._ws_cache == cached
    for _ in range(3):
        v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(v, lsb.lora_shrink(x, A, seg, torch.zeros_like(v)))
        assert torch.equal(v, want)
