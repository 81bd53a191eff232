"""The decode-step example: its layer's outputs against the same step computed
in 64 bits from the layer's own weights and the cache's contents.

Tolerance 1e-2 (1 + |value|), that of the adapters' parity tests: three rounded
16-bit stages (projection, attention, projection) follow one another."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")


def load():
    spec = importlib.util.spec_from_file_location("decode_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def weight(raw):
    codes, scales, zeros = raw
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(1).double()
    group = q.shape[1] // scales.shape[1]
    return (q - zeros.double().repeat_interleave(group, 1)) * scales.double().repeat_interleave(group, 1)


def adapted(x, w, a, bs, ids):
    y = x @ w.T
    for t, l in enumerate(ids):
        if l >= 0:
            y[t] += torch.cat([(x[t] @ a[l].double().T) @ b[l].double().T for b in bs])
    return y


def test_example_matches_the_step_in_64_bits():
    m = load()
    seen = []

    def inspect(layer, cache, x, y, o, ids, start, parents):
        qkv = adapted(x.double(), weight(layer.raw_qkv), layer.a_qkv, layer.b_qkv, ids)
        h, kv, d, page = layer.heads, layer.kv_heads, layer.dim, cache.page_size
        q = qkv[:, :h * d].view(-1, h, d)
        k_all, v_all = (p.double() for p in cache.layer(0))
        want = torch.zeros_like(q)
        for b in range(3):
            ctx, n = int(cache.seq_len[b]), int(start[b + 1] - start[b])
            pos = torch.arange(ctx + n, device="cuda")
            rows = cache.table[b].long()[pos // page]
            k, v = k_all[rows, pos % page], v_all[rows, pos % page]
            # the drafted rows hold what the layer computed
            for j, got in ((1, k), (2, v)):
                ref = qkv[start[b]:start[b + 1]].split([h * d, kv * d, kv * d], 1)[j].view(n, kv, d)
                assert bool(((got[ctx:] - ref).abs() <= 1e-2 * (1 + ref.abs())).all())
            for i in range(n):
                sees = list(range(ctx)) + [ctx + j for j in m.path_to(parents, int(start[b]), i)]
                for head in range(h):
                    g = head // (h // kv)
                    w = torch.softmax(k[sees, g] @ q[start[b] + i, head] / d ** 0.5, 0)
                    want[start[b] + i, head] = w @ v[sees, g]
        assert bool(((o.double() - want).abs() <= 1e-2 * (1 + want.abs())).all())
        ref = adapted(o.double().flatten(1), weight(layer.raw_o), layer.a_o, layer.b_o, ids)
        assert bool(((y.double() - ref).abs() <= 1e-2 * (1 + ref.abs())).all())
        named = np.bincount(cache.table.cpu().numpy()[cache.table.cpu().numpy() >= 0], minlength=cache.num_pages)
        assert np.array_equal(named, cache.refs.cpu().numpy())
        seen.append(len(ids))

    cache = m.run(steps=3, seed=1, verbose=False, inspect=inspect)
    assert len(seen) == 3
    assert bool((cache.refs == 0).all()) and bool((cache.table == -1).all()) and bool((cache.seq_len == 0).all())
