"""Cases and timing bodies of the decode-step operators around the adapters.

Three operators share a serving step with the adapters' shrink and expand:

* ``q4``: the base projection under the adapters, ``y[t, c] = sum_h x[t, h] s[c, h / g] (q[c, h] - z[c, h / g])``
  with 4-bit codes q, one scale s (and optionally one zero z, else 8) for each group of g inputs;
* ``attn``: attention of a step's drafted tokens (a tree for each sequence, one token in the simplest case)
  over a paged key / value cache;
* ``pages``: the cache's page operations: copying pages, forking sequences, keeping the accepted path of a
  drafted tree, freeing.

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is set, through
``lora_serving_build_amd``.  ``exact`` computes the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
_DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # The key (or value) projection of one decoding token: the smallest product, bound by latency.
        {"name": "q4 one token", "op": "q4", "T": 1, "n": 1024, "k": 4096, "group": 128, "zeros": False, "dtype": "f16"},
        # A gate or up projection of the 8192-wide layer for a few sequences: the widest weight.
        {"name": "q4 wide", "op": "q4", "T": 4, "n": 28672, "k": 8192, "group": 128, "zeros": True, "dtype": "bf16"},
        # The down projection of the same layer for a full decode batch: the longest contraction.
        {"name": "q4 long", "op": "q4", "T": 16, "n": 8192, "k": 28672, "group": 64, "zeros": False, "dtype": "bf16"},
        # A verification step: drafted tokens of several sequences, sizes that fill no tile, the finest groups.
        {"name": "q4 verify odd", "op": "q4", "T": 77, "n": 5003, "k": 4064, "group": 32, "zeros": True, "dtype": "f16"},
        # One sequence, one token, a short context: the smallest attention call.
        {"name": "attn one token", "op": "attn", "B": 1, "nodes": 1, "ctx": 509, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "f16"},
        # An ordinary decode batch, ragged contexts, one token each.
        {"name": "attn decode batch", "op": "attn", "B": 64, "nodes": 1, "ctx": 4096, "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "dtype": "bf16"},
        # Two long contexts with a short drafted tree: few rows over a long axis.
        {"name": "attn long", "op": "attn", "B": 2, "nodes": 5, "ctx": 120011, "heads": 32, "kv_heads": 4, "dim": 128, "page": 32, "dtype": "f16"},
        # Wide drafted trees in a batch: many rows share a context.
        {"name": "attn trees", "op": "attn", "B": 16, "nodes": 48, "ctx": 6001, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # One prompt forked into a few branches, which are freed again: the smallest page call.
        {"name": "pages fork few", "op": "pages", "kind": "fork_free", "n": 3, "ctx": 700, "pools": 16, "pages": 512, "page": 16, "kv_heads": 8, "dim": 128, "dtype": "f16"},
        # A beam step over a batch: every sequence takes the state of another, its last page copied in every layer.
        {"name": "pages reorder", "op": "pages", "kind": "reorder", "n": 96, "ctx": 300, "pools": 64, "pages": 2048, "page": 16, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # The accepted paths of a batch of drafted trees, made contiguous in every layer.
        {"name": "pages accept", "op": "pages", "kind": "accept", "n": 48, "ctx": 257, "pools": 64, "pages": 1300, "page": 16, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # Whole pages copied in every layer (a swap, a prefix made private).
        {"name": "pages copy", "op": "pages", "kind": "copy", "n": 200, "ctx": 0, "pools": 64, "pages": 900, "page": 16, "kv_heads": 8, "dim": 128, "dtype": "f16"},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    dtype = rng.choice(("f16", "bf16"))
    op = rng.choice(("q4", "attn", "pages"))
    if op == "q4":
        # a width of the adapters' own workloads, or one that fills no tile (rows stay 16-byte aligned)
        k = rng.choice((1024, 2048, 4096, 8192, 16384, 28672)) if rng.random() < 0.5 else 8 * (2 * _between(rng, 64, 1792) + 1)
        return {"op": op, "T": _between(rng, 1, 128), "n": 2 * _between(rng, 256, 14336) + 1 if rng.random() < 0.5 else 1024 * rng.choice((1, 2, 4, 8, 16, 28)), "k": k,
                "group": rng.choice((32, 64, 128)), "zeros": rng.random() < 0.5, "dtype": dtype}
    dim = rng.choice((64, 80, 128, 128, 256))
    if op == "attn":
        kv = rng.choice((1, 2, 4, 8))
        return {"op": op, "B": _between(rng, 1, 64), "nodes": _between(rng, 1, 64), "ctx": _between(rng, 16, 120000),
                "heads": kv * rng.choice((1, 3, 4, 8)), "kv_heads": kv, "dim": dim, "page": rng.choice((16, 24, 32, 64)), "dtype": dtype}
    kind = rng.choice(("fork_free", "reorder", "accept", "copy"))
    n, ctx, page = _between(rng, 1, 128), _between(rng, 17, 1500), rng.choice((16, 24, 32))
    pages = 2 * n + 7 if kind == "copy" else (n + 1) * (-(-ctx // page) + 6)
    return {"op": op, "kind": kind, "n": n, "ctx": ctx, "pools": 2 * _between(rng, 1, 40), "pages": pages, "page": page,
            "kv_heads": rng.choice((2, 4, 8)), "dim": dim, "dtype": dtype}


def _cache_bytes(c):
    return c["pools"] * c["pages"] * c["page"] * c["kv_heads"] * c["dim"] * 2


def draw(rng: random.Random):
    most = {"q4": 1.25e8, "attn": 5e8, "pages": 8e8}  # bytes: a listed case has more
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] > most[c["op"]] or w["flops"] > 6.5e10:
            continue
        if c["op"] == "pages" and _cache_bytes(c) > 4.5e9:
            continue
        if c["op"] == "attn" and c["B"] * (c["ctx"] + c["nodes"]) * c["kv_heads"] * (c["dim"] + c["nodes"] * c["heads"] / c["kv_heads"] / 2) > 2.5e8:
            continue  # the plain form's padded scores and keys
        return c


def _lengths(c):
    """Context length and node count of each sequence: ragged, fixed by the case."""
    B = c["B"]
    ctx = [max(0, c["ctx"] * (B - (b * 7) % B) // B - 3 * (b % 5)) for b in range(B)]
    nodes = [max(1, c["nodes"] - (b * 5) % (c["nodes"] // 2 + 1)) for b in range(B)]
    return ctx, nodes


def _seq_lengths(c):
    """Cached tokens of each sequence of a page case."""
    return [max(1, c["ctx"] - 3 * (i * 5 % 7) * (c["ctx"] > 32)) for i in range(c["n"])]


def work(case):
    c = case
    if c["op"] == "q4":
        g = -(-c["k"] // c["group"])
        return {"bytes": c["n"] * ((c["k"] + 1) // 2) + c["n"] * g * (3 if c["zeros"] else 2) + 2 * c["T"] * (c["k"] + c["n"]),
                "flops": 2 * c["T"] * c["n"] * c["k"]}
    if c["op"] == "attn":
        ctx, nodes = _lengths(c)
        keys = sum(a + b for a, b in zip(ctx, nodes))
        return {"bytes": 4 * keys * c["kv_heads"] * c["dim"] + 4 * sum(nodes) * c["heads"] * c["dim"],
                "flops": 4 * sum((a + b) * b for a, b in zip(ctx, nodes)) * c["heads"] * c["dim"]}
    row = 2 * c["kv_heads"] * c["dim"] * c["pools"]
    if c["kind"] == "copy":
        rows = c["n"] * c["page"]
    elif c["kind"] == "accept":
        rows = sum(_path(c, i)[1] for i in range(c["n"]))
    elif c["kind"] == "reorder":
        rows = sum(x % c["page"] for i, x in enumerate(_seq_lengths(c)))
    else:
        rows = c["n"] * (_seq_lengths(c)[0] % c["page"])
    return {"bytes": 2 * rows * row + 1, "flops": 0}


def _path(c, i):
    """Drafted and accepted node counts of sequence i of an accept case."""
    drafted = 24 + i % 9
    return drafted, 3 + i % 5


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    out = torch.empty(shape, dtype=dtype, device=_DEV)
    return out.normal_(0.0, std, generator=g)


def _int32(v):
    return torch.tensor(np.asarray(v, np.int32), device=_DEV)


def prepare(case, seed):
    c, g, rs = case, _gen(seed), np.random.RandomState(seed % (1 << 32))
    s = {"case": dict(c)}
    dt = _DT[c["dtype"]]
    if c["op"] == "q4":
        groups = -(-c["k"] // c["group"])
        s["x"] = _normal(g, (c["T"], c["k"]), dt)
        s["codes"] = torch.randint(0, 256, (c["n"], (c["k"] + 1) // 2), dtype=torch.uint8, device=_DEV, generator=g)
        spread = torch.rand((c["n"], groups), device=_DEV, generator=g)
        s["scales"] = ((0.5 + spread) * (0.25 / math.sqrt(c["k"]))).to(dt)
        s["zeros"] = torch.randint(4, 12, (c["n"], groups), dtype=torch.uint8, device=_DEV, generator=g) if c["zeros"] else None
        s["y"] = torch.empty((c["T"], c["n"]), dtype=dt, device=_DEV)
        if own:  # a server lays its weights out once, when it loads them
            import lora_serving_build_amd as lsb
            s["weight"] = lsb.lora_q4_pack(s["codes"], s["scales"], s["zeros"], c["k"], c["group"])
    elif c["op"] == "attn":
        ctx, nodes = _lengths(c)
        total = sum(nodes)
        held = [-(-(a + b) // c["page"]) for a, b in zip(ctx, nodes)]
        num = sum(held) + 5
        order = rs.permutation(num).astype(np.int32)
        table = np.full((c["B"], max(held)), -1, np.int32)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        words = -(-max(nodes) // 64)
        mask = np.zeros((total, words), np.uint64)
        row = 0
        for n in nodes:  # each node sees itself and its ancestors
            first = row
            for i in range(n):
                if i:
                    mask[row] = mask[first + rs.randint(max(0, i - 9), i)]
                mask[row, i // 64] |= np.uint64(1) << np.uint64(i % 64)
                row += 1
        s["q"] = _normal(g, (total, c["heads"], c["dim"]), dt)
        s["k"] = _normal(g, (num, c["page"], c["kv_heads"], c["dim"]), dt)
        s["v"] = _normal(g, (num, c["page"], c["kv_heads"], c["dim"]), dt)
        s["table"] = torch.from_numpy(table).to(_DEV)
        s["ctx"] = _int32(ctx)
        s["start"] = _int32(np.concatenate([[0], np.cumsum(nodes)]))
        s["mask"] = torch.from_numpy(mask.view(np.int64)).to(_DEV)
        s["out"] = torch.empty_like(s["q"])
        s["longest"], s["most"] = max(a + b for a, b in zip(ctx, nodes)), max(nodes)
        s["scale"] = 1.0 / math.sqrt(c["dim"])
    else:
        _prepare_pages(c, s, g, rs, dt)
    return s


def _prepare_pages(c, s, g, rs, dt):
    n, page, pages = c["n"], c["page"], c["pages"]
    s["pool"] = _normal(g, (c["pools"], pages, page, c["kv_heads"], c["dim"]), dt)
    order = rs.permutation(pages).astype(np.int32)
    if c["kind"] == "copy":
        s["src"], s["dst"] = _int32(order[:n]), _int32(order[n:2 * n])
        seqs, width, lens, extra = 1, 4, [0], [0]
    else:
        lens = _seq_lengths(c)
        extra = [0] * n
        if c["kind"] == "fork_free":
            lens = lens[:1] + [0] * n
            extra = [0] * (n + 1)
            s["src"], s["dst"] = _int32([0] * n), _int32(range(1, n + 1))
        elif c["kind"] == "reorder":
            # the better half of the beams is kept twice
            kept = rs.permutation(n)[: max(1, n // 2)]
            s["src"], s["dst"] = _int32(kept[rs.randint(0, len(kept), n)]), _int32(range(n))
        else:
            counts = [_path(c, i) for i in range(n)]
            extra = [d for d, _ in counts]
            path = np.zeros((n, max(a for _, a in counts)), np.int32)
            for i, (d, a) in enumerate(counts):
                path[i, :a] = np.sort(rs.permutation(d)[:a])
            s["seqs"], s["drafted"] = _int32(range(n)), _int32(extra)
            s["path"], s["accepted"] = _int32(path), _int32([a for _, a in counts])
            s["new_len"] = torch.empty(n, dtype=torch.int32, device=_DEV)
        seqs = len(lens)
        width = max(-(-(a + b) // page) for a, b in zip(lens, extra)) + 2
    table = np.full((seqs, width), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    at = 0
    for i, (a, b) in enumerate(zip(lens, extra)):
        h = -(-(a + b) // page)
        table[i, :h] = order[at:at + h]
        refs[order[at:at + h]] = 1
        at += h
    s["table"], s["refs"], s["lens"] = torch.from_numpy(table).to(_DEV), torch.from_numpy(refs).to(_DEV), _int32(lens)
    s["status"] = torch.empty(n, dtype=torch.int32, device=_DEV)
    if own:
        import lora_serving_build_amd as lsb
        s["cache"] = lsb.PageCache(s["pool"], s["refs"], s["table"], s["lens"])


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if own:
        import lora_serving_build_amd as lsb
        if c["op"] == "q4":
            return lsb.lora_q4_matmul(s["x"], s["weight"], s["y"])
        if c["op"] == "attn":
            return lsb.lora_tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["start"], s["out"], s["scale"], mask=s["mask"])
        if c["kind"] == "copy":
            lsb.lora_pages_copy(s["cache"], s["src"], s["dst"])
            return s["pool"]
        if c["kind"] == "accept":
            lsb.lora_pages_accept(s["cache"], s["seqs"], s["drafted"], s["path"], s["accepted"], s["new_len"])
            return s["pool"], s["new_len"]
        lsb.lora_pages_fork(s["cache"], s["src"], s["dst"], s["status"])
        if c["kind"] == "fork_free":
            lsb.lora_pages_free(s["cache"], s["dst"])
        return s["pool"], s["table"], s["refs"], s["lens"], s["status"]
    if c["op"] == "q4":
        return _plain_q4(s, c)
    if c["op"] == "attn":
        return _plain_attention(s, c)
    if c["kind"] == "copy":
        s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
        return s["pool"]
    if c["kind"] == "accept":
        return _plain_accept(s, c)
    return _plain_fork(s, c)


def _plain_q4(s, c):
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).flatten(1)[:, : c["k"]].float()
    scale = s["scales"].float().repeat_interleave(c["group"], 1)[:, : c["k"]]
    zero = s["zeros"].float().repeat_interleave(c["group"], 1)[:, : c["k"]] if c["zeros"] else 8.0
    return ((s["x"].float() @ ((q - zero) * scale).T)).to(s["y"].dtype)


def _plain_attention(s, c):
    B, kv, G, D, page = c["B"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["page"]
    L, N = s["longest"], s["most"]
    at = torch.arange(L, device=_DEV)
    rows = s["table"].long().clamp(min=0)[:, at // page] * page + at % page
    k = s["k"].flatten(0, 1)[rows].float().transpose(1, 2)  # B, kv, L, D
    v = s["v"].flatten(0, 1)[rows].float().transpose(1, 2)
    i = torch.arange(N, device=_DEV)
    count = s["start"].diff().long()
    row = (s["start"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, N, kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, kv, G * N, D)
    node = at - s["ctx"].long()[:, None]  # B, L: which drafted node a position holds
    inside = (node >= 0) & (node < count[:, None])
    bits = s["mask"][row].gather(2, (node.clamp(0, N - 1) // 64)[:, None].expand(B, N, L))
    sees = (bits >> (node.clamp(min=0) % 64)[:, None]) & 1
    seen = (node < 0)[:, None] | (inside[:, None] & (sees == 1))  # B, N, L
    score = (q @ k.transpose(2, 3)).view(B, kv, G, N, L) * s["scale"]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, kv, G * N, L) @ v).view(B, kv, G, N, D) / total.clamp(min=1e-38)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, kv * G, D)
    # the rows of each sequence in order, without the padding
    return o[i < count[:, None]].to(s["q"].dtype)


def _plain_accept(s, c):
    page, n = c["page"], c["n"]
    most = s["path"].shape[1]
    j = torch.arange(most, device=_DEV)
    seqs = s["seqs"].long()
    base = s["lens"].long()[seqs][:, None]
    live = j < s["accepted"][:, None]
    table = s["table"].long()[seqs]
    src, dst = (base + s["path"])[live], (base + j)[live]
    who = torch.arange(n, device=_DEV)[:, None].expand(n, most)[live]
    rows = s["pool"][:, table[who, src // page], src % page]
    s["pool"][:, table[who, dst // page], dst % page] = rows
    s["new_len"] = s["lens"][seqs] + s["accepted"]
    return s["pool"], s["new_len"]


def _plain_fork(s, c):
    page, n = c["page"], c["n"]
    src, dst = s["src"].long(), s["dst"].long()
    pool, table, refs, lens = s["pool"], s["table"], s["refs"], s["lens"]
    width = table.shape[1]
    w = torch.arange(width, device=_DEV)
    length = lens[src]
    full, rest = length // page, length % page
    rows, old = table[src], table[dst]
    need = rest > 0
    order = torch.argsort((refs != 0).to(torch.int8), stable=True)
    rank = need.long().cumsum(0)
    fits = (rank <= (refs == 0).sum()) | ~need
    take = need & fits
    fresh = order[(rank - 1).clamp(min=0)].to(torch.int32)
    new = torch.where(w < full[:, None], rows, -1)
    new = torch.where((w == full[:, None]) & take[:, None], fresh[:, None], new)
    shared = (w < full[:, None]) & fits[:, None]
    one = torch.ones((), dtype=torch.int32, device=_DEV)
    spare = torch.cat((refs, refs.new_zeros(1)))  # the last entry takes what is not counted
    P = refs.shape[0]
    spare.index_put_((torch.where(shared, rows, P).long(),), one, accumulate=True)
    spare.index_put_((torch.where(take, fresh, P).long(),), one, accumulate=True)
    gone = (old >= 0) & fits[:, None]
    spare.index_put_((torch.where(gone, old, P).long(),), -one, accumulate=True)
    last = rows.gather(1, full.long().clamp(max=width - 1)[:, None])[:, 0].long()
    # rows of the last page that hold tokens
    r = torch.arange(page, device=_DEV)
    copied = (r < rest[:, None]) & take[:, None]
    a, b = last[:, None].expand(n, page)[copied], fresh.long()[:, None].expand(n, page)[copied]
    rr = r.expand(n, page)[copied]
    pool[:, b, rr] = pool[:, a, rr]
    table[dst] = torch.where(fits[:, None], new, old)
    lens[dst] = torch.where(fits, length, lens[dst])
    s["status"] = torch.where(fits, 0, 1).to(torch.int32)
    refs.copy_(spare[:P])
    if c["kind"] == "fork_free":
        held = table[dst]
        spare = torch.cat((refs, refs.new_zeros(1)))
        spare.index_put_((torch.where(held >= 0, held, P).long(),), -one, accumulate=True)
        refs.copy_(spare[:P])
        table[dst] = -1
        lens[dst] = 0
    return pool, table, refs, lens, s["status"]


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "pages":
        return None  # whole numbers and moved values: no computed number
    s = prepare(case, seed)
    if c["op"] == "q4":
        y = torch.zeros((c["T"], c["n"]), dtype=torch.float64, device=_DEV)
        x = s["x"].double()
        for g in range(s["scales"].shape[1]):  # group by group: sum (q - z) x, then times s
            lo, hi = g * c["group"], min(c["k"], (g + 1) * c["group"])
            b = s["codes"][:, lo // 2:(hi + 1) // 2].to(torch.int64)
            w = torch.zeros((c["n"], 2 * b.shape[1]), dtype=torch.float64, device=_DEV)
            w[:, 0::2] = (b % 16).double()
            w[:, 1::2] = (b // 16).double()
            w = w[:, : hi - lo] - (s["zeros"][:, g:g + 1].double() if c["zeros"] else 8.0)
            y += (x[:, lo:hi] @ w.T) * s["scales"][:, g].double()
        return y
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=_DEV)
    start, ctx = s["start"].tolist(), s["ctx"].tolist()
    G = c["heads"] // c["kv_heads"]
    words = s["mask"].cpu().numpy().view(np.uint64)
    for b in range(c["B"]):
        n, length = start[b + 1] - start[b], ctx[b]
        held = s["table"][b, : -(-(length + n) // c["page"])].long()
        k = s["k"][held].flatten(0, 1)[: length + n].double()
        v = s["v"][held].flatten(0, 1)[: length + n].double()
        seen = np.ones((n, length + n), bool)
        for i in range(n):
            for j in range(n):
                seen[i, length + j] = bool((int(words[start[b] + i, j // 64]) >> (j % 64)) & 1)
        seen = torch.from_numpy(seen).to(_DEV)
        for h in range(c["heads"]):
            z = s["q"][start[b]:start[b + 1], h].double() @ k[:, h // G].T / math.sqrt(c["dim"])
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            out[start[b]:start[b + 1], h] = torch.softmax(z, -1) @ v[:, h // G]
    return out
