"""Tree attention where values are not finite beside missing pages, and where
one position outweighs many (lora_tree_attention), against the definition in 64
bits.  The tolerance is that of test_decode_attention_gpu."""
import numpy as np
import pytest
import torch

from test_decode_attention_gpu import DT, Batch

pytestmark = pytest.mark.gpu


def position(b, seq, p):
    return b.table[seq, p // b.page], p % b.page


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nodes,heads,kv,dim", [(1, 16, 8, 128), (3, 64, 8, 128), (9, 64, 8, 64), (3, 32, 4, 256), (4, 24, 4, 80)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_missing_pages_and_values_that_are_not_finite(nodes, heads, kv, dim, dtype, value):
    """Pages of the context are missing, and seen values beside them are not
    finite in one column: that column of their head is spoilt, the others are
    the definition's.  Twelve sequences, so that a workgroup takes several tiles
    of positions one after the other."""
    B = 12
    b = Batch([nodes] * B, [1400 - 7 * i for i in range(B)], heads, kv, dim, 16, dtype, seed=nodes + dim)
    hit = [37, 390, 70, 1000]                          # beside a missing page, three times; beside none
    for s in range(B):
        b.table[s, [3, 25, 61]] = [-1, -7, 10 ** 6]
        for p in hit:
            b.v[position(b, s, p)][0, 5] = value
    got = b.run()
    spoilt = got[:, :heads // kv, 5].double().cpu().numpy()
    assert not np.isfinite(spoilt).any()
    if value == float("inf"):
        assert (spoilt > 0).all()
    for s in range(B):
        for p in hit:
            b.v[position(b, s, p)][0, 5] = 0.0         # the definition's other columns
    got[:, :heads // kv, 5] = torch.from_numpy(b.expect()[0][:, :heads // kv, 5]).to(got)
    b.check(got)


def outweighed(dtype, gap, ctx, nodes, heads, kv, dim, sink_value, seed):
    """A batch whose first position scores `gap` above all others in every row,
    with value sink_value; the others score alike, their values of one sign."""
    b = Batch([nodes], [ctx], heads, kv, dim, 16, dtype, mask="none", seed=seed)
    b.q[:] = 0
    b.q[:, :, 0] = 4.0
    b.scale = 0.25
    at = np.arange(ctx)
    pages, slots = torch.from_numpy(b.table[0, at // 16].astype(np.int64)).cuda(), torch.from_numpy(at % 16).cuda()
    b.k[pages, slots] = 0
    b.k[pages[:1], slots[:1], :, 0] = gap
    b.v[pages, slots] = b.v[pages, slots].abs() + 0.5
    b.v[pages[:1], slots[:1]] = sink_value
    return b


def check_alike(b, gap, out, lse):
    """Every row of an outweighed batch against the same weighted mean.  The
    tolerance is that of test_decode_attention_gpu and half the step of a subnormal
    weight: 2^-34 of the heaviest one in binary16."""
    ctx = b.ctx[0]
    at = np.arange(ctx)
    v = b.v[b.table[0, at // 16], at % 16, 0].double().cpu().numpy()
    w = np.where(at == 0, 1.0, np.exp(-gap))
    want, mag = w @ v / w.sum(), w @ np.abs(v) / w.sum()
    half, sums, score = torch.finfo(DT[b.dtype]).eps / 2, (64 + ctx / 128) * 2.0 ** -23, gap * (b.dim + 8) * 2.0 ** -23
    tol = np.abs(want) * half * 1.001 + mag * (half + 2 * score + 2 * sums + 2.0 ** -20) + 2.0 ** -24
    tol += 2.0 ** -34 * np.abs(v[1:]).sum(0) / w.sum()
    worst = np.max(np.abs(out.double().cpu().numpy() - want) / tol)
    assert worst <= 1, worst
    g = lse.double().cpu().numpy()
    assert np.abs(g - gap - np.log(w.sum())).max() <= score + sums + 2.0 ** -18 + gap * 2.0 ** -22


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [8.0, 11.0, 15.0, 16.0, 16.75, 17.5, 20.0])
@pytest.mark.parametrize("nodes,heads,dim", [(1, 4, 128), (1, 2, 64), (1, 2, 256), (12, 8, 128), (40, 8, 64), (12, 4, 256)])
def test_one_position_outweighs_thousands(dtype, gap, nodes, heads, dim):
    """The mass of thousands of positions, each far below the heaviest one,
    reaches the result, which is theirs alone: the heaviest has the value 0."""
    for ctx in (700, 6000):
        b = outweighed(dtype, gap, ctx, nodes, heads, 1, dim, 0.0, seed=int(gap * 4) + dim)
        lse = torch.empty(nodes, heads, device="cuda")
        check_alike(b, gap, b.run(lse=lse), lse)


@pytest.mark.parametrize("nodes,heads", [(1, 2), (40, 4)])
def test_small_weights_of_a_long_context(nodes, heads):
    """120000 positions behind one that outweighs them all."""
    for gap in (15.5, 17.0):
        b = outweighed("f16", gap, 120000, nodes, heads, 1, 64, 0.0, seed=3)
        lse = torch.empty(nodes, heads, device="cuda")
        check_alike(b, gap, b.run(lse=lse), lse)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_lse_of_single_positions(dtype):
    """A row that sees one position: o is its value, lse its score."""
    b = Batch([2, 1], [1, 1], 4, 2, 64, 16, dtype, mask="none", seed=5)
    lse = torch.empty(3, 4, device="cuda")
    out = b.run(lse=lse)
    b.check(out, lse)
    v = torch.stack([b.v[position(b, s, 0)] for s in (0, 0, 1)]).repeat_interleave(2, 1)
    assert torch.equal(out, v)


@pytest.mark.parametrize("nodes,ctx,heads,kv,dim,page", [
    ([1], [509], 32, 8, 128, 16), ([2], [700], 8, 1, 96, 16), ([1, 1, 1], [31, 320, 3300], 8, 2, 64, 16),
    ([3, 2], [5000, 40], 8, 2, 80, 24), ([40], [1500], 4, 4, 128, 16), ([33, 17], [500, 900], 2, 1, 64, 16),
    ([12], [1100], 8, 2, 72, 32),
])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weights_in_two_parts(nodes, ctx, heads, kv, dim, page, dtype):
    """Up to 64 rows a sequence, of dims up to 128, the weights' rounding does not
    show in o: the tolerance has its square (what two 16-bit parts leave over) in
    its place."""
    b = Batch(nodes, ctx, heads, kv, dim, page, dtype, seed=dim + sum(ctx))
    got = b.run()
    o, _, mag, spread = b.expect()
    half = torch.finfo(DT[dtype]).eps / 2
    sums, score = (64 + max(ctx) / 128) * 2.0 ** -23, (spread * (dim + 8) * 2.0 ** -23)[..., None]
    tol = np.abs(o) * half * 1.001 + mag * (half * half + 2 * score + 2 * sums + 2.0 ** -20 + (max(ctx) + 64) * 2.0 ** -34) + 2.0 ** -24
    assert np.max(np.abs(got.double().cpu().numpy() - o) / tol) <= 1


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nodes", [2, 12])
def test_infinite_value_with_a_small_weight(nodes, dtype):
    """A drafted node's infinite value reaches the rows that see it, whatever its
    weight, and its finite columns have both parts of the weight."""
    b = Batch([nodes], [300], 8, 2, 128, 16, dtype, mask="chain", seed=nodes)
    p = position(b, 0, 300)
    b.v[p][1, 7] = float("inf")
    got = b.run()
    assert bool(torch.isposinf(got[:, 4:, 7]).all())
    b.v[p][1, 7] = 0.0
    got[:, 4:, 7] = torch.from_numpy(b.expect()[0][:, 4:, 7]).to(got)
    b.check(got)
