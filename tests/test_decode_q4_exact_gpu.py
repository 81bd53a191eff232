"""4-bit products whose every sum is exact, compared bit for bit, and products
of infinities and of very large inputs.

Exact sums: x and the scales are powers of two or small whole numbers, so each
partial sum is a whole number below 2^24 times one power of two, in whatever
order it is taken; y is its rounding."""
import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb
from test_decode_q4_gpu import DT, make, reference

pytestmark = pytest.mark.gpu

# Every form of the product, by tokens and shape: tails of k and n, groups that
# end beyond k, splits that end inside a chunk.
SHAPES = [
    # T, n, k, group, zeros
    (1, 33, 129, 32, True),
    (1, 512, 4096, 128, True),
    (4, 200, 8192, 128, False),
    (9, 4096, 20480, 128, True),
    (11, 4096, 20480, 128, False),
    (16, 8200, 4000, 64, True),
    (17, 96, 1032, 32, True),
    (26, 512, 10752, 32, True),
    (40, 8192, 1024, 32, False),
    (58, 505, 16888, 32, True),
    (64, 28672, 1024, 64, True),
    (77, 5003, 4064, 32, True),
    (90, 512, 21990, 128, True),
    (122, 22012, 512, 32, True),
    (128, 8192, 8192, 128, False),
    (257, 512, 10745, 32, True),
    (16, 70000, 300, 128, False),
    (30, 66000, 260, 64, True),
    (90, 40000, 384, 128, True),
]


def whole(T, n, k, group, zeros, dtype, seed):
    """Inputs whose sums are exact."""
    _, codes, _, z = make(T, n, k, group, zeros, dtype, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randint(-2, 3, (T, k), device="cuda", generator=g).to(DT[dtype])
    scales = (2.0 ** torch.randint(-9, -6, (n, -(-k // group)), device="cuda", generator=g)).to(DT[dtype])
    return x, codes, scales, z


def product(x, codes, scales, z, k, group):
    w = lsb.lora_q4_pack(codes, scales, z, k, group)
    y = torch.full((x.shape[0], codes.shape[0]), float("nan"), dtype=x.dtype, device="cuda")
    return lsb.lora_q4_matmul(x, w, y)


def expected(x, codes, scales, z, k, group, dtype):
    y, terms = reference(x, codes, scales, z, k, group, "f16")
    # Whole numbers of the smallest scale.  A group's sums before its scale are
    # whole too, and below 128 x 2 (128 + 15) in either type.
    assert (terms * 2 ** 9).max() < 2 ** 24 and np.array_equal(np.round(y * 2 ** 9), y * 2 ** 9)
    return torch.from_numpy(y).cuda().to(x.dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,n,k,group,zeros", SHAPES)
def test_exact_sums(T, n, k, group, zeros, dtype):
    """x everywhere, and x in the last inputs, the last group, one group in the
    middle and one input alone."""
    x, codes, scales, z = whole(T, n, k, group, zeros, dtype, seed=T + n + k)
    assert torch.equal(product(x, codes, scales, z, k, group), expected(x, codes, scales, z, k, group, dtype))
    last, mid = (k - 1) // group * group, k // 2 // group * group
    for lo, hi in ((max(0, k - 8), k), (last, k), (mid, min(k, mid + group)), (k - 1, k), (0, 1), (max(0, k - 129), k)):
        part = torch.zeros_like(x)
        part[:, lo:hi] = x[:, lo:hi]
        part[:, lo] = 1.0
        assert torch.equal(product(part, codes, scales, z, k, group),
                           expected(part, codes, scales, z, k, group, dtype)), (lo, hi)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,n,k,group,zeros", [s for s in SHAPES if s[0] * s[1] * s[2] < 2e9])
def test_infinities(T, n, k, group, zeros, dtype):
    """Infinite inputs give what the definition gives: an infinity of the sign
    of (q - z) x, NaN where q = z or where infinities of both signs meet."""
    x, codes, scales, z = whole(T, n, k, group, zeros, dtype, seed=T + n)
    inf = float("inf")
    x[0, k - 1] = inf
    if T > 3:
        x[1, k // 2] = -inf
        x[2, 0], x[2, k - 1] = inf, inf
        x[3, 0], x[3, k // 3] = inf, float("nan")
    if T > 20:
        x[T - 1, 3], x[T - 1, k - 2] = inf, -inf
    ref = reference(torch.where(torch.isfinite(x), x, 0), codes, scales, z, k, group, dtype)[0]
    unit = torch.eye(k, dtype=x.dtype, device="cuda")[~torch.isfinite(x).all(0)]  # the inputs that are not finite somewhere
    w = dict(zip(torch.nonzero(~torch.isfinite(x).all(0))[:, 0].tolist(), reference(unit, codes, scales, z, k, group, dtype)[0]))
    with np.errstate(invalid="ignore"):
        for t, h in torch.nonzero(~torch.isfinite(x)).tolist():
            ref[t] += w[h] * float(x[t, h])
    got = product(x, codes, scales, z, k, group).double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    there = ~np.isnan(ref)
    assert np.array_equal(got[there], torch.from_numpy(ref).to(DT[dtype]).double().numpy()[there])
    assert np.isposinf(ref[0]).any() and np.isneginf(ref[0]).any()
    old = torch.full((T, n), 3.0, dtype=x.dtype, device="cuda")
    lsb.lora_q4_matmul(x, lsb.lora_q4_pack(codes, scales, z, k, group), old, add_inputs=True)
    added = old.double().cpu().numpy()
    far = ~np.isfinite(ref)
    assert np.array_equal(added[far], got[far], equal_nan=True)
    assert np.array_equal(added[~far], torch.from_numpy(ref + 3.0).to(x.dtype).double().numpy()[~far])


@pytest.mark.parametrize("T,n,k,group,zeros", [(1, 64, 1024, 128, True), (6, 512, 4096, 64, False), (40, 8192, 1024, 32, True),
                                               (58, 505, 16888, 32, True)])
def test_very_large_inputs(T, n, k, group, zeros):
    """bfloat16 inputs near the type's end whose products with the weights are
    far below it."""
    x, codes, scales, z = whole(T, n, k, group, zeros, "bf16", seed=n)
    scales = scales * 2.0 ** -20
    big = x * 2.0 ** 125                                # |x| up to 2^126, the sums of x beyond 2^128
    ref = reference(x, codes, scales, z, k, group, "bf16")[0] * 2.0 ** 125
    got = product(big, codes, scales, z, k, group)
    assert torch.equal(got, torch.from_numpy(ref).cuda().to(torch.bfloat16))
