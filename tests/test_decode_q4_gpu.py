"""4-bit products (lora_q4_pack, lora_q4_matmul) against the definition in 64
bits.

Tolerance of y: half a step of its type, plus fp32 sums.  A term passes through
at most 32 additions inside a matrix-core step, 4 steps of a block, the blocks
and the waves: (48 + k / 128) roundings of at most 2^-23 of the sum of the
terms' magnitudes (bfloat16 sums (128 + q) x and takes (128 + z) x away, so
those are its terms)."""
import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(T, n, k, group, zeros, dtype, seed, x_scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    groups = -(-k // group)
    x = torch.empty(T, k, device="cuda").normal_(0, x_scale, generator=g).to(DT[dtype])
    codes = torch.randint(0, 256, (n, (k + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand(n, groups, device="cuda", generator=g) * 0.1 + 0.01).to(DT[dtype])
    z = torch.randint(0, 16, (n, groups), dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    return x, codes, scales, z


def reference(x, codes, scales, z, k, group, dtype):
    """y in 64 bits, and the sum of the terms' magnitudes."""
    c = codes.cpu().numpy()
    q = np.empty((c.shape[0], 2 * c.shape[1]))
    q[:, 0::2], q[:, 1::2] = c & 15, c >> 4
    q = q[:, :k]
    s = np.repeat(scales.double().cpu().numpy(), group, 1)[:, :k]
    zz = np.repeat(z.cpu().numpy().astype(float), group, 1)[:, :k] if z is not None else 8.0
    xd = x.double().cpu().numpy()
    y = xd @ ((q - zz) * s).T
    terms = (256.0 + q + zz) * s if dtype == "bf16" else np.abs(q - zz) * s
    return y, np.abs(xd) @ terms.T


def check(y, ref, terms, k, dtype, old=None):
    got = y.double().cpu().numpy()
    if old is not None:
        ref, terms = ref + old, terms + np.abs(old)
    tol = np.abs(ref) * torch.finfo(DT[dtype]).eps / 2 * 1.001 + terms * (48 + k / 128) * 2.0 ** -23 + 2.0 ** -24
    worst = np.max(np.abs(got - ref) / tol)
    assert worst <= 1, worst


CASES = [
    # T, n, k, group, zeros, dtype
    (1, 1, 1, 32, False, "f16"),
    (1, 16, 128, 128, False, "bf16"),
    (1, 1024, 4096, 128, True, "f16"),
    (1, 1000, 2048, 128, False, "bf16"),
    (2, 15, 31, 32, True, "bf16"),
    (3, 17, 129, 64, True, "f16"),
    (15, 48, 130, 32, False, "f16"),
    (16, 64, 1024, 64, True, "bf16"),
    (17, 96, 1032, 32, True, "f16"),
    (31, 250, 777, 96, False, "bf16"),
    (33, 129, 512, 256, True, "f16"),
    (64, 512, 1024, 128, True, "bf16"),
    (77, 203, 4064, 32, True, "f16"),
    (100, 130, 640, 512, False, "bf16"),
    (130, 300, 264, 64, False, "f16"),
    (128, 1024, 512, 128, False, "f16"),
    (260, 33, 1280, 128, True, "bf16"),
    (4, 2048, 8192, 128, True, "bf16"),
    (16, 512, 16384, 64, False, "f16"),
    (16, 8200, 4000, 64, False, "bf16"),
    (40, 8192, 1024, 32, True, "f16"),
    (100, 4099, 1032, 128, True, "bf16"),
    (30, 14336, 2048, 128, False, "f16"),
    (60, 16384, 2048, 64, True, "bf16"),
    (90, 16390, 2056, 32, False, "f16"),
    (128, 16384, 2048, 128, True, "bf16"),
    (200, 8192, 4096, 128, True, "f16"),
    (11, 4096, 20480, 128, False, "bf16"),
    # the forms that split k over workgroups, by tokens
    (1, 509, 10744, 32, True, "f16"),
    (26, 512, 10752, 32, False, "bf16"),
    (58, 505, 16888, 32, True, "bf16"),
    (90, 512, 21990, 128, False, "f16"),
    (122, 22012, 512, 32, True, "bf16"),
    (257, 512, 10745, 32, False, "f16"),
]


@pytest.mark.parametrize("T,n,k,group,zeros,dtype", CASES)
def test_product(T, n, k, group, zeros, dtype):
    x, codes, scales, z = make(T, n, k, group, zeros, dtype, seed=T * 7 + n + k)
    w = lsb.lora_q4_pack(codes, scales, z, k, group)
    ref, terms = reference(x, codes, scales, z, k, group, dtype)
    y = torch.full((T, n), float("nan"), dtype=DT[dtype], device="cuda")
    assert lsb.lora_q4_matmul(x, w, y) is y
    check(y, ref, terms, k, dtype)
    again = torch.empty_like(y)
    lsb.lora_q4_matmul(x, w, again)
    assert torch.equal(y, again)                       # same inputs, same bits
    old = torch.randn(T, n, device="cuda").to(DT[dtype])
    y = old.clone()
    lsb.lora_q4_matmul(x, w, y, add_inputs=True)
    check(y, ref, terms, k, dtype, old.double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("x_off,x_pad,y_off,y_pad", [(0, 8, 0, 4), (0, 3, 0, 1), (1, 8, 2, 4), (8, 8, 4, 8)])
def test_strides_and_offsets(dtype, x_off, x_pad, y_off, y_pad):
    """Rows at any stride and alignment; nothing beyond a row's n outputs is
    written, and nothing beyond its k inputs is read into the result."""
    T, n, k, group = 19, 100, 264, 64
    x, codes, scales, z = make(T, n, k, group, True, dtype, seed=5)
    w = lsb.lora_q4_pack(codes, scales, z, k, group)
    xb = torch.full((T, x_off + k + x_pad), float("nan"), dtype=DT[dtype], device="cuda")
    xb[:, x_off:x_off + k] = x
    yb = torch.full((T, y_off + n + y_pad), -7.0, dtype=DT[dtype], device="cuda")
    lsb.lora_q4_matmul(xb[:, x_off:x_off + k], w, yb[:, y_off:y_off + n])
    ref, terms = reference(x, codes, scales, z, k, group, dtype)
    check(yb[:, y_off:y_off + n], ref, terms, k, dtype)
    outside = torch.cat((yb[:, :y_off], yb[:, y_off + n:]), 1)
    assert bool((outside == -7.0).all())


def test_pack_takes_padded_rows():
    T, n, k, group, dtype = 4, 40, 200, 64, "f16"
    x, codes, scales, z = make(T, n, k, group, True, dtype, seed=9)
    wide = lambda t: torch.cat((t, torch.full_like(t, 1)), 1)[:, : t.shape[1]]  # noqa: E731
    a = lsb.lora_q4_pack(codes, scales, z, k, group)
    b = lsb.lora_q4_pack(wide(codes), wide(scales), wide(z), k, group)
    assert torch.equal(a.packed, b.packed)


def test_nan_and_infinity_stay_in_their_rows():
    T, n, k, group, dtype = 18, 64, 256, 128, "bf16"
    x, codes, scales, z = make(T, n, k, group, False, dtype, seed=11)
    w = lsb.lora_q4_pack(codes, scales, z, k, group)
    clean = lsb.lora_q4_matmul(x, w, torch.empty(T, n, dtype=DT[dtype], device="cuda")).clone()
    x[3, 5] = float("nan")
    x[17, 0] = float("inf")
    y = lsb.lora_q4_matmul(x, w, torch.empty(T, n, dtype=DT[dtype], device="cuda"))
    keep = [t for t in range(T) if t not in (3, 17)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[17]).any())


def test_no_tokens():
    w = lsb.lora_q4_pack(*make(1, 16, 128, 128, False, "f16", 1)[1:3], None, 128, 128)
    y = torch.full((1, 16), 3.0, dtype=torch.float16, device="cuda")
    lsb.lora_q4_matmul(torch.empty(0, 128, dtype=torch.float16, device="cuda"), w, y[:0])
    assert bool((y == 3.0).all())


def test_stream_and_graph():
    """On a side stream, and captured in a graph that is replayed between
    eager work."""
    T, n, k, group, dtype = 9, 320, 1024, 128, "bf16"
    x, codes, scales, z = make(T, n, k, group, True, dtype, seed=21)
    w = lsb.lora_q4_pack(codes, scales, z, k, group)
    want = lsb.lora_q4_matmul(x, w, torch.empty(T, n, dtype=DT[dtype], device="cuda")).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = torch.zeros(T, n, dtype=DT[dtype], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        lsb.lora_q4_matmul(x, w, y)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lsb.lora_q4_matmul(x, w, y)
    for i in range(3):
        x2 = x * (i + 1)
        keep = x.clone()
        x.copy_(x2)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, lsb.lora_q4_matmul(x, w, torch.empty_like(y)))
        x.copy_(keep)


def test_binding_refusals_on_the_gpu():
    x, codes, scales, z = make(4, 32, 128, 64, False, "f16", 1)
    w = lsb.lora_q4_pack(codes, scales, None, 128, 64)
    y = torch.empty(4, 32, dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        lsb.lora_q4_matmul(x.bfloat16(), w, y)
    with pytest.raises(ValueError):
        lsb.lora_q4_matmul(x[:, :64], w, y)
    with pytest.raises(ValueError):
        lsb.lora_q4_matmul(x, w, y[:3])
    with pytest.raises(ValueError):
        lsb.lora_q4_matmul(x.t().contiguous().t(), w, y)
    with pytest.raises(ValueError):
        lsb.lora_q4_matmul(x.cpu(), w, y)
