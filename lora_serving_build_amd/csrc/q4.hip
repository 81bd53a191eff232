// Products with 4-bit weights and group scales (lora_q4_pack, lora_q4_matmul).
//
//   y[t, c] (+)= sum_g s[c, g] sum_{h in g} (q[c, h] - z[c, g]) x[t, h]
//
// The matrix cores take 16 rows of codes against 16 tokens: a code becomes a
// 16-bit number with two bit operations, so even one token is cheapest on
// them (the other 15 columns are free, and no sum over lanes is left).
#include "decode_kernels.h"
#include "lora_device.h"

namespace lora {
namespace {

// ---------------------------------------------------------------- packing
// One thread per dword of codes; the first threads of a (tile, block) unit
// also write its scales and zeros.  Rows and inputs beyond the weight get code
// 8, scale 0 and zero 8.
__global__ void __launch_bounds__(256) q4_pack_kernel(const uint8_t* __restrict__ codes, int64_t ld_codes,
                                                      const uint16_t* __restrict__ scales, int64_t ld_scales,
                                                      const uint8_t* __restrict__ zeros, int64_t ld_zeros,
                                                      int32_t n, int32_t k, int32_t group, Q4Layout lay,
                                                      uint8_t* __restrict__ packed) {
  const int64_t unit = blockIdx.x;
  const int tile = (int)(unit / lay.blocks), block = (int)(unit % lay.blocks);
  const int d = threadIdx.x, lane = d >> 2, w = d & 3;
  const int row = tile * 16 + (lane & 15);
  const int h0 = block * 128 + w * 32 + (lane >> 4) * 8;
  uint32_t out = 0;
  for (int j = 0; j < 4; ++j) {
    uint32_t lo = 8, hi = 8;
    const int h = h0 + 2 * j;
    if (row < n && h < k) {
      const uint32_t b = codes[(int64_t)row * ld_codes + h / 2];
      lo = b & 15u;
      if (h + 1 < k) hi = b >> 4;
    }
    out |= (lo << (4 * j)) | (hi << (16 + 4 * j));
  }
  reinterpret_cast<uint32_t*>(packed)[unit * 256 + d] = out;
  if (d < lay.sub * 16) {
    const int sub = d / 16, r = tile * 16 + d % 16;
    const int h = block * 128 + sub * (128 / lay.sub);
    const bool in = r < n && h < k;
    const int g = h / group;
    reinterpret_cast<uint16_t*>(packed + lay.scales_at)[unit * lay.sub * 16 + d] =
        in ? scales[(int64_t)r * ld_scales + g] : (uint16_t)0;
    if (zeros)
      (packed + lay.zeros_at)[unit * lay.sub * 16 + d] = in ? (uint8_t)(zeros[(int64_t)r * ld_zeros + g] & 15u) : 8;
  }
}

// ---------------------------------------------------------------- codes to 16-bit numbers
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) { return (a & mask) | bits; }

// The 8 codes of a dword as matrix-core operand elements.
// binary16: a code in bits 0..3 under the exponent of 1024 reads 1024 + q, one
// in bits 4..7 under the exponent of 64 reads 64 + q; a packed subtraction of
// 1024 + z or 64 + z leaves q - z exactly.  lo, hi: those two in both halves.
// bfloat16 has no packed subtraction: a code under the exponent of 128 reads
// 128 + q, and the caller takes (128 + z) sum x away from the sum.
template <int DT>
__device__ __forceinline__ u32x4 q4_numbers(uint32_t d, f16x2 lo, f16x2 hi) {
  if constexpr (DT == 0) {
    const uint32_t e = d >> 8;
    u32x4 r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, and_or(d, 0x000f000fu, 0x64006400u)) - lo);
    r.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, and_or(d, 0x00f000f0u, 0x54005400u)) - hi);
    r.z = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, and_or(e, 0x000f000fu, 0x64006400u)) - lo);
    r.w = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, and_or(e, 0x00f000f0u, 0x54005400u)) - hi);
    return r;
  } else {
    return u32x4{and_or(d, 0x000f000fu, 0x43004300u), and_or(d >> 4, 0x000f000fu, 0x43004300u),
                 and_or(d >> 8, 0x000f000fu, 0x43004300u), and_or(d >> 12, 0x000f000fu, 0x43004300u)};
  }
}

struct Q4Args {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* packed;
  int64_t scales_at, zeros_at;  // zeros_at = 0: every zero is 8
  int32_t n, k, tiles, blocks;
  int32_t T;
  uint16_t* y;
  int64_t ldy;
  int add;
  int y_vec;  // y rows of four outputs are 8-byte aligned and whole
};

// ---------------------------------------------------------------- product
// One workgroup: MT row tiles x NT token tiles, the blocks of k dealt out to
// its W waves in turn; the waves' sums meet in LDS and are added in wave
// order.  D of the matrix core: lane l holds outputs 4 (l / 16) + 0..3 of
// token l % 16.
template <int DT, int SUB, int MT, int NT, int W, bool VEC>
__global__ void __launch_bounds__(W* kWave) q4_kernel(Q4Args a) {
  __shared__ float sums[W][MT * NT][4][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, quad = lane >> 4;
  const int tile0 = blockIdx.x * MT;
  const int t0 = blockIdx.y * (16 * NT);

  // Tokens beyond T read the last row; their columns are not stored.
  const uint16_t* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = t0 + i * 16 + col;
    xr[i] = a.x + (int64_t)(t < a.T ? t : a.T - 1) * a.ldx;
  }
  // Row tiles beyond the last read the last one; their rows are not stored.
  int64_t unit0[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) unit0[m] = (int64_t)(tile0 + m < a.tiles ? tile0 + m : a.tiles - 1) * a.blocks;

  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int b = wave; b < a.blocks; b += W) {
    u32x4 xv[4][NT];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int h = b * 128 + s * 32 + quad * 8;
        if constexpr (VEC) {
          xv[s][i] = load8_16_masked(xr[i], h, a.k, true);
        } else {
          xv[s][i] = load8_16<false>(xr[i] + h, a.k - h);
        }
      }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t unit = unit0[m] + b;
      const u32x4 codes = reinterpret_cast<const u32x4*>(a.packed)[unit * 64 + lane];
#pragma unroll
      for (int g = 0; g < SUB; ++g) {
        const u32x2 sc = *reinterpret_cast<const u32x2*>(a.packed + a.scales_at + (unit * SUB + g) * 32 + quad * 8);
        f32x4 scale;
        float lo, hi;
        unpack2<DT>(sc.x, &lo, &hi);
        scale.x = lo;
        scale.y = hi;
        unpack2<DT>(sc.y, &lo, &hi);
        scale.z = lo;
        scale.w = hi;
        f16x2 z_lo{}, z_hi{};
        f32x4 base = f32x4{136.f, 136.f, 136.f, 136.f};
        if constexpr (DT == 0) {
          const uint32_t z = a.zeros_at ? a.packed[a.zeros_at + (unit * SUB + g) * 16 + col] : 8u;
          z_lo = __builtin_bit_cast(f16x2, 0x64006400u | z | (z << 16));
          z_hi = __builtin_bit_cast(f16x2, 0x54005400u | (z << 4) | (z << 20));
        } else if (a.zeros_at) {
          const uint32_t z = *reinterpret_cast<const uint32_t*>(a.packed + a.zeros_at + (unit * SUB + g) * 16 + quad * 4);
          base = f32x4{128.f + (float)(z & 255u), 128.f + (float)((z >> 8) & 255u),
                       128.f + (float)((z >> 16) & 255u), 128.f + (float)(z >> 24)};
        }
        f32x4 part[NT], xs[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) part[i] = xs[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = g * (4 / SUB); s < (g + 1) * (4 / SUB); ++s) {
          const u32x4 w = q4_numbers<DT>(codes[s], z_lo, z_hi);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            part[i] = mfma16x16x32<DT>(w, xv[s][i], part[i]);
            if constexpr (DT == 1) {
              const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
              xs[i] = mfma16x16x32<DT>(ones, xv[s][i], xs[i]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if constexpr (DT == 1) part[i] -= base * xs[i];
          acc[m][i] += scale * part[i];
        }
      }
    }
  }

#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sums[wave][m * NT + i][e][lane] = acc[m][i][e];
  __syncthreads();
  // One thread adds one output quad: MT * NT * 64 quads.
  for (int o = threadIdx.x; o < MT * NT * kWave; o += W * kWave) {
    const int l = o & (kWave - 1), mi = o / kWave, m = mi / NT, i = mi % NT;
    const int t = t0 + i * 16 + (l & 15);
    const int c = (tile0 + m) * 16 + (l >> 4) * 4;
    float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] += sums[w][mi][e][l];
    if (t >= a.T || c >= a.n) continue;
    uint16_t* y = a.y + (int64_t)t * a.ldy + c;
    if (a.y_vec) {
      if (a.add) {
        const u32x2 old = *reinterpret_cast<const u32x2*>(y);
        float p, q;
        unpack2<DT>(old.x, &p, &q);
        r[0] += p;
        r[1] += q;
        unpack2<DT>(old.y, &p, &q);
        r[2] += p;
        r[3] += q;
      }
      *reinterpret_cast<u32x2*>(y) = u32x2{cvt_pack2<DT>(r[0], r[1]), cvt_pack2<DT>(r[2], r[3])};
    } else {
      for (int e = 0; e < 4 && c + e < a.n; ++e)
        y[e] = (uint16_t)from_f32<DT>(r[e] + (a.add ? to_f32<DT>(y[e]) : 0.f));
    }
  }
}

template <int DT, int SUB, int NT>
hipError_t launch(const Q4Args& a, bool vec, hipStream_t s) {
  constexpr int MT = 1, W = 8;
  const dim3 grid((a.tiles + MT - 1) / MT, (a.T + 16 * NT - 1) / (16 * NT));
  if (vec)
    q4_kernel<DT, SUB, MT, NT, W, true><<<grid, W * kWave, 0, s>>>(a);
  else
    q4_kernel<DT, SUB, MT, NT, W, false><<<grid, W * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, int SUB>
hipError_t launch_nt(const Q4Args& a, bool vec, hipStream_t s) {
  return a.T <= 16 ? launch<DT, SUB, 1>(a, vec, s) : launch<DT, SUB, 2>(a, vec, s);
}

template <int DT>
hipError_t launch_sub(const Q4Args& a, int sub, bool vec, hipStream_t s) {
  switch (sub) {
    case 1: return launch_nt<DT, 1>(a, vec, s);
    case 2: return launch_nt<DT, 2>(a, vec, s);
    default: return launch_nt<DT, 4>(a, vec, s);
  }
}

}  // namespace

hipError_t launch_q4_pack(const uint8_t* codes, int64_t ld_codes, const uint16_t* scales, int64_t ld_scales,
                          const uint8_t* zeros, int64_t ld_zeros, int32_t n, int32_t k, int32_t group,
                          void* packed, hipStream_t s) {
  const Q4Layout lay = q4_layout(n, k, group, zeros != nullptr);
  q4_pack_kernel<<<dim3((unsigned)((int64_t)lay.tiles * lay.blocks)), 256, 0, s>>>(
      codes, ld_codes, scales, ld_scales, zeros, ld_zeros, n, k, group, lay, static_cast<uint8_t*>(packed));
  return hipGetLastError();
}

hipError_t launch_q4_matmul(const uint16_t* x, int64_t ldx, const void* packed, int32_t n, int32_t k,
                            int32_t group, bool zeros, int32_t T, uint16_t* y, int64_t ldy, int add,
                            int dtype, bool x_vec, bool y_vec, hipStream_t s) {
  const Q4Layout lay = q4_layout(n, k, group, zeros);
  Q4Args a;
  a.x = x;
  a.ldx = ldx;
  a.packed = static_cast<const uint8_t*>(packed);
  a.scales_at = (int64_t)lay.scales_at;
  a.zeros_at = zeros ? (int64_t)lay.zeros_at : 0;
  a.n = n;
  a.k = k;
  a.tiles = lay.tiles;
  a.blocks = lay.blocks;
  a.T = T;
  a.y = y;
  a.ldy = ldy;
  a.add = add;
  a.y_vec = y_vec ? 1 : 0;
  return dtype == 0 ? launch_sub<0>(a, lay.sub, x_vec, s) : launch_sub<1>(a, lay.sub, x_vec, s);
}

}  // namespace lora
