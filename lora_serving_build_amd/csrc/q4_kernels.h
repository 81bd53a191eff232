// Kernels of the products with 4-bit weights, and the choice between them.
//
//   y[t, c] (+)= sum_g s[c, g] sum_{h in g} (q[c, h] - z[c, g]) x[t, h]
//
// The matrix cores take 16 rows of codes against 16 tokens: a code becomes a
// 16-bit number with two bit operations, so even one token is cheapest on
// them (the other 15 columns are free, and no sum over lanes is left).
//
// Included by one source file for each type (q4_f16.hip, q4_bf16.hip).
#pragma once

#include <type_traits>

#include "decode_kernels.h"
#include "lora_device.h"

namespace lora {
namespace {

// ---------------------------------------------------------------- codes to 16-bit numbers
// The masks and exponents of q4_numbers.  v_and_or_b32 takes no literals and
// one scalar operand: with the masks in scalar and the exponents in vector
// registers it is one instruction; from constants the compiler makes two.
template <int DT>
struct Q4Bits {
  uint32_t low, high, low_exp, high_exp;
  __device__ __forceinline__ Q4Bits() {
    low = 0x000f000fu;
    high = 0x00f000f0u;
    low_exp = DT == 0 ? 0x64006400u : 0x43004300u;
    high_exp = 0x54005400u;
    asm("" : "+s"(low), "+s"(high));
    asm("" : "+v"(low_exp), "+v"(high_exp));
  }
};

// The 8 codes of a dword as matrix-core operand elements.
// binary16: a code in bits 0..3 under the exponent of 1024 reads 1024 + q, one
// in bits 4..7 under the exponent of 64 reads 64 + q; a packed subtraction of
// 1024 + z or 64 + z leaves q - z exactly.  lo, hi: those two in both halves.
// bfloat16 has no packed subtraction: a code under the exponent of 128 reads
// 128 + q, and the caller takes (128 + z) sum x away from the sum.
template <int DT>
__device__ __forceinline__ u32x4 q4_numbers(uint32_t d, const Q4Bits<DT>& k, f16x2 lo, f16x2 hi) {
  if constexpr (DT == 0) {
    const uint32_t e = d >> 8;
    u32x4 r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (d & k.low) | k.low_exp) - lo);
    r.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (d & k.high) | k.high_exp) - hi);
    r.z = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (e & k.low) | k.low_exp) - lo);
    r.w = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (e & k.high) | k.high_exp) - hi);
    return r;
  } else {
    return u32x4{(d & k.low) | k.low_exp, ((d >> 4) & k.low) | k.low_exp, ((d >> 8) & k.low) | k.low_exp,
                 ((d >> 12) & k.low) | k.low_exp};
  }
}

// ---------------------------------------------------------------- scales, zeros, results
// Codes of MT row tiles for one block of 128 inputs, with scales and zeros.
template <int SUB, int MT>
struct Q4Codes {
  u32x4 codes[MT];
  u32x2 scales[MT][SUB];
  uint32_t zeros[MT][SUB];
};

template <int DT, int SUB, bool ZEROS, int MT>
__device__ __forceinline__ void q4_load(const Q4Args& a, const int64_t (&unit0)[MT], int b, int lane,
                                        Q4Codes<SUB, MT>* r) {
  const int col = lane & 15, quad = lane >> 4;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t unit = unit0[m] + b;
    r->codes[m] = reinterpret_cast<const u32x4*>(a.packed)[unit * 64 + lane];
#pragma unroll
    for (int g = 0; g < SUB; ++g) {
      r->scales[m][g] = *reinterpret_cast<const u32x2*>(a.packed + a.scales_at + (unit * SUB + g) * 32 + quad * 8);
      if constexpr (ZEROS) {
        const uint8_t* z = a.packed + a.zeros_at + (unit * SUB + g) * 16;
        r->zeros[m][g] = DT == 0 ? (uint32_t)z[col] : *reinterpret_cast<const uint32_t*>(z + quad * 4);
      } else {
        r->zeros[m][g] = DT == 0 ? 8u : 0x08080808u;
      }
    }
  }
}

// A sub-group's scales as the results hold rows (4 quad + e), and what the
// codes' zeros become: the operand rows' in binary16, the results' in bfloat16.
template <int DT>
struct Q4Scale {
  f32x4 scale, base;
  f16x2 z_lo, z_hi;
};

template <int DT>
__device__ __forceinline__ Q4Scale<DT> q4_scale(u32x2 scales, uint32_t z) {
  Q4Scale<DT> r;
  float lo, hi;
  unpack2<DT>(scales.x, &lo, &hi);
  r.scale.x = lo;
  r.scale.y = hi;
  unpack2<DT>(scales.y, &lo, &hi);
  r.scale.z = lo;
  r.scale.w = hi;
  if constexpr (DT == 0) {
    r.base = f32x4{0.f, 0.f, 0.f, 0.f};
    r.z_lo = __builtin_bit_cast(f16x2, 0x64006400u | z | (z << 16));
    r.z_hi = __builtin_bit_cast(f16x2, 0x54005400u | (z << 4) | (z << 20));
  } else {
    r.z_lo = r.z_hi = f16x2{};
    r.base = f32x4{128.f + (float)(z & 255u), 128.f + (float)((z >> 8) & 255u), 128.f + (float)((z >> 16) & 255u),
                   128.f + (float)(z >> 24)};
  }
  return r;
}

// bfloat16 takes (128 + z) sum x away from sum (128 + q) x.  Where x is infinite
// or its sums pass fp32's range that is inf - inf, although sum (q - z) x is an
// infinity with a sign, or in range.  Results that are not finite are therefore
// taken again, from the definition, in 64 bits.  That costs nothing where all are
// finite, little where a token has a NaN (which decides all of its results), and
// milliseconds where one has infinities (4 for 28672 x 8192).
__device__ __forceinline__ bool q4_finite(f32x4 r) {
  return fabsf(r.x) + fabsf(r.y) + fabsf(r.z) + fabsf(r.w) < INFINITY;
}

// Outputs c .. c + 3 (those below n) of token t for the lanes that need them.
// Every lane of the wave calls it.
__device__ __forceinline__ f32x4 q4_again(const Q4Args& a, int lane, bool needed, int t, int c) {
  bool nan = false;
  for (uint64_t left = __ballot(needed); left;) {  // token after token
    const int token = __builtin_amdgcn_readlane(t, __ffsll((unsigned long long)left) - 1);
    const uint16_t* x = a.x + (int64_t)token * a.ldx;
    bool found = false;
    for (int h0 = 0; h0 < a.k && !__any(found); h0 += 16 * kWave)
#pragma unroll
      for (int j = 0; j < 16; ++j) found |= (x[min(h0 + j * kWave + lane, a.k - 1)] & 0x7fffu) > 0x7f80u;
    nan |= __any(found) && t == token;
    left &= ~__ballot(t == token);
  }
  if (!needed) return f32x4{0.f, 0.f, 0.f, 0.f};
  if (nan) return f32x4{NAN, NAN, NAN, NAN};
  const uint16_t* x = a.x + (int64_t)t * a.ldx;
  const int per_scale = 128 / a.sub;
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int e = 0; e < 4 && c + e < a.n; ++e) {
    const int tile = (c + e) / 16, row = (c + e) % 16;
    double sum = 0;
#pragma unroll 1
    for (int h0 = 0; h0 < a.k && sum == sum; h0 += 8) {
      // Eight inputs: a dword as packed, one scale.
      const int64_t unit = (int64_t)tile * a.blocks + h0 / 128;
      const int in = h0 % 128, w = in / 32, quad = in / 8 % 4;
      const uint32_t d = reinterpret_cast<const uint32_t*>(a.packed)[unit * 256 + (row + 16 * quad) * 4 + w];
      const int64_t at = (unit * a.sub + in / per_scale) * 16 + row;
      const int z = a.zeros_at ? a.packed[a.zeros_at + at] : 8;
      const float scale = to_f32<1>(reinterpret_cast<const uint16_t*>(a.packed + a.scales_at)[at]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = h0 + j < a.k ? to_f32<1>(x[h0 + j]) : 0.f;
        const int q = (d >> (j / 2 * 4 + j % 2 * 16)) & 15u;
        if (h0 + j < a.k) sum += (double)((float)(q - z) * scale) * (double)v;
      }
    }
    if (e == 0) r.x = (float)sum;
    if (e == 1) r.y = (float)sum;
    if (e == 2) r.z = (float)sum;
    if (e == 3) r.w = (float)sum;
  }
  return r;
}

// Outputs c .. c + 3 of token t (those below n).
template <int DT>
__device__ __forceinline__ void q4_store(const Q4Args& a, int t, int c, f32x4 r) {
  uint16_t* y = a.y + (int64_t)t * a.ldy + c;
  if (a.y_vec) {
    if (c >= a.n) return;
    if (a.add) {
      const u32x2 old = *reinterpret_cast<const u32x2*>(y);
      float p, q;
      unpack2<DT>(old.x, &p, &q);
      r.x += p;
      r.y += q;
      unpack2<DT>(old.y, &p, &q);
      r.z += p;
      r.w += q;
    }
    *reinterpret_cast<u32x2*>(y) = u32x2{cvt_pack2<DT>(r.x, r.y), cvt_pack2<DT>(r.z, r.w)};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < a.n) y[e] = (uint16_t)from_f32<DT>(r[e] + (a.add ? to_f32<DT>(y[e]) : 0.f));
  }
}

// ---------------------------------------------------------------- product
// For few tokens or a small weight: one workgroup takes MT row tiles and 16 NT
// tokens, the blocks of k dealt out to its eight waves in turn; the waves' sums
// meet in LDS and are added in wave order, so there is one launch and no
// workspace.  D of the
// matrix core: lane l holds outputs 4 (l / 16) + 0..3 of token l % 16.
// Bound by memory for wide weights (28672 x 8192, groups of 128 with zeros, 4
// tokens: 30 us, 123 MB, 4.1 TB/s; 25 us where the last call left the weight in
// the last-level cache), by what the L2s deliver of x for more tokens, by
// latencies for small ones (1024 x 4096, one token: 3.9 us).  More waves carry
// it better than loads further ahead: two or three blocks in flight a wave cost
// registers and measured up to half as slow again.
constexpr int kWavesPerTile = 8;

template <int DT, int SUB, bool ZEROS, int MT, int NT, bool VEC>
__global__ void __launch_bounds__(kWavesPerTile* kWave) q4_kernel(Q4Args a) {
  constexpr int W = kWavesPerTile;
  __shared__ __align__(16) f32x4 sums[W][MT * NT][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, quad = lane >> 4;
  const int tile0 = blockIdx.x * MT, t0 = blockIdx.y * (16 * NT);
  const Q4Bits<DT> bits;
  // Tokens beyond T read the last row; their columns are not stored.
  const uint16_t* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xr[i] = a.x + (int64_t)min(t0 + i * 16 + col, a.T - 1) * a.ldx;
  // Row tiles beyond the last read the last one; their rows are not stored.
  int64_t unit0[MT];
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    unit0[m] = (int64_t)(tile0 + m < a.tiles ? tile0 + m : a.tiles - 1) * a.blocks;
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (int b = wave; b < a.blocks; b += W) {
    Q4Codes<SUB, MT> r;
    q4_load<DT, SUB, ZEROS, MT>(a, unit0, b, lane, &r);
    u32x4 x[NT][4];
    const int h = b * 128 + quad * 8;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int at = h + s * 32;
        x[i][s] = VEC ? *reinterpret_cast<const u32x4*>(xr[i] + (at < a.k ? at : a.k - 8)) : load8_16<false>(xr[i] + at, a.k - at);
      }
    if (VEC && (b + 1) * 128 > a.k) {  // inputs beyond k
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (h + s * 32 >= a.k) x[i][s] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int g = 0; g < SUB; ++g) {
      f32x4 xs[NT];
      if constexpr (DT == 1) {  // sums of x, in every row
        const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          xs[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = g * (4 / SUB); s < (g + 1) * (4 / SUB); ++s) xs[i] = mfma16x16x32<DT>(ones, x[i][s], xs[i]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const Q4Scale<DT> sc = q4_scale<DT>(r.scales[m][g], r.zeros[m][g]);
        f32x4 part[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) part[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = g * (4 / SUB); s < (g + 1) * (4 / SUB); ++s) {
          const u32x4 w = q4_numbers<DT>(r.codes[m][s], bits, sc.z_lo, sc.z_hi);
#pragma unroll
          for (int i = 0; i < NT; ++i) part[i] = mfma16x16x32<DT>(w, x[i][s], part[i]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (DT == 1) part[i][e] = __builtin_fmaf(-sc.base[e], xs[i][e], part[i][e]);
            acc[m][i][e] = __builtin_fmaf(sc.scale[e], part[i][e], acc[m][i][e]);
          }
      }
    }
  }

#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) sums[wave][m * NT + i][lane] = acc[m][i];
  __syncthreads();
  for (int o = threadIdx.x; o < MT * NT * kWave; o += W * kWave) {
    const int l = o & (kWave - 1), mi = o / kWave, m = mi / NT, t = t0 + mi % NT * 16 + (l & 15);
    f32x4 r = sums[0][mi][l];
#pragma unroll
    for (int w = 1; w < W; ++w) r += sums[w][mi][l];
    const int c = (tile0 + m) * 16 + (l >> 4) * 4;
    if constexpr (DT == 1) {
      const bool again = t < a.T && c < a.n && !q4_finite(r);
      if (__any(again)) {
        const f32x4 exact = q4_again(a, l, again, t, c);
        if (again) r = exact;
      }
    }
    if (t < a.T) q4_store<DT>(a, t, c, r);
  }
}

// ---------------------------------------------------------------- product with shared x
// For more than a few tokens x is read as often as the weight or more: each
// row tile of codes (8 k bytes) meets 2 T k bytes of it.  Here the eight waves
// of a workgroup take row tiles of their own (MT each) and share x through
// LDS, in the order in which the matrix core takes it, double-buffered; the
// next chunk's x is on its way in registers, the next block's codes too.  The
// workgroups of one row group split k, and a second kernel adds their sums in
// order.  The sums of x that a bfloat16 product needs are taken while x is
// staged.
// 8192 outputs of 28672 inputs, groups of 64, 16 tokens: 31 us for 126 MB (4.1
// TB/s; 26 us from the last-level cache) and 5 us for the sums of 8 splits; waves
// that split k need 38.  128 tokens, 8192 x 8192: 36 us, 480 TFLOP/s, bound by the
// reads of x from LDS and the scaling of the sub-groups' sums.  Groups of 32 with
// zeros spill: 28 registers in bfloat16 for 128 tokens, 11 for 16 (14 without
// splits), and 5 in binary16 for 16.
constexpr int kShareWaves = 8;

// AGAIN: results that are not finite are taken again here (bfloat16 without
// splits; with splits the kernel that adds them does it, and this one keeps its
// registers: 128 tokens, groups of 64: 39 us against 44).
template <int DT, int SUB, bool ZEROS, int MT, int NT, bool AGAIN>
__global__ void __launch_bounds__(kShareWaves* kWave, NT <= 2 ? 4 : 2) q4_shared_kernel(Q4Args a, int splits) {
  constexpr int CB = NT >= 8 ? 1 : 8 / NT;  // blocks of a chunk: up to 32 KiB of x
  constexpr int OPS = CB * NT * 4;          // operands of 16 tokens x 32 inputs
  constexpr int MINE = (OPS + kShareWaves - 1) / kShareWaves;
  __shared__ __align__(16) u32x4 xs[2][MINE * kShareWaves][kWave];
  __shared__ float sums[DT == 1 ? 2 : 1][DT == 1 ? MINE * kShareWaves : 1][16];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, quad = lane >> 4;
  const int tile0 = (blockIdx.x / splits * kShareWaves + wave) * MT, split = blockIdx.x % splits;
  const int t0 = blockIdx.y * (16 * NT);
  const int first = (int)((int64_t)a.blocks * split / splits), last = (int)((int64_t)a.blocks * (split + 1) / splits);
  const Q4Bits<DT> bits;

  int64_t unit0[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) unit0[m] = (int64_t)(tile0 + m < a.tiles ? tile0 + m : a.tiles - 1) * a.blocks;

  // Operand f of a chunk: 16-token tile f / 4 % NT, step f % 4 of its block
  // f / (4 NT).  This wave stages operands wave, wave + 8, ...; what lies beyond
  // the split, or beyond the chunk's operands, is staged too and not used
  // (nothing here is conditional: the compiler would move the loads into the
  // conditions, where each waits for the one before).
  u32x4 xreg[MINE];
  auto fetch_as = [&](int chunk, auto vec) {
#pragma unroll
    for (int j = 0; j < MINE; ++j) {
      const int f = wave + j * kShareWaves;
      const int b = min(first + chunk * CB + f / (4 * NT), last - 1), t = t0 + f / 4 % NT * 16 + col;
      const int h = b * 128 + f % 4 * 32 + quad * 8;
      const uint16_t* row = a.x + (int64_t)(t < a.T ? t : a.T - 1) * a.ldx;
      xreg[j] = vec ? *reinterpret_cast<const u32x4*>(row + (h < a.k ? h : a.k - 8)) : load8_16<false>(row + h, a.k - h);
    }
  };
  auto fetch = [&](int chunk) {
    if (a.x_vec)
      fetch_as(chunk, std::true_type());
    else
      fetch_as(chunk, std::false_type());
  };
  auto stash = [&](int chunk) {
#pragma unroll
    for (int j = 0; j < MINE; ++j) {
      const int f = wave + j * kShareWaves;
      // Inputs beyond k read as 0 (here and not in the fetch, which would wait
      // for its loads there).
      if ((first + chunk * CB + f / (4 * NT) + 1) * 128 > a.k && (first + chunk * CB + f / (4 * NT)) * 128 + f % 4 * 32 + quad * 8 >= a.k)
        xreg[j] = u32x4{0u, 0u, 0u, 0u};
      xs[chunk & 1][f][lane] = xreg[j];
      if constexpr (DT == 1) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          unpack2<DT>(xreg[j][e], &lo, &hi);
          sum += lo + hi;
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        sums[chunk & 1][f][col] = sum;  // four lanes, one value
      }
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  Q4Codes<SUB, MT> next;
  fetch(0);
  q4_load<DT, SUB, ZEROS, MT>(a, unit0, first, lane, &next);
  stash(0);
  fetch(1);
  __syncthreads();
  const int chunks = (last - first + CB - 1) / CB;
  for (int c = 0; c < chunks; ++c) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const int b = first + c * CB + cb;
      if (b >= last) break;
      const Q4Codes<SUB, MT> now = next;
      q4_load<DT, SUB, ZEROS, MT>(a, unit0, min(b + 1, last - 1), lane, &next);
      __builtin_amdgcn_sched_barrier(0);  // the next codes leave before this block's products
#pragma unroll
      for (int g = 0; g < SUB; ++g) {
        f32x4 part[MT][NT];
        Q4Scale<DT> sc[MT];
        float total[NT];
#pragma unroll
        for (int m = 0; m < MT; ++m) sc[m] = q4_scale<DT>(now.scales[m][g], now.zeros[m][g]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          total[i] = 0.f;
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int s = g * (4 / SUB); s < (g + 1) * (4 / SUB); ++s) {
          u32x4 w[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) w[m] = q4_numbers<DT>(now.codes[m][s], bits, sc[m].z_lo, sc[m].z_hi);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const int f = (cb * NT + i) * 4 + s;
            const u32x4 x = xs[c & 1][f][lane];
#pragma unroll
            for (int m = 0; m < MT; ++m) part[m][i] = mfma16x16x32<DT>(w[m], x, part[m][i]);
            if constexpr (DT == 1) total[i] += sums[c & 1][f][col];
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (DT == 1) part[m][i][e] = __builtin_fmaf(-sc[m].base[e], total[i], part[m][i][e]);
              acc[m][i][e] = __builtin_fmaf(sc[m].scale[e], part[m][i][e], acc[m][i][e]);
            }
      }
    }
    if (c + 1 == chunks) break;
    stash(c + 1);
    fetch(c + 2);
    __syncthreads();
  }

  uint32_t again = 0;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = (tile0 + m) * 16 + quad * 4;
    if (tile0 + m >= a.tiles) continue;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = t0 + i * 16 + col;
      if (t >= a.T) continue;
      if (!AGAIN && splits > 1)
        *reinterpret_cast<f32x4*>(a.partial + ((int64_t)split * a.T + t) * (a.tiles * 16) + row) = acc[m][i];
      else if (!AGAIN || q4_finite(acc[m][i]))
        q4_store<DT>(a, t, row, acc[m][i]);
      else
        again |= 1u << (m * NT + i);
    }
  }
  if constexpr (AGAIN) {
#pragma unroll 1
    for (int mi = 0; mi < MT * NT && __any(again >> mi); ++mi) {
      const bool mine = (again >> mi) & 1;
      if (!__any(mine)) continue;
      const int row = (tile0 + mi / NT) * 16 + quad * 4, t = t0 + mi % NT * 16 + col;
      const f32x4 exact = q4_again(a, lane, mine, t, row);
      if (mine) q4_store<DT>(a, t, row, exact);
    }
  }
}

// y from the sums of the splits, four outputs a thread.  4 to 5 us, most of it
// the launch and two memory latencies.
template <int DT>
__global__ void __launch_bounds__(256) q4_add_kernel(Q4Args a, int splits) {
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4, t = blockIdx.x;
  const bool in = c < a.n;
  const int64_t width = (int64_t)a.tiles * 16;
  const float* p = a.partial + t * width + (in ? c : 0);
  f32x4 sum = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 4
  for (int s = 1; s < splits; ++s) sum += *reinterpret_cast<const f32x4*>(p + s * a.T * width);
  if constexpr (DT == 1) {
    const bool again = in && !q4_finite(sum);
    if (__any(again)) {
      const f32x4 exact = q4_again(a, threadIdx.x & (kWave - 1), again, t, c);
      if (again) sum = exact;
    }
  }
  if (in) q4_store<DT>(a, t, c, sum);
}

// ---------------------------------------------------------------- launch
// How a product is run.
struct Q4Plan {
  bool shared;   // x through LDS, k split over workgroups
  int mt, nt;    // row tiles and token tiles of a workgroup (of a wave, if shared)
  int splits;
};

// The cheapest of the kernels' forms by a cost in microseconds, fitted to
// timings of all of them for 2 to 128 tokens, 1024 x 4096 to 28672 x 8192, one
// sub-group of zeros a block in bfloat16 and four in binary16.
//
// Waves that split k: 4, and a round of 256 workgroups takes an eighth of the
// blocks at `step` each.  The wider forms read x and the codes less often but
// leave fewer workgroups; four sub-groups a block cost more scales and sums.
// Waves that share x: 10 (two launches, the sums written and read), and one of
// the splits' blocks at `step` each.
// Measured, microseconds, first against second kind, best forms: 4096 x 4096,
// 64 tokens 8.7 / 14.8; 5003 x 4064, 77 tokens 16 / 20; 8192 x 8192, 16 tokens
// 12.1 / 12.6, 128 tokens 43 / 38; 8192 outputs of 28672, 16 tokens 37 / 32;
// 28672 x 8192, 4 tokens 27 / 30, 64 tokens 85 / 60.
inline Q4Plan q4_plan(int32_t T, int32_t tiles, int32_t blocks, int sub) {
  struct Form {
    int mt, nt;
    double step, step4;  // with up to two sub-groups a block, with four
  };
  static const Form split_k[] = {{1, 1, 0.70, 0.80}, {2, 1, 0.85, 1.25}, {4, 1, 1.20, 2.10},
                                 {4, 2, 2.20, 3.10}, {4, 3, 3.00, 4.00}};
  static const Form share_x[] = {{2, 1, 0.60, 0.65}, {1, 2, 0.50, 0.65}, {2, 4, 1.55, 1.80},
                                 {2, 6, 2.30, 2.80}, {2, 8, 3.60, 4.00}};
  Q4Plan best{false, 1, 1, 1};
  double least = 0;
  for (const Form& f : split_k) {
    const int64_t passes = (T + 16 * f.nt - 1) / (16 * f.nt), wgs = (tiles + f.mt - 1) / f.mt * passes;
    const double cost = 4 + (double)((wgs + 255) / 256) * ((blocks + kWavesPerTile - 1) / kWavesPerTile) *
                                (sub == 4 ? f.step4 : f.step);
    if (least == 0 || cost < least) {
      least = cost;
      best = Q4Plan{false, f.mt, f.nt, 1};
    }
  }
  for (const Form& f : share_x) {
    // The form that just holds T; above 128 tokens the widest, in passes.
    if (16 * f.nt < T && f.nt < 8) continue;
    // As many workgroups as CUs at most, so that none gets a second one while
    // others wait; where that leaves one split, two workgroups a CU if they fit
    // (up to 32 tokens).  Each split has four blocks at least.  512 row tiles, 16
    // tokens, k = 28672: 33 us with 8 splits (256 workgroups), 42 with 10.
    const int64_t passes = (T + 16 * f.nt - 1) / (16 * f.nt);
    const int64_t groups = (tiles + f.mt * kShareWaves - 1) / (f.mt * kShareWaves) * passes;
    int64_t splits = 256 / groups;
    if (splits <= 1 && f.nt <= 2) splits = 512 / groups;
    if (splits > blocks / 4) splits = blocks / 4;
    if (splits < 1) splits = 1;
    const double cost = (splits > 1 ? 10 : 6) + (double)((groups * splits + 255) / 256) *
                                                    ((blocks + splits - 1) / splits) * (sub == 4 ? f.step4 : f.step);
    if (cost < least) {
      least = cost;
      best = Q4Plan{true, f.mt, f.nt, (int)splits};
    }
    break;
  }
  return best;
}

template <int DT, int SUB, bool ZEROS, int MT, int NT>
hipError_t launch_tiles(const Q4Args& a, hipStream_t s) {
  const dim3 grid((a.tiles + MT - 1) / MT, (a.T + 16 * NT - 1) / (16 * NT));
  if (a.x_vec)
    q4_kernel<DT, SUB, ZEROS, MT, NT, true><<<grid, kWavesPerTile * kWave, 0, s>>>(a);
  else
    q4_kernel<DT, SUB, ZEROS, MT, NT, false><<<grid, kWavesPerTile * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, int SUB, bool ZEROS, int MT, int NT>
hipError_t launch_shared(const Q4Args& a, int splits, hipStream_t s) {
  const int groups = (a.tiles + MT * kShareWaves - 1) / (MT * kShareWaves);
  const dim3 grid(groups * splits, (a.T + 16 * NT - 1) / (16 * NT));
  if (DT == 1 && splits == 1)
    q4_shared_kernel<DT, SUB, ZEROS, MT, NT, DT == 1><<<grid, kShareWaves * kWave, 0, s>>>(a, splits);
  else
    q4_shared_kernel<DT, SUB, ZEROS, MT, NT, false><<<grid, kShareWaves * kWave, 0, s>>>(a, splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  q4_add_kernel<DT><<<dim3(a.T, (a.n + 1023) / 1024), 256, 0, s>>>(a, splits);
  return hipGetLastError();
}

template <int DT, int SUB, bool ZEROS>
hipError_t launch_plan(const Q4Args& a, hipStream_t s) {
  const Q4Plan p = q4_plan(a.T, a.tiles, a.blocks, SUB);
  switch ((p.shared ? 64 : 0) + p.nt * 4 + p.mt - 1) {
    case 1 * 4 + 0: return launch_tiles<DT, SUB, ZEROS, 1, 1>(a, s);
    case 1 * 4 + 1: return launch_tiles<DT, SUB, ZEROS, 2, 1>(a, s);
    case 1 * 4 + 3: return launch_tiles<DT, SUB, ZEROS, 4, 1>(a, s);
    case 2 * 4 + 3: return launch_tiles<DT, SUB, ZEROS, 4, 2>(a, s);
    case 3 * 4 + 3: return launch_tiles<DT, SUB, ZEROS, 4, 3>(a, s);
    case 64 + 1 * 4 + 1: return launch_shared<DT, SUB, ZEROS, 2, 1>(a, p.splits, s);
    case 64 + 2 * 4 + 0: return launch_shared<DT, SUB, ZEROS, 1, 2>(a, p.splits, s);
    case 64 + 4 * 4 + 1: return launch_shared<DT, SUB, ZEROS, 2, 4>(a, p.splits, s);
    case 64 + 6 * 4 + 1: return launch_shared<DT, SUB, ZEROS, 2, 6>(a, p.splits, s);
    case 64 + 8 * 4 + 1: return launch_shared<DT, SUB, ZEROS, 2, 8>(a, p.splits, s);
  }
  return hipErrorInvalidValue;  // not reached
}

template <int DT>
hipError_t launch_type(const Q4Args& a, int sub, hipStream_t s) {
  if (a.zeros_at) {
    if (sub == 1) return launch_plan<DT, 1, true>(a, s);
    return sub == 2 ? launch_plan<DT, 2, true>(a, s) : launch_plan<DT, 4, true>(a, s);
  }
  if (sub == 1) return launch_plan<DT, 1, false>(a, s);
  return sub == 2 ? launch_plan<DT, 2, false>(a, s) : launch_plan<DT, 4, false>(a, s);
}

}  // namespace
}  // namespace lora
