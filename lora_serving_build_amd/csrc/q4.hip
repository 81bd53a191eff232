// Packing of 4-bit weights and group scales (lora_q4_pack), and the launch of
// their products.
#include "decode_kernels.h"
#include "lora_device.h"

namespace lora {
namespace {

// ---------------------------------------------------------------- packing
// One thread per dword of codes; the first threads of a (tile, block) unit
// also write its scales and zeros.  Rows and inputs beyond the weight get code
// 8, scale 0 and zero 8.  Codes are read as dwords where they are aligned (28672
// x 8192: 92 us for 246 MB, 217 by bytes; a copy of as much takes 51).  A weight
// is packed once, when it is loaded.
__global__ void __launch_bounds__(256) q4_pack_kernel(const uint8_t* __restrict__ codes, int64_t ld_codes,
                                                      const uint16_t* __restrict__ scales, int64_t ld_scales,
                                                      const uint8_t* __restrict__ zeros, int64_t ld_zeros,
                                                      int32_t n, int32_t k, int32_t group, Q4Layout lay,
                                                      bool words, uint8_t* __restrict__ packed) {
  const int64_t unit = blockIdx.x;
  const int tile = (int)(unit / lay.blocks), block = (int)(unit % lay.blocks);
  const int d = threadIdx.x, lane = d >> 2, w = d & 3;
  const int row = tile * 16 + (lane & 15);
  const int h0 = block * 128 + w * 32 + (lane >> 4) * 8;
  uint32_t out = 0x88888888u;
  if (row < n && h0 < k) {
    const uint8_t* p = codes + (int64_t)row * ld_codes + h0 / 2;
    uint32_t eight;  // inputs h0 .. h0 + 7 in the order of the rows
    if (words && h0 + 8 <= k) {
      eight = *reinterpret_cast<const uint32_t*>(p);
    } else {
      eight = 0;
      for (int j = 0; j < 4; ++j) {
        uint32_t b = h0 + 2 * j < k ? p[j] : 0x88u;
        if (h0 + 2 * j + 1 >= k) b = (b & 15u) | 0x80u;
        eight |= b << (8 * j);
      }
    }
    out = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = eight >> (8 * j);
      out |= ((b & 15u) << (4 * j)) | (((b >> 4) & 15u) << (16 + 4 * j));
    }
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

}  // namespace

hipError_t launch_q4_pack(const uint8_t* codes, int64_t ld_codes, const uint16_t* scales, int64_t ld_scales,
                          const uint8_t* zeros, int64_t ld_zeros, int32_t n, int32_t k, int32_t group,
                          void* packed, hipStream_t s) {
  const Q4Layout lay = q4_layout(n, k, group, zeros != nullptr);
  const bool words = ((reinterpret_cast<uintptr_t>(codes) | (uintptr_t)ld_codes) & 3) == 0;  // dwords of codes are aligned
  q4_pack_kernel<<<dim3((unsigned)((int64_t)lay.tiles * lay.blocks)), 256, 0, s>>>(
      codes, ld_codes, scales, ld_scales, zeros, ld_zeros, n, k, group, lay, words, static_cast<uint8_t*>(packed));
  return hipGetLastError();
}

hipError_t launch_q4_matmul(const uint16_t* x, int64_t ldx, const void* packed, int32_t n, int32_t k,
                            int32_t group, bool zeros, int32_t T, uint16_t* y, int64_t ldy, int add,
                            int dtype, bool x_vec, bool y_vec, void* workspace, hipStream_t s) {
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
  a.sub = lay.sub;
  a.T = T;
  a.y = y;
  a.ldy = ldy;
  a.add = add;
  a.partial = static_cast<float*>(workspace);
  a.x_vec = x_vec ? 1 : 0;
  a.y_vec = y_vec ? 1 : 0;
  return dtype == 0 ? launch_q4_f16(a, lay.sub, s) : launch_q4_bf16(a, lay.sub, s);
}

}  // namespace lora
