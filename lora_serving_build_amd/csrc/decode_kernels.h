// Launchers of the decode-step kernels (4-bit products, tree attention, page
// operations), called by the C-ABI layer (decode_api.hip) after it has
// validated every argument.  They return the hipError_t of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lora {

// ---------------------------------------------------------------- 4-bit products
// Packed form of a weight: three sections, each indexed by (row tile of 16
// outputs, block of 128 inputs), the block index running fastest.
//   codes   1024 bytes: lane l of a wave owns 16 bytes, its four dwords being
//           the four 32-input steps of the block; dword w holds the codes of
//           row l % 16, inputs 32 w + 8 (l / 16) + 0..7, input 2 j in bits
//           4 j.. and input 2 j + 1 in bits 16 + 4 j..
//   scales  sub x 16 values of 16 bits, one row of 16 for each of the block's
//           sub-groups (sub = 1, 2 or 4 sub-groups of 128, 64 or 32 inputs;
//           a group wider than that repeats its scale)
//   zeros   sub x 16 bytes, the same order
struct Q4Layout {
  int32_t tiles, blocks, sub;
  size_t scales_at, zeros_at, bytes;
};

inline Q4Layout q4_layout(int32_t n, int32_t k, int32_t group, bool zeros) {
  Q4Layout l;
  l.tiles = (n + 15) / 16;
  l.blocks = (k + 127) / 128;
  l.sub = group % 128 == 0 ? 1 : group % 64 == 0 ? 2 : 4;
  const size_t units = (size_t)l.tiles * (size_t)l.blocks;
  l.scales_at = units * 1024;
  l.zeros_at = l.scales_at + units * (size_t)l.sub * 32;
  l.bytes = l.zeros_at + (zeros ? units * (size_t)l.sub * 16 : 0);
  return l;
}

struct Q4Args {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* packed;
  int64_t scales_at, zeros_at;  // zeros_at = 0: every zero is 8
  int32_t n, k, tiles, blocks, sub;
  int32_t T;
  uint16_t* y;
  int64_t ldy;
  int add;
  float* partial;  // sums of the splits, [splits][T][16 tiles]
  int x_vec;  // x rows are 16-byte aligned and k a multiple of 8
  int y_vec;  // y rows of four outputs are 8-byte aligned and whole
};

hipError_t launch_q4_f16(const Q4Args& a, int sub, hipStream_t s);
hipError_t launch_q4_bf16(const Q4Args& a, int sub, hipStream_t s);

// Bytes of the splits' sums of a product (0: it does not split k).
size_t q4_workspace(int32_t T, int32_t n, int32_t k, int32_t group);

hipError_t launch_q4_pack(const uint8_t* codes, int64_t ld_codes, const uint16_t* scales, int64_t ld_scales,
                          const uint8_t* zeros, int64_t ld_zeros, int32_t n, int32_t k, int32_t group,
                          void* packed, hipStream_t s);

// x_vec: x is 16-byte aligned, ldx and k are multiples of 8; y_vec: y is
// 8-byte aligned, ldy and n are multiples of 4.
hipError_t launch_q4_matmul(const uint16_t* x, int64_t ldx, const void* packed, int32_t n, int32_t k,
                            int32_t group, bool zeros, int32_t T, uint16_t* y, int64_t ldy, int add,
                            int dtype, bool x_vec, bool y_vec, void* workspace, hipStream_t s);

// ---------------------------------------------------------------- pages
constexpr int kMaxPageEntries = 2048;
constexpr int kMaxPath = 256;

// lora_page_cache as the kernels take it.
struct PageView {
  uint8_t* pool;
  int64_t pool_stride, page_stride, row_bytes;
  int32_t chunks, num_pools, num_pages, page_size;
  int32_t* refs;
  int32_t* table;
  int64_t ld_table;
  int32_t max_seqs, max_pages;
  int32_t* seq_len;
};

struct AppendArgs {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_token, k_head, v_token, v_head;
  int32_t k_pool, v_pool, heads, dim;
  const int32_t* seqs;
  const int32_t* start;
  int32_t n;
};

size_t fork_workspace(int32_t n, int32_t max_pages);
size_t compact_workspace(int32_t num_pages);

hipError_t launch_pages_resize(const PageView& c, const int32_t* seqs, const int32_t* lens, const int32_t* extra,
                               int32_t n, int32_t* status, hipStream_t s);
hipError_t launch_pages_copy(const PageView& c, const int32_t* src, const int32_t* dst, int32_t n, hipStream_t s);
hipError_t launch_pages_fork(const PageView& c, const int32_t* src, const int32_t* dst, int32_t n, int32_t* status,
                             void* workspace, hipStream_t s);
hipError_t launch_pages_free(const PageView& c, const int32_t* seqs, int32_t n, hipStream_t s);
hipError_t launch_pages_append(const PageView& c, const AppendArgs& a, int32_t T, hipStream_t s);
hipError_t launch_pages_accept(const PageView& c, const int32_t* seqs, const int32_t* drafted, const int32_t* path,
                               int64_t ld_path, int32_t columns, const int32_t* accepted, int32_t n, int32_t* new_len,
                               hipStream_t s);
hipError_t launch_pages_compact(const PageView& c, int32_t* live, void* workspace, hipStream_t s);

// ---------------------------------------------------------------- tree attention
struct AttnArgs {
  const uint16_t* q;
  int64_t q_token, q_head;
  const uint16_t* k;
  const uint16_t* v;
  int64_t kv_page, kv_token, kv_head;
  int32_t num_pages, page_size;
  uint32_t page_mul, page_shift;  // set by the launcher: division by page_size
  const int32_t* table;
  int64_t ld_table;
  int32_t max_pages;
  const int32_t* ctx;
  const int32_t* start;
  const uint64_t* mask;  // NULL: node i sees nodes 0..i
  int64_t ld_mask;
  int32_t mask_words;
  uint16_t* out;
  int64_t out_token, out_head;
  float* lse;  // [T][heads] or NULL
  int32_t B, T, heads, kv_heads, dim;
  float scale_log2;    // scale times log2 e
  float* partial;      // workspace
};

// Threads of the call's largest launch, of a table of `positions` in a row.
int64_t attention_threads(int32_t B, int32_t T, int32_t heads, int32_t kv_heads, int32_t dim, int64_t positions);
size_t attention_workspace(int32_t B, int32_t T, int32_t heads, int32_t kv_heads, int32_t dim);
hipError_t launch_attention(const AttnArgs& a, int dtype, hipStream_t s);

}  // namespace lora
