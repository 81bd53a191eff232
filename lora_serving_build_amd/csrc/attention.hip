// Attention of a step's drafted tokens over a paged cache (lora_tree_attention).
//
//   o[i, h] = sum_p w_p v[p] / sum_p w_p,  w_p = 2^(scale log2(e) q[i, h] . k[p] - m)
//
// Rows: the nodes of a sequence times the G = heads / kv_heads query heads that
// share a key head, so one pass over the keys serves all of them.  A workgroup
// takes 16 RT rows of one (sequence, key head) and a run of positions; its four
// waves take 32 positions each in turn, with a running maximum and sum of their
// own, and meet in LDS at the end.  Long sequences are cut into several runs
// (so that few rows still fill the GPU); a second kernel joins those.
#include "decode_kernels.h"
#include "lora_device.h"

namespace lora {
namespace {

constexpr int kWaves = 4;
constexpr int kKeys = 32;                 // positions of one wave's step
constexpr int kTile = kWaves * kKeys;     // positions of one workgroup's step
constexpr int kCus = 256;

__device__ __forceinline__ bool in_range(int32_t v, int32_t n) { return (uint32_t)v < (uint32_t)n; }

// ---------------------------------------------------------------- work items
// A sequence as the kernels see it, whatever the buffers hold.
struct Seq {
  int n, q0, ctx, len;  // nodes, first row, context, positions
};

__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
  Seq s;
  const int lo = min(max(a.start[b], 0), a.T), hi = min(max(a.start[b + 1], 0), a.T);
  s.q0 = lo;
  s.n = max(hi - lo, 0);
  const int64_t most = (int64_t)a.max_pages * a.page_size;
  s.ctx = (int)min((int64_t)max(a.ctx[b], 0), most);
  s.len = (int)min((int64_t)s.ctx + s.n, most);
  return s;
}

struct Item {
  Seq s;
  int b, rt, h, split, splits, tiles;  // tiles: steps of a run
  int slot;                            // of the partial result, if splits > 1
};

// Workspace: the run length and the first slot of each sequence (-1: not cut),
// then the slots.  Every workgroup finds its item from the lengths by itself
// (a wave's prefix sums over the sequences), so there is no plan to keep.
struct Space {
  int32_t* tiles;
  int32_t* first;
  float* slots;
};

__device__ __forceinline__ Space space(const AttnArgs& a) {
  Space w;
  w.tiles = reinterpret_cast<int32_t*>(a.partial);
  w.first = w.tiles + 4;
  w.slots = a.partial + 4 + (a.B + 3) / 4 * 4;
  return w;
}

__device__ __forceinline__ int row_tiles(int n, int group, int rows) { return (n * group + rows - 1) / rows; }
__device__ __forceinline__ int key_tiles(int len) { return max((len + kTile - 1) / kTile, 1); }

// Item number `work`; false if there are fewer.  Items of a sequence: (run,
// head) units in groups of eight, the row tiles of a group's units one after
// the other, so that the row tiles that read the same keys are eight workgroups
// apart and share an XCD's L2.
template <int ROWS>
__device__ __forceinline__ bool find_item(const AttnArgs& a, int work, int slots, Item* it) {
  const int lane = threadIdx.x & (kWave - 1);
  const int group = a.heads / a.kv_heads;
  uint32_t units = 0;
  for (int base = 0; base < a.B; base += kWave) {
    int mine = 0;
    if (base + lane < a.B) {
      const Seq s = sequence(a, base + lane);
      mine = row_tiles(s.n, group, ROWS) * key_tiles(s.len) * a.kv_heads;
    }
    units += (uint32_t)__builtin_amdgcn_readlane(wave_inclusive_sum(mine), kWave - 1);
  }
  const int tiles = max((int)((units + slots - 1) / slots), 1);
  if (work == 0 && threadIdx.x == 0) *space(a).tiles = tiles;
  int before = 0, slots_before = 0;
  bool found = false;
  for (int base = 0; base < a.B; base += kWave) {
    Seq s{0, 0, 0, 0};
    int rts = 0, splits = 0;
    if (base + lane < a.B) {
      s = sequence(a, base + lane);
      rts = row_tiles(s.n, group, ROWS);
      splits = (key_tiles(s.len) + tiles - 1) / tiles;
    }
    const int count = rts * splits * a.kv_heads, cut = splits > 1 ? count : 0;
    const int end = before + wave_inclusive_sum(count);
    const int slot_end = slots_before + wave_inclusive_sum(cut);
    if (work == 0 && threadIdx.x < kWave && base + lane < a.B)
      space(a).first[base + lane] = splits > 1 ? slot_end - cut : -1;
    const uint64_t m = __ballot(work < end && work >= end - count);
    if (m && !found) {
      found = true;
      const int f = __ffsll((unsigned long long)m) - 1;
      it->b = base + f;
      it->s.n = __builtin_amdgcn_readlane(s.n, f);
      it->s.q0 = __builtin_amdgcn_readlane(s.q0, f);
      it->s.ctx = __builtin_amdgcn_readlane(s.ctx, f);
      it->s.len = __builtin_amdgcn_readlane(s.len, f);
      it->tiles = tiles;
      it->splits = __builtin_amdgcn_readlane(splits, f);
      const int rt_all = __builtin_amdgcn_readlane(rts, f);
      const int u_all = it->splits * a.kv_heads, whole = u_all / 8 * 8;
      int p = work - __builtin_amdgcn_readlane(end - count, f), u;
      if (p < whole * rt_all) {
        const int g = p / (8 * rt_all), r = p % (8 * rt_all);
        it->rt = r / 8;
        u = g * 8 + r % 8;
      } else {
        p -= whole * rt_all;
        it->rt = p / (u_all - whole);
        u = whole + p % (u_all - whole);
      }
      it->split = u / a.kv_heads;
      it->h = u % a.kv_heads;
      it->slot = __builtin_amdgcn_readlane(slot_end - cut, f) + u * rt_all + it->rt;
    }
    before = __builtin_amdgcn_readlane(end, kWave - 1);
    slots_before = __builtin_amdgcn_readlane(slot_end, kWave - 1);
    if (found && work != 0) break;
  }
  return found;
}

// Floats of one slot: 16 RT rows of DP sums, then their maxima and weights.
template <int DP, int RT>
constexpr int slot_floats() { return 16 * RT * (DP + 2); }

// Target number of items: the workgroups that are resident at once.
template <int DP, int RT>
constexpr int item_target() { return kCus * (DP * RT <= 128 ? 3 : DP * RT <= 256 ? 2 : 1); }

// ---------------------------------------------------------------- main kernel
// Transposed 16-bit read from LDS: within 16 lanes, lane 4 r + c reads 4
// elements (row r, columns 4 c ..), and lane l receives column l of the four
// rows.
__device__ __forceinline__ u32x2 lds_read_transposed(const uint16_t* p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p)));
}

template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t two) {
  const uint32_t e = DT == 0 ? 0x7c00u : 0x7f80u;
  return (two & e) == e || ((two >> 16) & e) == e;
}

template <int DT, int DP, int RT>
__global__ void __launch_bounds__(kWaves* kWave) attention_kernel(AttnArgs a, int slots, int max_slots) {
  constexpr int ROWS = 16 * RT;
  constexpr int KS = DP / 32;             // matrix-core steps of a score
  constexpr int DT_ = DP / 16;            // tiles of the output's columns
  constexpr int PITCH = DP + 16;          // of a staged value row, in elements: rows start 8 banks apart
  constexpr int LPR = DP / 8;             // lanes per value row
  constexpr int RPL = kWave / LPR;        // value rows per load
  constexpr int VL = kKeys / RPL;         // loads per step
  constexpr int STAGE = kKeys * PITCH * 2;                    // bytes of one wave's values
  constexpr int JOIN = 16 * (DP + 4) * 4;                     // bytes of one wave's sums of 16 rows
  __shared__ __align__(16) uint8_t lds[kWaves * (STAGE > JOIN ? STAGE : JOIN)];
  __shared__ float row_max[kWaves][ROWS], row_sum[kWaves][ROWS];

  Item it;
  if (!find_item<ROWS>(a, blockIdx.x, slots, &it)) return;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, quad = lane >> 4;
  const int group = a.heads / a.kv_heads, rows = it.s.n * group;
  const int row0 = it.rt * ROWS;
  const int begin = it.split * it.tiles * kTile;
  const int end = min(it.s.len, begin + it.tiles * kTile);

  // Queries: lane col of tile r holds row row0 + 16 r + col, elements
  // 32 s + 8 quad .. of it.  Rows beyond the last read the last one.
  u32x4 q[RT][KS];
  int node[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = min(row0 + r * 16 + col, rows - 1);
    node[r] = row / group;
    const uint16_t* p = a.q + (it.s.q0 + node[r]) * a.q_token + (it.h * group + row % group) * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) q[r][s] = load8_16_masked(p, s * 32 + quad * 8, a.dim, true);
  }
  const uint16_t* kbase = a.k + it.h * a.kv_head;
  const uint16_t* vbase = a.v + it.h * a.kv_head;
  const int32_t* table = a.table + (int64_t)it.b * a.ld_table;
  uint16_t* stage = reinterpret_cast<uint16_t*>(lds + wave * STAGE);

  f32x4 o[RT][DT_];
  float m[RT], l[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < DT_; ++d) o[r][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (int key0 = begin + wave * kKeys; key0 < end; key0 += kTile) {
    // Lane l holds the cache row of position key0 + l % 32, or -1.
    const int pos = key0 + (lane & 31);
    int64_t at = -1;
    if (pos < end) {
      const int32_t page = table[pos / a.page_size];
      if (in_range(page, a.num_pages)) at = page * a.kv_page + pos % a.page_size * a.kv_token;
    }
    const uint32_t there = (uint32_t)__ballot(at >= 0);  // both halves of the wave agree
    const int64_t safe = at < 0 ? 0 : at;

    u32x4 k[2][KS];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint16_t* p = kbase + __shfl(safe, t * 16 + col);
#pragma unroll
      for (int s = 0; s < KS; ++s) k[t][s] = load8_16_masked(p, s * 32 + quad * 8, a.dim, true);
    }
    u32x4 v[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int r = i * RPL + lane / LPR;
      const uint16_t* p = vbase + __shfl(safe, r);
      const int d = lane % LPR * 8;
      v[i] = *reinterpret_cast<const u32x4*>(p + (d < a.dim ? d : a.dim - 8));
      if (!((there >> r) & 1)) v[i] = u32x4{0u, 0u, 0u, 0u};
    }

    // Scores: lane holds positions key0 + 16 t + 4 quad + e of row col.
    f32x4 sc[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) sc[r][t] = mfma16x16x32<DT>(k[t][s], q[r][s], sc[r][t]);
        sc[r][t] *= a.scale_log2;
      }
    const bool drafted = key0 + kKeys > it.s.ctx;
    if (drafted || there != 0xffffffffu) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = t * 16 + quad * 4 + e;
            const int j = key0 + i - it.s.ctx;
            bool seen = (there >> i) & 1;
            if (seen && j >= 0) {
              if (a.mask) {
                seen = j < a.mask_words * 64 &&
                       ((a.mask[(int64_t)(it.s.q0 + node[r]) * a.ld_mask + j / 64] >> (j % 64)) & 1);
              } else {
                seen = j <= node[r];
              }
            }
            if (!seen) sc[r][t][e] = -INFINITY;
          }
    }

    // Running maximum and sum; weights as the next operand.
    u32x4 w[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float top = m[r];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[r][t][e]);
      top = max_over_lane_groups(top);
      const float base = top == -INFINITY ? 0.f : top;
      if (__any(top != m[r])) {
        const float shrink = __builtin_amdgcn_exp2f(m[r] - base);
        l[r] *= shrink;
#pragma unroll
        for (int d = 0; d < DT_; ++d) o[r][d] *= shrink;
      }
      m[r] = top;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[r][t][e] = __builtin_amdgcn_exp2f(sc[r][t][e] - base);
          l[r] += sc[r][t][e];
        }
        w[r][2 * t] = cvt_pack2<DT>(sc[r][t][0], sc[r][t][1]);
        w[r][2 * t + 1] = cvt_pack2<DT>(sc[r][t][2], sc[r][t][3]);
      }
    }

    // Values that are not finite are kept out of the products with weight 0:
    // they are staged as 0 and added below to the rows that see them.
    uint32_t odd = 0;  // positions of the step with such values
    if (drafted) {
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        bool bad = false;
#pragma unroll
        for (int x = 0; x < 4; ++x) bad |= not_finite<DT>(v[i][x]);
        const uint64_t lanes = __ballot(bad);
        if (lanes) {
#pragma unroll
          for (int r = 0; r < RPL; ++r)
            if ((lanes >> (r * LPR)) & ((LPR == 64 ? 0ull : 1ull << LPR) - 1ull)) odd |= 1u << (i * RPL + r);
          if ((odd >> (i * RPL + lane / LPR)) & 1) v[i] = u32x4{0u, 0u, 0u, 0u};
        }
      }
    }

    // Values through LDS (the wave's own part): rows in, columns out.
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < VL; ++i)
      *reinterpret_cast<u32x4*>(stage + (i * RPL + lane / LPR) * PITCH + lane % LPR * 8) = v[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int d = 0; d < DT_; ++d) {
      // Elements 0..3: positions 4 quad + 0..3 of the first 16, 4..7 of the second.
      const uint16_t* p = stage + (quad * 4 + (col >> 2)) * PITCH + d * 16 + (col & 3) * 4;
      const u32x2 lo = lds_read_transposed(p), hi = lds_read_transposed(p + 16 * PITCH);
      const u32x4 vt = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
      for (int r = 0; r < RT; ++r) o[r][d] = mfma16x16x32<DT>(vt, w[r], o[r][d]);
    }
    __builtin_amdgcn_wave_barrier();

    while (odd) {
      const int i = __ffs(odd) - 1;
      odd &= odd - 1;
      const uint16_t* p = vbase + __shfl(safe, i);
      const int src = (i % 16 / 4) * 16 + col;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float weight = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __shfl(sc[r][t][e], src);
            if (i / 16 == t && i % 4 == e) weight = x;
          }
#pragma unroll
        for (int d = 0; d < DT_; ++d) {
          const int c = d * 16 + quad * 4;
          const u32x2 two = *reinterpret_cast<const u32x2*>(p + (c < a.dim ? c : a.dim - 4));
          float x[4];
          unpack2<DT>(two.x, &x[0], &x[1]);
          unpack2<DT>(two.y, &x[2], &x[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (weight != 0.f) o[r][d][e] += weight * x[e];
        }
      }
    }
  }

  // Join the waves: 16 rows at a time through LDS.
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float x = l[r];
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    if (quad == 0) {
      row_max[wave][r * 16 + col] = m[r];
      row_sum[wave][r * 16 + col] = x;
    }
  }
  constexpr int JP = DP + 4;
  float* join = reinterpret_cast<float*>(lds);
  float* slot = nullptr;
  if (it.splits > 1) {
    if (it.slot >= max_slots) return;  // only where start is not ascending
    slot = space(a).slots + (int64_t)it.slot * slot_floats<DP, RT>();
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < DT_; ++d)
      *reinterpret_cast<f32x4*>(join + (wave * 16 + col) * JP + d * 16 + quad * 4) = o[r][d];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * DP / 4; e += kWaves * kWave) {
      const int i = e / (DP / 4), c = e % (DP / 4) * 4, in_tile = r * 16 + i, row = row0 + in_tile;
      if (row >= rows) continue;
      float top = row_max[0][in_tile];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, row_max[w][in_tile]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(row_max[w][in_tile] - base);
        sum += f * row_sum[w][in_tile];
        x += *reinterpret_cast<const f32x4*>(join + (w * 16 + i) * JP + c) * f;
      }
      if (slot) {
        *reinterpret_cast<f32x4*>(slot + in_tile * DP + c) = x;
        if (c == 0) {
          slot[ROWS * DP + in_tile] = top;
          slot[ROWS * DP + ROWS + in_tile] = sum;
        }
        continue;
      }
      const int t = it.s.q0 + row / group, h = it.h * group + row % group;
      if (a.lse && c == 0)
        a.lse[(int64_t)t * a.heads + h] = sum > 0.f ? (base + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f : (sum == 0.f ? -INFINITY : sum);
      if (c >= a.dim) continue;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<u32x2*>(a.out + t * a.out_token + h * a.out_head + c) =
          u32x2{cvt_pack2<DT>(x.x * inv, x.y * inv), cvt_pack2<DT>(x.z * inv, x.w * inv)};
    }
  }
}

// ---------------------------------------------------------------- join of runs
// One block per row (token, head): wave w takes runs w, w + 4, ...; 64 lanes
// hold the DP columns.
template <int DT, int DP, int RT>
__global__ void __launch_bounds__(kWaves* kWave) join_kernel(AttnArgs a, int max_slots) {
  constexpr int ROWS = 16 * RT, PER = DP / kWave;
  const Space sp = space(a);
  const int t = blockIdx.x / a.heads, head = blockIdx.x % a.heads;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int group = a.heads / a.kv_heads;
  // The sequence of token t.
  int b = -1;
  for (int base = 0; base < a.B && b < 0; base += kWave) {
    const bool mine = base + lane < a.B && a.start[base + lane] <= t && t < a.start[base + lane + 1];
    const uint64_t m = __ballot(mine);
    if (m) b = base + __ffsll((unsigned long long)m) - 1;
  }
  if (b < 0) return;
  const int first = sp.first[b];
  if (first < 0) return;
  const Seq s = sequence(a, b);
  const int tiles = *sp.tiles;
  const int splits = (key_tiles(s.len) + tiles - 1) / tiles, rts = row_tiles(s.n, group, ROWS);
  const int row = (t - s.q0) * group + head % group, rt = row / ROWS, in_tile = row % ROWS;
  auto slot_of = [&](int split) {
    const int64_t i = min((int64_t)first + ((int64_t)split * a.kv_heads + head / group) * rts + rt, (int64_t)max_slots - 1);
    return sp.slots + i * slot_floats<DP, RT>();
  };
  float top = -INFINITY;
  for (int i = lane; i < splits; i += kWave) top = fmaxf(top, slot_of(i)[ROWS * DP + in_tile]);
#pragma unroll
  for (int x = 1; x < kWave; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = wave; i < splits; i += kWaves) {
    const float* p = slot_of(i);
    const float f = __builtin_amdgcn_exp2f(p[ROWS * DP + in_tile] - base);
    sum += f * p[ROWS * DP + ROWS + in_tile];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] += f * p[in_tile * DP + e * kWave + lane];
  }
  __shared__ float part[kWaves][DP + 1];
#pragma unroll
  for (int e = 0; e < PER; ++e) part[wave][e * kWave + lane] = acc[e];
  if (lane == 0) part[wave][DP] = sum;
  __syncthreads();
  sum = part[0][DP] + part[1][DP] + part[2][DP] + part[3][DP];
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int c = threadIdx.x; c < a.dim; c += kWaves * kWave)
    a.out[t * a.out_token + head * a.out_head + c] =
        (uint16_t)from_f32<DT>((part[0][c] + part[1][c] + part[2][c] + part[3][c]) * inv);
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)t * a.heads + head] =
        sum > 0.f ? (base + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f : (sum == 0.f ? -INFINITY : sum);
}

template <int DT, int DP, int RT>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
  constexpr int ROWS = 16 * RT, target = item_target<DP, RT>();
  const int64_t group = a.heads / a.kv_heads;
  // Every sequence has at most one row tile that is not full.
  const int64_t tiles = a.T * group / ROWS + (a.B < a.T * group ? a.B : a.T * group);
  attention_kernel<DT, DP, RT><<<(unsigned)(target + tiles * a.kv_heads), kWaves * kWave, 0, s>>>(a, target, 2 * target);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  join_kernel<DT, DP, RT><<<(unsigned)(a.T * a.heads), kWaves * kWave, 0, s>>>(a, 2 * target);
  return hipGetLastError();
}

// Rows of a workgroup: what an average sequence has, up to what the registers
// hold.
int choose_rt(int64_t B, int64_t T, int group, int dp) {
  const int64_t rows = (T * group + B - 1) / B;
  const int most = dp == 256 ? 2 : 4;
  const int rt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  return rt < most ? rt : most;
}

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s) {
  const int dp = padded_dim(a.dim), rt = choose_rt(a.B, a.T, a.heads / a.kv_heads, dp);
  switch (dp * 8 + rt) {
    case 64 * 8 + 1: return launch<DT, 64, 1>(a, s);
    case 64 * 8 + 2: return launch<DT, 64, 2>(a, s);
    case 64 * 8 + 4: return launch<DT, 64, 4>(a, s);
    case 128 * 8 + 1: return launch<DT, 128, 1>(a, s);
    case 128 * 8 + 2: return launch<DT, 128, 2>(a, s);
    case 128 * 8 + 4: return launch<DT, 128, 4>(a, s);
    case 256 * 8 + 1: return launch<DT, 256, 1>(a, s);
    default: return launch<DT, 256, 2>(a, s);
  }
}

}  // namespace

size_t attention_workspace(int32_t B, int32_t T, int32_t heads, int32_t kv_heads, int32_t dim) {
  // 2 x item_target slots of 16 RT (DP + 2) floats, for every RT.
  const int dp = padded_dim(dim), rt = choose_rt(B, T, heads / kv_heads, dp);
  const int per_cu = dp * rt <= 128 ? 3 : dp * rt <= 256 ? 2 : 1;
  return (4 + ((size_t)B + 3) / 4 * 4 + (size_t)2 * kCus * per_cu * 16 * rt * (dp + 2)) * 4;
}

hipError_t launch_attention(const AttnArgs& args, int dtype, hipStream_t s) {
  AttnArgs a = args;
  if (a.num_pages == 0) {  // nothing is there to be read: any legal address will do
    a.k = a.v = a.q;
    a.kv_head = 0;
  }
  return dtype == 0 ? launch_dt<0>(a, s) : launch_dt<1>(a, s);
}

}  // namespace lora
