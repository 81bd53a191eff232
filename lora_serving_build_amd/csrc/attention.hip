// Attention of a step's drafted tokens over a paged cache (lora_tree_attention).
//
//   o[i, h] = sum_p w_p v[p] / sum_p w_p,  w_p = 2^(scale log2(e) q[i, h] . k[p] - m)
//
// Rows: the nodes of a sequence times the G = heads / kv_heads query heads that
// share a key head, so one pass over the keys serves all of them.  A line is one
// row tile of one (sequence, key head), as long as the sequence's tiles of
// positions.  The lines of a call, end to end, are cut into equal parts, two for
// each CU: ragged lengths and few rows cost no idle workgroups.  A line that lies
// in one part is finished there; the pieces
// of one that was cut are joined by a second kernel.
#include "decode_kernels.h"
#include "lora_device.h"

namespace lora {
namespace {

constexpr int kWaves = 4;
constexpr int kKeys = 32;                 // positions of one wave's step
constexpr int kTile = kWaves * kKeys;     // positions of one workgroup's step
constexpr int kCus = 256;

__device__ __forceinline__ bool in_range(int32_t v, int32_t n) { return (uint32_t)v < (uint32_t)n; }

// ---------------------------------------------------------------- work
// A sequence as the kernels see it, whatever the buffers hold.
struct Seq {
  int n, q0, ctx, len;  // nodes, first row, context, positions
};

// descends (optional): set if the sequence ends before it starts.
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b, bool* descends = nullptr) {
  Seq s;
  const int lo = min(max(a.start[b], 0), a.T), hi = min(max(a.start[b + 1], 0), a.T);
  if (descends) *descends |= hi < lo;
  s.q0 = lo;
  s.n = max(hi - lo, 0);
  const int64_t most = (int64_t)a.max_pages * a.page_size;
  s.ctx = (int)min((int64_t)max(a.ctx[b], 0), most);
  s.len = (int)min((int64_t)s.ctx + s.n, most);
  return s;
}

__device__ __forceinline__ int row_tiles(int n, int group, int rows) { return (n * group + rows - 1) / rows; }
__device__ __forceinline__ int key_tiles(int len, int keys) { return max((len + keys - 1) / keys, 1); }

// Positions of a table up to which lines are not cut: four steps of eight waves.
constexpr int kShortLine = 4 * 8 * kKeys;

// Number of parts: the workgroups that are resident at once with head dims of 65
// to 128.  Dims up to 64 leave room for a third on a CU with up to 64 rows; of
// dims above 128 the kernel for few rows has one on a CU, so its parts take two
// rounds.
constexpr int kParts = kCus * 2;

// What a line costs besides its tiles, in tiles: its start (pages, first keys,
// queries) and end are not hidden.  Parts are equal in cost, so that those of
// many short lines do not end last.
template <int ROWS>
constexpr int line_cost() { return ROWS > 16 ? 3 : 1; }

// Positions of a tile that the waves share (what two workgroups' LDS holds).
template <int DP>
constexpr int wide_tile() { return DP == 256 ? 32 : 64; }

// Workspace: the cost of a part and of a line besides its tiles, and where each sequence's lines start (a line
// after the other: key heads, row tiles running fastest; a line's cost comes
// before its tiles), then two slots for each part: a line cut by the part's
// start leaves its sums in the first, one cut by its end only in the second.
struct Space {
  int32_t* part;
  int32_t* first;
  float* slots;
};

__device__ __forceinline__ Space space(const AttnArgs& a) {
  Space w;
  w.part = reinterpret_cast<int32_t*>(a.partial);
  w.first = w.part + 4;
  w.slots = a.partial + 4 + (a.B + 3) / 4 * 4;
  return w;
}

// Floats of one slot: the rows' DP sums, then their maxima and weights.
template <int DP, int ROWS>
constexpr int slot_floats() { return ROWS * (DP + 2); }

// tiles0: where the line's tiles start.
__device__ __forceinline__ int slot_of(int part, int part_cost, int tiles0) {
  return 2 * part + (tiles0 <= part * part_cost ? 0 : 1);
}

struct Place {
  Seq s;
  int b, h, rt, rts, tiles;  // sequence, key head, row tile of rts, tiles of the line
  int line, at, end;         // start of the line, of this piece and end of the part (costs from the call's start)
  int part, part_cost, cost;  // cost of a line besides its tiles
};

__device__ __forceinline__ void enter_sequence(const AttnArgs& a, int rows, int keys, int b, Place* p) {
  p->b = b;
  p->s = sequence(a, b);
  p->s.n = __builtin_amdgcn_readfirstlane(p->s.n);
  p->s.q0 = __builtin_amdgcn_readfirstlane(p->s.q0);
  p->s.ctx = __builtin_amdgcn_readfirstlane(p->s.ctx);
  p->s.len = __builtin_amdgcn_readfirstlane(p->s.len);
  p->rts = row_tiles(p->s.n, a.heads / a.kv_heads, rows);
  p->tiles = key_tiles(p->s.len, keys);
}

// The start of the workgroup's part; false if it has none.  Every wave finds
// it by itself from the lengths (prefix sums over the sequences), so there is
// no plan to keep.  Neighbouring parts, whose lines often read the same keys,
// go to one XCD and its L2.
template <int ROWS, int KEYS, int COST>
__device__ __forceinline__ bool find_part(const AttnArgs& a, Place* p) {
  const int lane = threadIdx.x & (kWave - 1);
  const int group = a.heads / a.kv_heads;
  const int part = (blockIdx.x & 7) * (kParts / 8) + (blockIdx.x >> 3);
  auto lines_of = [&](const Seq& s) { return row_tiles(s.n, group, ROWS) * a.kv_heads; };
  // Sequence base + lane, empty beyond the last; the first 64 are read once.
  bool descends = false;
  auto read = [&](int base) {
    return base + lane < a.B ? sequence(a, base + lane, &descends) : Seq{0, 0, 0, 0};
  };
  const Seq head = read(0);
  auto seq_at = [&](int base) { return base == 0 ? head : read(base); };
  uint32_t lines = 0, tiles = 0;
  for (int base = 0; base < a.B; base += kWave) {
    const Seq s = seq_at(base);
    const int l = lines_of(s);
    lines += (uint32_t)__builtin_amdgcn_readlane(wave_inclusive_sum(l), kWave - 1);
    tiles += (uint32_t)__builtin_amdgcn_readlane(wave_inclusive_sum(l * key_tiles(s.len, KEYS)), kWave - 1);
  }
  // Starts that do not ascend can name more rows than there are, and 32 bits may
  // not hold their tiles: there are no parts, and nothing to join (cost 0).
  if (__any(descends)) {
    if (part == 0 && threadIdx.x == 0) space(a).part[0] = 0;
    return false;
  }
  // With fewer tiles than parts every tile is a part.
  const int cost = tiles <= (uint32_t)kParts ? 0 : COST;
  const uint32_t total = tiles + lines * cost;
  const int part_cost = max((int)((total + kParts - 1) / kParts), cost + 1);
  p->cost = cost;
  p->part = part;
  p->part_cost = part_cost;
  p->at = part * part_cost;
  p->end = min((int)total, p->at + part_cost);
  if (part == 0 && threadIdx.x == 0) {
    space(a).part[0] = part_cost;
    space(a).part[1] = cost;
  }
  int before = 0, b = -1, start = 0;
  for (int base = 0; base < a.B; base += kWave) {
    const Seq s = seq_at(base);
    const int mine = lines_of(s) * (cost + key_tiles(s.len, KEYS));
    const int end = before + wave_inclusive_sum(mine);
    if (part == 0 && threadIdx.x < kWave && base + lane < a.B) space(a).first[base + lane] = end - mine;
    const uint64_t m = __ballot(p->at < end && p->at >= end - mine);
    if (m && b < 0) {
      const int f = __ffsll((unsigned long long)m) - 1;
      b = base + f;
      start = __builtin_amdgcn_readlane(end - mine, f);
    }
    before = __builtin_amdgcn_readlane(end, kWave - 1);
    if (b >= 0 && part != 0) break;
  }
  if (b < 0 || p->at >= p->end) return false;
  enter_sequence(a, ROWS, KEYS, b, p);
  const int line = (p->at - start) / (cost + p->tiles);
  p->h = line / p->rts;
  p->rt = line % p->rts;
  p->line = start + line * (cost + p->tiles);
  return true;
}

// Line number blockIdx.x, whole, as a part of its own; false if there are fewer.
template <int ROWS, int KEYS>
__device__ __forceinline__ bool find_line(const AttnArgs& a, Place* p) {
  const int lane = threadIdx.x & (kWave - 1);
  const int group = a.heads / a.kv_heads, line = blockIdx.x;
  int before = 0;
  for (int base = 0; base < a.B; base += kWave) {
    int mine = 0;
    if (base + lane < a.B) mine = row_tiles(sequence(a, base + lane).n, group, ROWS) * a.kv_heads;
    const int end = before + wave_inclusive_sum(mine);
    const uint64_t m = __ballot(line < end && line >= end - mine);
    if (m) {
      const int f = __ffsll((unsigned long long)m) - 1;
      enter_sequence(a, ROWS, KEYS, base + f, p);
      const int at = line - __builtin_amdgcn_readlane(end - mine, f);
      p->h = at / p->rts;
      p->rt = at % p->rts;
      p->line = p->at = p->part = p->cost = 0;
      p->end = p->part_cost = p->tiles;
      return true;
    }
    before = __builtin_amdgcn_readlane(end, kWave - 1);
  }
  return false;
}

// The line after the one of *p, in a part that goes on.
template <int ROWS, int KEYS>
__device__ __forceinline__ void next_line(const AttnArgs& a, Place* p) {
  p->line += p->cost + p->tiles;
  p->at = p->line;
  if (++p->rt < p->rts) return;
  p->rt = 0;
  if (++p->h < a.kv_heads) return;
  p->h = 0;
  int b = p->b + 1;
  do enter_sequence(a, ROWS, KEYS, b, p);
  while (p->rts == 0 && ++b < a.B);
}

// ---------------------------------------------------------------- pieces of both kernels
// Transposed 16-bit read from LDS: within 16 lanes, lane 4 r + c reads 4
// elements (row r, columns 4 c ..), and lane l receives column l of the four
// rows.
__device__ __forceinline__ u32x2 lds_read_transposed(const uint16_t* p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p)));
}

// Whether one of the 8 N values is an infinity or NaN: the largest magnitude's
// pattern tells (in four chains, since a wave may be alone on its SIMD).
template <int DT, int N>
__device__ __forceinline__ bool not_finite(const u32x4 (&v)[N]) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  u16x2 most[4] = {};
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      most[x] = __builtin_elementwise_max(most[x], __builtin_bit_cast(u16x2, v[i][x] & 0x7fff7fffu));
  most[0] = __builtin_elementwise_max(__builtin_elementwise_max(most[0], most[1]), __builtin_elementwise_max(most[2], most[3]));
  const unsigned short e = DT == 0 ? 0x7c00 : 0x7f80;
  return most[0].x >= e || most[0].y >= e;
}
template <int DT>
__device__ __forceinline__ bool not_finite(u32x4 v) {
  const u32x4 one[1] = {v};
  return not_finite<DT, 1>(one);
}

// Rows of a step (a bit each) to which `lanes` of its i-th load of VL belong.
template <int VL>
__device__ __forceinline__ uint32_t rows_of(int i, uint64_t lanes) {
  constexpr int RPL = kKeys / VL, LPR = kWave / RPL;
  uint32_t rows = 0;
  if (lanes) {
#pragma unroll
    for (int x = 0; x < RPL; ++x)
      if ((lanes >> (x * LPR)) & ((1ull << LPR) - 1ull)) rows |= 1u << (i * RPL + x);
  }
  return rows;
}

// pos / page_size for 0 <= pos < 2^31: the high half of a product with
// ceil(2^(31 + s) / page_size), s the bits of page_size - 1, shifted by s - 1.
// The excess of the factor is below 1, so that of the quotient is below
// 2^31 / 2^(31 + s) <= 1 / page_size, too little to reach the next whole number.
__device__ __forceinline__ int page_of_position(const AttnArgs& a, int pos) {
  return a.page_mul ? (int)(__umulhi((uint32_t)pos, a.page_mul) >> a.page_shift) : pos;
}

// Offset (elements) of position pos of the sequence in page `page`, the id that
// its table row holds for page number w; -1 if that is no page of the cache.
__device__ __forceinline__ int64_t cache_row(const AttnArgs& a, int page, int w, int pos) {
  return in_range(page, a.num_pages) ? page * a.kv_page + (pos - w * a.page_size) * a.kv_token : (int64_t)-1;
}

// Queries of one row tile as matrix-core operand: lane col holds row
// `row` (elements 32 s + 8 quad .. of it).  A negative scale turns their sign.
template <int DP>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Place& it, int node, int head, int quad,
                                             u32x4 (&q)[DP / 32]) {
  const uint16_t* p = a.q + (it.s.q0 + node) * a.q_token + head * a.q_head;
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
  for (int s = 0; s < DP / 32; ++s) {
    q[s] = load8_16_masked(p, s * 32 + quad * 8, a.dim, true);
    q[s] ^= u32x4{flip, flip, flip, flip};
  }
}

// First word of a row's mask (all ones without one).
__device__ __forceinline__ uint64_t first_mask_word(const AttnArgs& a, const Place& it, int node) {
  if (!a.mask) return ~0ull;
  return a.mask_words > 0 ? a.mask[(int64_t)(it.s.q0 + node) * a.ld_mask] : 0ull;
}

// Which of the positions key0 .. key0 + 31 row `node` sees, one bit each;
// `there`: the positions that exist; `word`: the first of the row's mask.
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs& a, const Place& it, int node, uint64_t word, int key0,
                                              uint32_t there) {
  const int j0 = key0 - it.s.ctx;  // the node at position key0; at least -31 where it matters
  if (j0 <= -32) return there;
  uint32_t bits;
  if (a.mask) {
    // 32 bits from bit j0 on of the row's words; all ones before bit 0, zeros
    // behind the last word.
    const uint64_t* row = a.mask + (int64_t)(it.s.q0 + node) * a.ld_mask;
    const int w = j0 >> 6, sh = j0 & 63, last = a.mask_words - 1;
    uint64_t lo = w < 0 ? ~0ull : w == 0 ? word : 0ull, hi = w < 0 ? word : 0ull;
    if (w >= 0 && last > 0) {
      if (w > 0 && w <= last) lo = row[w];
      if (w < last) hi = row[w + 1];
    }
    bits = (uint32_t)((lo >> sh) | (sh ? hi << (64 - sh) : 0ull));
  } else {
    const int ones = node - j0 + 1;
    bits = ones >= 32 ? ~0u : ones <= 0 ? 0u : (1u << ones) - 1u;
  }
  return bits & there;
}

// -inf into the scores of positions that are not seen: s[t][e] is position
// 16 t + 4 quad + e of the 32.
__device__ __forceinline__ void mask_scores(uint32_t seen, int quad, f32x4 (&s)[2]) {
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!((seen >> (t * 16 + quad * 4 + e)) & 1)) s[t][e] = -INFINITY;
}

// log2 of what a weight of 1 stands for, from the row's reference score m.  In
// binary16 that is 2^9 below the reference, so that the weights use the upper end
// of the type's range (2^15 at most, see weigh) and those far below the heaviest
// are not lost while the sum l counts them: from 2^-23 of the reference down
// they have fewer bits, and the last step is 2^-33 of it.
template <int DT>
__device__ __forceinline__ float weight_base(float m, float c) { return __builtin_fmaf(m, c, DT == 0 ? -9.f : 0.f); }

// 16-bit parts in which a weight meets the values.  Two (the weight rounded, and
// what that left over) leave o with little more than its own rounding, and are
// free where the kernels wait for memory: 64 sequences of one token 115 us with
// two and 117 with one, 64 rows 79 and 79.  With 128 rows they would cost a sixth
// (dim 128: 152 us against 130, dim 64: 108 against 92), with dim 256 up to a
// third (16 rows: 197 against 154, for want of registers): there a weight is
// rounded once, to the cache's type.
template <int DP, int ROWS>
constexpr int weight_parts() { return DP <= 128 && ROWS <= 64 ? 2 : 1; }

// One step of the running softmax of RT row tiles: raw scores in, weights out
// (and as the 16-bit operands of the value product).  c = |scale| log2 e.  The
// reference scores m follow the maxima only when one has grown by 2^6 in
// weight: until then the weights are at most 2^6 of the reference's, which loses
// nothing in fp32 sums and saves the scaling of l and o.  One branch for all row
// tiles: their chains of dependent operations run side by side.
template <int DT, int PARTS, int RT, int N>
__device__ __forceinline__ void weigh(f32x4 (&s)[RT][2], float c, float (&m)[RT], float (&l)[RT], f32x4 (&o)[RT][N],
                                      u32x4 (&w)[PARTS][RT]) {
  float top[RT];
  bool grown = false;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    top[r] = fmaxf(fmaxf(fmaxf(s[r][0].x, s[r][0].y), fmaxf(s[r][0].z, s[r][0].w)),
                   fmaxf(fmaxf(s[r][1].x, s[r][1].y), fmaxf(s[r][1].z, s[r][1].w)));
    top[r] = max_over_lane_groups(top[r]);
    grown |= (top[r] - m[r]) * c > 6.f;
  }
  if (__any(grown)) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float now = fmaxf(top[r], m[r]);
      const float shrink = m[r] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[r] - now) * c);
      l[r] *= shrink;
#pragma unroll
      for (int d = 0; d < N; ++d) o[r][d] *= shrink;
      m[r] = now;
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float base = m[r] == -INFINITY ? 0.f : -weight_base<DT>(m[r], c);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[r][t][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][t][e], c, base));
        l[r] += s[r][t][e];
      }
    w[0][r] = u32x4{cvt_pack2<DT>(s[r][0].x, s[r][0].y), cvt_pack2<DT>(s[r][0].z, s[r][0].w),
                    cvt_pack2<DT>(s[r][1].x, s[r][1].y), cvt_pack2<DT>(s[r][1].z, s[r][1].w)};
    if constexpr (PARTS == 2) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float a, b;
        unpack2<DT>(w[0][r][x], &a, &b);
        w[1][r][x] = cvt_pack2<DT>(s[r][x / 2][x % 2 * 2] - a, s[r][x / 2][x % 2 * 2 + 1] - b);
      }
    }
  }
}

// Adds the value row p (position i of the step), which is not finite
// throughout and was kept out of the products, to the rows that see it.
template <int DT, int PARTS, int RT, int N>
__device__ __forceinline__ void add_odd_value(const uint16_t* p, int i, int dim, int col, int quad,
                                              const u32x4 (&w)[PARTS][RT], int r, f32x4 (&o)[N]) {
  // Weight of position 16 t + 4 q + e: lane (q, col), half e % 2 of dword 2 t + e / 2.
  float weight = 0.f;
#pragma unroll
  for (int part = 0; part < PARTS; ++part) {
    uint32_t two = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i / 16 * 2 + i % 4 / 2 == x) two = w[part][r][x];
    two = __shfl(two, (i % 16 / 4) * 16 + col);
    weight += to_f32<DT>(i % 2 ? two >> 16 : two & 0xffffu);
  }
#pragma unroll
  for (int d = 0; d < N; ++d) {
    __builtin_amdgcn_sched_barrier(0);  // one load at a time: registers count, time does not
    const int c = d * 16 + quad * 4;
    const u32x2 four = *reinterpret_cast<const u32x2*>(p + (c < dim ? c : dim - 4));
    float x[4];
    unpack2<DT>(four.x, &x[0], &x[1]);
    unpack2<DT>(four.y, &x[2], &x[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (weight != 0.f) o[d][e] += weight * x[e];
  }
}

__device__ __forceinline__ float log_sum(float base_log2, float sum) {
  return sum > 0.f ? (base_log2 + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f : sum == 0.f ? -INFINITY : sum;
}

// Scale of the exponent: never 0, which would turn a masked -inf into NaN.
__device__ __forceinline__ float exponent_scale(const AttnArgs& a) { return fmaxf(fabsf(a.scale_log2), 1e-30f); }

// Where a row's result goes: row maxima in units of log2.
template <int DT>
__device__ __forceinline__ void store_quad(const AttnArgs& a, int t, int h, int c, f32x4 x, float inv) {
  if (c < a.dim)
    *reinterpret_cast<u32x2*>(a.out + t * a.out_token + h * a.out_head + c) =
        u32x2{cvt_pack2<DT>(x.x * inv, x.y * inv), cvt_pack2<DT>(x.z * inv, x.w * inv)};
}

// ---------------------------------------------------------------- few rows
// Waves of a workgroup take different positions.  Keys go from memory straight
// into the matrix core's operand; values pass through the wave's own part of
// LDS, which turns rows into columns.  The next step's keys and values are on
// their way while this one's are used.  WHOLE: a workgroup takes one line, for
// contexts so short that nothing needs to be cut and joined; else one of the
// call's equal parts.
// Bound by memory: 64 sequences of one token, 546 MB of keys and values in
// 16-token pages, 64 heads over 8 key heads of 128: 112 us, 4.9 TB/s (a copy
// reads and writes 4.8).  One token over 509 positions, 32 heads: 10.4 us of
// dependent latencies (lengths, page, keys, softmax, join of the waves).  Dim 256
// takes all 256 vector registers and 170 to 230 accumulation registers: one wave
// a SIMD.
template <int DT, int DP, int W, bool WHOLE>
__global__ void __launch_bounds__(W* kWave, DP == 256 ? 1 : 2) attention_kernel(AttnArgs a) {
  constexpr int ROWS = 16, TILE = W * kKeys;
  constexpr int PARTS = weight_parts<DP, ROWS>();
  constexpr int KS = DP / 32;             // matrix-core steps of a score
  constexpr int OT = DP / 16;             // tiles of the output's columns
  constexpr int PITCH = DP + 16;          // of a staged value row, in elements: rows start 8 banks apart
  constexpr int LPR = DP / 8;             // lanes per value row
  constexpr int RPL = kWave / LPR;        // value rows per load
  constexpr int VL = kKeys / RPL;         // loads per step
  constexpr int JP = DP + 4;              // pitch of a row of sums
  constexpr int STAGE = kKeys * PITCH * 2;  // bytes of one wave's values
  constexpr int JOIN = ROWS * JP * 4;       // bytes of one wave's sums
  __shared__ __align__(16) uint8_t lds[W * (STAGE > JOIN ? STAGE : JOIN)];
  __shared__ float row_max[W][ROWS], row_sum[W][ROWS];

  Place it;
  if (WHOLE ? !find_line<ROWS, TILE>(a, &it) : !find_part<ROWS, TILE, line_cost<ROWS>()>(a, &it)) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, quad = lane >> 4;
  const int group = a.heads / a.kv_heads;
  const float c = exponent_scale(a);
  uint16_t* stage = reinterpret_cast<uint16_t*>(lds + wave * STAGE);
  float* join = reinterpret_cast<float*>(lds);

  for (;;) {
    const int rows = it.s.n * group, row0 = it.rt * ROWS;
    const int from = max(it.at - it.line - it.cost, 0), to = min(it.tiles, it.end - it.line - it.cost);
    if (to > from) {
    const int begin = from * TILE, end = min(it.s.len, to * TILE);

    const int my_row = min(row0 + col, rows - 1);  // rows beyond the last read the last one
    const int node = my_row / group;
    const uint64_t word = first_mask_word(a, it, node);
    u32x4 q[KS];
    load_queries<DP>(a, it, node, it.h * group + my_row % group, quad, q);
    const uint16_t* kbase = a.k + it.h * a.kv_head;
    const uint16_t* vbase = a.v + it.h * a.kv_head;
    const int32_t* table = a.table + (int64_t)it.b * a.ld_table;

    f32x4 o[1][OT];
    float m[1] = {-INFINITY}, l[1] = {0.f};
#pragma unroll
    for (int d = 0; d < OT; ++d) o[0][d] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Page of position key0 + lane % 32 (of the last one, where that is beyond
    // the end), and the cache row that follows from it.
    auto page_of = [&](int key0) { return table[page_of_position(a, min(key0 + (lane & 31), end - 1))]; };
    auto row_of = [&](int key0, int page) {
      const int pos = key0 + (lane & 31);
      return pos < end ? cache_row(a, page, page_of_position(a, pos), pos) : (int64_t)-1;
    };
    u32x4 k[2][KS], v[VL];
    auto load = [&](int64_t safe) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint16_t* p = kbase + __shfl(safe, t * 16 + col);
#pragma unroll
        for (int s = 0; s < KS; ++s) k[t][s] = load8_16_masked(p, s * 32 + quad * 8, a.dim, true);
      }
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const uint16_t* p = vbase + __shfl(safe, i * RPL + lane / LPR);
        const int d = lane % LPR * 8;
        v[i] = *reinterpret_cast<const u32x4*>(p + (d < a.dim ? d : a.dim - 8));
      }
    };

    int key0 = begin + wave * kKeys;
    int page = 0;
    int64_t at = -1;
    if (key0 < end) {
      page = page_of(key0);
      at = row_of(key0, page);
      load(at < 0 ? 0 : at);
      page = page_of(key0 + TILE);
    }
    for (; key0 < end; key0 += TILE) {
      const uint32_t there = (uint32_t)__ballot(at >= 0);  // both halves of the wave agree
      const int64_t here = at < 0 ? 0 : at;

      // Scores: lane holds positions key0 + 16 t + 4 quad + e of row col.
      f32x4 sc[1][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sc[0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) sc[0][t] = mfma16x16x32<DT>(k[t][s], q[s], sc[0][t]);
      }

      // Values that are not finite are kept out of the products, where a weight
      // of 0 (not seen) or below 0 (what rounding left over) would make NaN of
      // them: their rows are staged as 0 and added below to the rows that see
      // them.  With one part, whose weights are never below 0, only steps are
      // looked at in which rows differ in what they see.
      uint32_t odd = 0;  // positions of the step with such values
      const bool drafted = key0 + kKeys > it.s.ctx;
      if (there != 0xffffffffu || (PARTS == 1 && drafted)) {
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const int r = i * RPL + lane / LPR;
          bool zero = !((there >> r) & 1);
          if (PARTS == 1 && drafted) {
            odd |= rows_of<VL>(i, __ballot(not_finite<DT>(v[i]) && !zero));
            zero |= (odd >> r) & 1;
          }
          if (zero) v[i] = u32x4{0u, 0u, 0u, 0u};
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      uint16_t* mine = stage + lane / LPR * PITCH + lane % LPR * 8;
#pragma unroll
      for (int i = 0; i < VL; ++i) *reinterpret_cast<u32x4*>(mine + i * RPL * PITCH) = v[i];
      if (PARTS == 2 && __any(not_finite<DT>(v))) {
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          odd |= rows_of<VL>(i, __ballot(not_finite<DT>(v[i])));
          if ((odd >> (i * RPL + lane / LPR)) & 1) *reinterpret_cast<u32x4*>(mine + i * RPL * PITCH) = u32x4{0u, 0u, 0u, 0u};
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

      // The next step.
      const int next = key0 + TILE;
      at = row_of(next, page);
      if (next < end) load(at < 0 ? 0 : at);
      page = page_of(next + TILE);

      if (drafted || there != 0xffffffffu) mask_scores(seen_bits(a, it, node, word, key0, there), quad, sc[0]);
      u32x4 w[PARTS][1];
      weigh<DT, PARTS, 1, OT>(sc, c, m, l, o, w);

      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int d = 0; d < OT; ++d) {
        // Elements 0..3: positions 4 quad + 0..3 of the first 16, 4..7 of the second.
        const uint16_t* p = stage + (quad * 4 + (col >> 2)) * PITCH + d * 16 + (col & 3) * 4;
        const u32x2 lo = lds_read_transposed(p), hi = lds_read_transposed(p + 16 * PITCH);
        const u32x4 vf = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int part = 0; part < PARTS; ++part) o[0][d] = mfma16x16x32<DT>(vf, w[part][0], o[0][d]);
      }
      __builtin_amdgcn_wave_barrier();

      while (odd) {
        const int i = __ffs(odd) - 1;
        odd &= odd - 1;
        add_odd_value<DT>(vbase + __shfl(here, i), i, a.dim, col, quad, w, 0, o[0]);
      }
    }

    // Join the waves.
    l[0] += __shfl_xor(l[0], 16);
    l[0] += __shfl_xor(l[0], 32);
    if (quad == 0) {
      row_max[wave][col] = weight_base<DT>(m[0], c);
      row_sum[wave][col] = l[0];
    }
    __syncthreads();  // every wave is done with its values
#pragma unroll
    for (int d = 0; d < OT; ++d)
      *reinterpret_cast<f32x4*>(join + (wave * ROWS + col) * JP + d * 16 + quad * 4) = o[0][d];
    __syncthreads();
    float* slot = nullptr;
    if (to - from < it.tiles)
      slot = space(a).slots + (int64_t)slot_of(it.part, it.part_cost, it.line + it.cost) * slot_floats<DP, ROWS>();
    for (int e = threadIdx.x; e < ROWS * DP / 4; e += W * kWave) {
      const int i = e / (DP / 4), cc = e % (DP / 4) * 4, row = row0 + i;
      if (row >= rows) continue;
      float top = row_max[0][i];
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, row_max[w][i]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = __builtin_amdgcn_exp2f(row_max[w][i] - base);
        sum += f * row_sum[w][i];
        x += *reinterpret_cast<const f32x4*>(join + (w * ROWS + i) * JP + cc) * f;
      }
      if (slot) {
        *reinterpret_cast<f32x4*>(slot + i * DP + cc) = x;
        if (cc == 0) {
          slot[ROWS * DP + i] = top;
          slot[ROWS * DP + ROWS + i] = sum;
        }
        continue;
      }
      const int t = it.s.q0 + row / group, h = it.h * group + row % group;
      if (a.lse && cc == 0) a.lse[(int64_t)t * a.heads + h] = log_sum(base, sum);
      store_quad<DT>(a, t, h, cc, x, sum == 0.f ? 0.f : 1.f / sum);
    }
    }
    if (WHOLE || it.line + it.cost + it.tiles >= it.end) return;
    __syncthreads();
    next_line<ROWS, TILE>(a, &it);
  }
}

// ---------------------------------------------------------------- many rows
// Waves of a workgroup take different rows (16 RT each) and share the tile of
// positions in LDS, double-buffered; half of the next tile at a time is on its
// way in registers while this one is used (all of it at once spills 31 more).  A
// tile costs one barrier.
// 128 rows (48-node trees of 16 sequences, 6000 positions at most, 64 heads over
// 8): 143 us for 67 GFLOP that rows see, 126 where keys and values are in the
// last-level cache; two waves a SIMD is what 256 registers a wave leave (dim 128
// spills 17 of them, 72 bytes a lane; dim 256 with 64 rows 41).  Without the loads
// 104 us remained, without the exponentials 139, without either product 128 to
// 136: bound by latencies.  18 us go to each 1000 positions of context, 40 to
// starts and ends of lines.  64 rows (two sequences of 24 to 40 rows, 180000
// positions, 369 MB): 77 us, 4.8 TB/s, bound by memory.
template <int DT, int DP, int RT>
__global__ void __launch_bounds__(kWaves* kWave, 2) attention_rows_kernel(AttnArgs a) {
  constexpr int ROWS = kWaves * 16 * RT;
  constexpr int KEYS = wide_tile<DP>();
  constexpr int PARTS = weight_parts<DP, ROWS>();
  constexpr int KS = DP / 32, OT = DP / 16;
  constexpr int KP = DP + 8, VP = DP + 16;   // pitches: key rows 4 banks apart, value rows 8
  constexpr int CPR = DP / 8;                // 16-byte pieces of a row
  constexpr int RPP = kWaves * kWave / CPR;  // rows per pass
  constexpr int PASS = KEYS / RPP;
  __shared__ __align__(16) uint16_t kt[2][KEYS * KP];
  __shared__ __align__(16) uint16_t vt[2][KEYS * VP];
  __shared__ int64_t where[4][KEYS];         // cache rows of a tile's positions (0 where there is none)
  __shared__ uint32_t odd_rows[2][KEYS / 32];

  Place it;
  if (!find_part<ROWS, KEYS, line_cost<ROWS>()>(a, &it)) return;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane & 15, quad = lane >> 4;
  const int group = a.heads / a.kv_heads;
  const float c = exponent_scale(a);
  const int piece = tid % CPR * 8, prow = tid / CPR;
  const int clamped = piece < a.dim ? piece : a.dim - 8;
  // Key columns beyond dim are never written again: they have to be finite.
  if (a.dim < DP) {
    for (int e = tid; e < KEYS * KP / 8; e += kWaves * kWave)
      reinterpret_cast<u32x4*>(kt[0])[e] = reinterpret_cast<u32x4*>(kt[1])[e] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
  }

  for (;;) {
    const int rows = it.s.n * group, row0 = it.rt * ROWS + wave * 16 * RT;
    const int from = max(it.at - it.line - it.cost, 0), to = min(it.tiles, it.end - it.line - it.cost);
    if (to > from) {
    const int begin = from * KEYS, end = min(it.s.len, to * KEYS);

    u32x4 q[RT][KS];
    int node[RT];
    uint64_t word[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = min(row0 + r * 16 + col, rows - 1);
      node[r] = row / group;
      word[r] = first_mask_word(a, it, node[r]);
      load_queries<DP>(a, it, node[r], it.h * group + row % group, quad, q[r]);
    }
    const uint16_t* vhead = a.v + it.h * a.kv_head;
    const uint16_t* kbase = a.k + it.h * a.kv_head + clamped;  // of this thread's pieces
    const uint16_t* vbase = vhead + clamped;
    const int32_t* table = a.table + (int64_t)it.b * a.ld_table;

    f32x4 o[RT][OT];
    float m[RT], l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < OT; ++d) o[r][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    u32x4 reg[PASS];  // the next tile's keys during the first half of this one, its values after that
    // Page of a position of tile n (each wave looks up all of them), and the
    // cache row that follows from it.  The two are apart so that the page is on
    // its way during a whole tile.
    auto find_page = [&](int n) {
      return table[page_of_position(a, min(begin + n * KEYS + tid % KEYS, max(end - 1, 0)))];
    };
    // Notes the cache rows of tile n; returns a bit for each that exists.
    auto note_rows = [&](int n, int page) {
      const int pos = begin + n * KEYS + tid % KEYS;
      const int64_t at = pos < end ? cache_row(a, page, page_of_position(a, pos), pos) : (int64_t)-1;
      where[n & 3][tid % KEYS] = at < 0 ? 0 : at;
      return (uint64_t)__ballot(at >= 0);
    };
    // Tile n's keys and values on their way into the registers, and from there
    // into its buffer.  Value rows that do not exist are staged as 0; so are
    // those that are not finite, which are noted (with weights in one part, which
    // are never below 0, only where rows differ in what they see).
    auto fetch = [&](int n, const uint16_t* base) {
#pragma unroll
      for (int i = 0; i < PASS; ++i) reg[i] = *reinterpret_cast<const u32x4*>(base + where[n & 3][prow + i * RPP]);
    };
    auto stash_keys = [&](int n) {
      if (piece < a.dim) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) *reinterpret_cast<u32x4*>(&kt[n & 1][(prow + i * RPP) * KP + piece]) = reg[i];
      }
    };
    auto all_there = [](uint64_t there) { return KEYS == 64 ? !~there : (uint32_t)there == ~0u; };
    // Whether every row sees all of tile n.
    auto plain = [&](int n, uint64_t there) { return begin + (n + 1) * KEYS <= it.s.ctx && all_there(there); };
    auto stash_values = [&](int n, uint64_t there) {
      if (PARTS == 2 || !plain(n, there)) {
        if (PARTS == 1 || !all_there(there)) {
#pragma unroll
          for (int i = 0; i < PASS; ++i)
            if (!((there >> (prow + i * RPP)) & 1)) reg[i] = u32x4{0u, 0u, 0u, 0u};
        }
        if (__builtin_expect(__any(not_finite<DT>(reg)), 0)) {
#pragma unroll
          for (int i = 0; i < PASS; ++i) {
            const int r = prow + i * RPP, first = lane / CPR * CPR;
            const uint64_t lanes = __ballot(not_finite<DT>(reg[i]));
            const bool odd = lanes && ((lanes >> first) & ((1ull << CPR) - 1ull));
            if (odd && lane == first) atomicOr(&odd_rows[n & 1][r / 32], 1u << (r % 32));
            if (odd) reg[i] = u32x4{0u, 0u, 0u, 0u};
          }
        }
      }
      if (piece < a.dim) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) *reinterpret_cast<u32x4*>(&vt[n & 1][(prow + i * RPP) * VP + piece]) = reg[i];
      }
    };

    const int tiles = end > begin ? (end - begin + KEYS - 1) / KEYS : 0;
    uint64_t there0 = 0, there1 = 0, there2 = 0;  // positions of tiles n, n + 1, n + 2
    if (tid < 2 * (KEYS / 32)) odd_rows[tid / (KEYS / 32)][tid % (KEYS / 32)] = 0;
    if (tiles > 0) {
      int page[3];
#pragma unroll
      for (int n = 0; n < 3; ++n) page[n] = find_page(n);
      there0 = note_rows(0, page[0]);
      there1 = note_rows(1, page[1]);
      there2 = note_rows(2, page[2]);
    }
    __syncthreads();
    if (tiles > 0) {
      fetch(0, kbase);
      stash_keys(0);
      fetch(0, vbase);
      stash_values(0, there0);
      fetch(1, kbase);
    }
    __syncthreads();

    for (int n = 0; n < tiles; ++n) {
      const int later = find_page(n + 3);
      const uint16_t* kb = kt[n & 1];
      const uint16_t* vb = vt[n & 1];
      // A wave whose rows all lie beyond the line's only helps with the staging.
      // In each half tile all key operands are read before the products that take
      // them, all value operands before the softmax: left to itself the compiler
      // reads each when it is due and waits for LDS every time.
#pragma unroll
      for (int half = 0; half < KEYS / 32; ++half) {
        if (half == KEYS / 32 - 1) {  // the next tile's keys are there: its values' turn
          stash_keys(n + 1);
          fetch(n + 1, vbase);
        }
        if (row0 >= rows) continue;
        const int key0 = begin + n * KEYS + half * 32;
        const uint32_t there = (uint32_t)(there0 >> (half * 32));
        u32x4 kf[2][KS];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int s = 0; s < KS; ++s)
            kf[t][s] = *reinterpret_cast<const u32x4*>(kb + (half * 32 + t * 16 + col) * KP + s * 32 + quad * 8);
        __builtin_amdgcn_sched_barrier(0);
        f32x4 sc[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int t = 0; t < 2; ++t) sc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) sc[r][t] = mfma16x16x32<DT>(kf[t][s], q[r][s], sc[r][t]);
        if (__builtin_expect(key0 + 32 > it.s.ctx || there != 0xffffffffu, 0)) {
#pragma unroll
          for (int r = 0; r < RT; ++r) mask_scores(seen_bits(a, it, node[r], word[r], key0, there), quad, sc[r]);
        }
        u32x4 vf[OT];
#pragma unroll
        for (int d = 0; d < OT; ++d) {
          const uint16_t* p = vb + (half * 32 + quad * 4 + (col >> 2)) * VP + d * 16 + (col & 3) * 4;
          const u32x2 lo = lds_read_transposed(p), hi = lds_read_transposed(p + 16 * VP);
          vf[d] = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
        __builtin_amdgcn_sched_barrier(0);
        u32x4 w[PARTS][RT];
        weigh<DT, PARTS, RT, OT>(sc, c, m, l, o, w);
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int d = 0; d < OT; ++d)
#pragma unroll
            for (int r = 0; r < RT; ++r) o[r][d] = mfma16x16x32<DT>(vf[d], w[part][r], o[r][d]);
        uint32_t odd = odd_rows[n & 1][half];
        while (__builtin_expect(odd != 0, 0)) {
          const int i = __ffs(odd) - 1;
          odd &= odd - 1;
          const uint16_t* p = vhead + where[n & 3][half * 32 + i];
#pragma unroll
          for (int r = 0; r < RT; ++r) add_odd_value<DT>(p, i, a.dim, col, quad, w, r, o[r]);
        }
      }
      // Buffer n & 1 is free after the barrier.  Its notes of odd rows, which every
      // wave reads before, are cleared between two barriers where there are any.
      stash_values(n + 1, there1);
      const bool noted = __builtin_amdgcn_readfirstlane(odd_rows[n & 1][0] | odd_rows[n & 1][KEYS / 32 - 1]) != 0;
      there0 = there1;
      there1 = there2;
      there2 = note_rows(n + 3, later);
      __syncthreads();
      if (noted) {
        if (tid < KEYS / 32) odd_rows[n & 1][tid] = 0;
        __syncthreads();
      }
      fetch(n + 2, kbase);
    }

    float* slot = nullptr;
    if (to - from < it.tiles)
      slot = space(a).slots + (int64_t)slot_of(it.part, it.part_cost, it.line + it.cost) * slot_floats<DP, ROWS>();
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float sum = l[r];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      const int in_tile = (wave * RT + r) * 16 + col, row = row0 + r * 16 + col;
      if (row >= rows) continue;
      const float top = weight_base<DT>(m[r], c), base = m[r] == -INFINITY ? 0.f : top;
      if (slot) {
#pragma unroll
        for (int d = 0; d < OT; ++d) *reinterpret_cast<f32x4*>(slot + in_tile * DP + d * 16 + quad * 4) = o[r][d];
        if (quad == 0) {
          slot[ROWS * DP + in_tile] = top;
          slot[ROWS * DP + ROWS + in_tile] = sum;
        }
        continue;
      }
      const int t = it.s.q0 + row / group, h = it.h * group + row % group;
      if (a.lse && quad == 0) a.lse[(int64_t)t * a.heads + h] = log_sum(base, sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int d = 0; d < OT; ++d) store_quad<DT>(a, t, h, d * 16 + quad * 4, o[r][d], inv);
    }
    }
    if (it.line + it.cost + it.tiles >= it.end) return;
    next_line<ROWS, KEYS>(a, &it);
  }
}

// ---------------------------------------------------------------- join of pieces
// For few rows, whose lines are cut into many pieces: a block of eight waves
// joins one row (token, head), wave w taking pieces w, w + 8, ...; 64 lanes hold
// the DP columns.  A wave reads a batch of pieces at once, with a running maximum
// and sum over the batches, so that few memory latencies follow the look-ups:
// 256 rows of some 85 pieces each in 8 us.
constexpr int kJoinWaves = 8;

template <int DT, int DP, int ROWS, int KEYS>
__global__ void __launch_bounds__(kJoinWaves* kWave) join_kernel(AttnArgs a) {
  constexpr int PER = DP / kWave;
  const Space sp = space(a);
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t = blockIdx.x / a.heads, head = blockIdx.x % a.heads;
  const int group = a.heads / a.kv_heads;
  // The sequence of token t.
  int b = -1;
  for (int base = 0; base < a.B && b < 0; base += kWave) {
    const bool mine = base + lane < a.B && a.start[base + lane] <= t && t < a.start[base + lane + 1];
    const uint64_t m = __ballot(mine);
    if (m) b = base + __ffsll((unsigned long long)m) - 1;
  }
  if (b < 0) return;
  const Seq s = sequence(a, b);
  const int part_cost = sp.part[0], cost = sp.part[1];
  if (part_cost == 0) return;
  const int tiles = key_tiles(s.len, KEYS), rts = row_tiles(s.n, group, ROWS);
  const int row = (t - s.q0) * group + head % group, rt = row / ROWS, in_tile = row % ROWS;
  const int tiles0 = sp.first[b] + (head / group * rts + rt) * (cost + tiles) + cost;
  const int part0 = tiles0 / part_cost, splits = min((tiles0 + tiles - 1) / part_cost, kParts - 1) - part0 + 1;
  if (splits < 2) return;
  auto piece = [&](int i) {
    return sp.slots + (int64_t)slot_of(part0 + i, part_cost, tiles0) * slot_floats<DP, ROWS>();
  };
  constexpr int BATCH = 12;
  float top = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int i0 = wave; i0 < splits; i0 += kJoinWaves * BATCH) {
    float m[BATCH], l[BATCH], v[BATCH][PER];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {  // pieces beyond the last: the last one, with no weight
      const float* p = piece(min(i0 + i * kJoinWaves, splits - 1));
      m[i] = p[ROWS * DP + in_tile];
      l[i] = p[ROWS * DP + ROWS + in_tile];
      if constexpr (PER == 1) {
        v[i][0] = p[in_tile * DP + lane];
      } else {
        typedef float Vec __attribute__((ext_vector_type(PER)));
        const Vec x = *reinterpret_cast<const Vec*>(p + in_tile * DP + lane * PER);
#pragma unroll
        for (int e = 0; e < PER; ++e) v[i][e] = x[e];
      }
    }
    float now = top;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) now = fmaxf(now, m[i]);
    const float base = now == -INFINITY ? 0.f : now;
    const float shrink = __builtin_amdgcn_exp2f(top - base);
    sum *= shrink;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= shrink;
    top = now;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (i0 + i * kJoinWaves >= splits) continue;
      const float f = __builtin_amdgcn_exp2f(m[i] - base);
      sum += f * l[i];
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] += f * v[i][e];
    }
  }
  {
    __shared__ float part[kJoinWaves][DP + 2];
#pragma unroll
    for (int e = 0; e < PER; ++e) part[wave][lane * PER + e] = acc[e];
    if (lane == 0) {
      part[wave][DP] = sum;
      part[wave][DP + 1] = top;
    }
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) top = fmaxf(top, part[w][DP + 1]);
    const float base = top == -INFINITY ? 0.f : top;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(part[w][DP + 1] - base);
      sum += f * part[w][DP];
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] += f * part[w][lane * PER + e];
    }
  }
  const float base = top == -INFINITY ? 0.f : top;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = a.out + t * a.out_token + head * a.out_head;
#pragma unroll
  for (int e = 0; e < PER; ++e)
    if (lane * PER + e < a.dim) out[lane * PER + e] = (uint16_t)from_f32<DT>(acc[e] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.heads + head] = log_sum(base, sum);
}

// For many rows: blocks take lines, kSlice rows of each (blockIdx.y), so that one
// look-up serves them and a line that was not cut costs one short block; a wave
// has four rows' pieces on their way at once.  48-node trees of 16 sequences, 64
// heads: 21 us (24 with a wave for each row), 4 us where no line is cut (16).
constexpr int kSlice = 32;

template <int DT, int DP, int ROWS, int KEYS>
__global__ void __launch_bounds__(kWaves* kWave) join_lines_kernel(AttnArgs a) {
  constexpr int PER = DP / kWave, AT_ONCE = 4, BATCH = DP == 256 ? 2 : 3;
  constexpr int SLICE = ROWS < kSlice ? ROWS : kSlice;
  typedef float Vec __attribute__((ext_vector_type(PER == 1 ? 2 : PER)));
  Place it;
  if (!find_line<ROWS, KEYS>(a, &it)) return;
  const Space sp = space(a);
  const int part_cost = sp.part[0], cost = sp.part[1];
  if (part_cost == 0) return;
  const int tiles0 = sp.first[it.b] + (it.h * it.rts + it.rt) * (cost + it.tiles) + cost;
  const int part0 = tiles0 / part_cost, splits = min((tiles0 + it.tiles - 1) / part_cost, kParts - 1) - part0 + 1;
  if (splits < 2) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = a.heads / a.kv_heads, rows = it.s.n * group, row0 = it.rt * ROWS;
  auto piece = [&](int i) {
    return sp.slots + (int64_t)slot_of(part0 + i, part_cost, tiles0) * slot_floats<DP, ROWS>();
  };
  for (int r0 = blockIdx.y * SLICE + wave * AT_ONCE; r0 < (blockIdx.y + 1) * SLICE && row0 + r0 < rows;
       r0 += kWaves * AT_ONCE) {
    float top[AT_ONCE], sum[AT_ONCE], acc[AT_ONCE][PER];
#pragma unroll
    for (int r = 0; r < AT_ONCE; ++r) {
      top[r] = -INFINITY;
      sum[r] = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[r][e] = 0.f;
    }
    for (int i0 = 0; i0 < splits; i0 += BATCH) {
      float m[BATCH][AT_ONCE], l[BATCH][AT_ONCE], v[BATCH][AT_ONCE][PER];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {  // pieces beyond the last: the last one, with no weight
        const float* p = piece(min(i0 + i, splits - 1));
#pragma unroll
        for (int r = 0; r < AT_ONCE; ++r) {
          m[i][r] = p[ROWS * DP + r0 + r];
          l[i][r] = p[ROWS * DP + ROWS + r0 + r];
          if constexpr (PER == 1) {
            v[i][r][0] = p[(r0 + r) * DP + lane];
          } else {
            const Vec x = *reinterpret_cast<const Vec*>(p + (r0 + r) * DP + lane * PER);
#pragma unroll
            for (int e = 0; e < PER; ++e) v[i][r][e] = x[e];
          }
        }
      }
#pragma unroll
      for (int r = 0; r < AT_ONCE; ++r) {
        float now = top[r];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) now = fmaxf(now, m[i][r]);
        const float base = now == -INFINITY ? 0.f : now;
        const float shrink = __builtin_amdgcn_exp2f(top[r] - base);
        sum[r] *= shrink;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[r][e] *= shrink;
        top[r] = now;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          if (i0 + i >= splits) continue;
          const float f = __builtin_amdgcn_exp2f(m[i][r] - base);
          sum[r] += f * l[i][r];
#pragma unroll
          for (int e = 0; e < PER; ++e) acc[r][e] += f * v[i][r][e];
        }
      }
    }
#pragma unroll
    for (int r = 0; r < AT_ONCE; ++r) {
      const int row = row0 + r0 + r;
      if (row >= rows) continue;
      const int t = it.s.q0 + row / group, head = it.h * group + row % group;
      const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
      uint16_t* out = a.out + t * a.out_token + head * a.out_head;
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (lane * PER + e < a.dim) out[lane * PER + e] = (uint16_t)from_f32<DT>(acc[r][e] * inv);
      if (a.lse && lane == 0)
        a.lse[(int64_t)t * a.heads + head] = log_sum(top[r] == -INFINITY ? 0.f : top[r], sum[r]);
    }
  }
}

// Most lines a call can have: every sequence has at most one row tile that is
// not full.
int64_t line_bound(int32_t B, int32_t T, int32_t heads, int32_t kv_heads, int tile_rows) {
  const int64_t rows = (int64_t)T * (heads / kv_heads);
  return (rows / tile_rows + (B < rows ? B : rows)) * kv_heads;
}
int64_t line_bound(const AttnArgs& a, int tile_rows) { return line_bound(a.B, a.T, a.heads, a.kv_heads, tile_rows); }

// ROWS = 16: the kernel for few rows; 64, 128: the one for many.
template <int DT, int DP, int ROWS>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
  constexpr int KEYS = ROWS > 16 ? wide_tile<DP>() : kTile;
  if constexpr (ROWS > 16)
    attention_rows_kernel<DT, DP, ROWS / 64><<<kParts, kWaves * kWave, 0, s>>>(a);
  else
    attention_kernel<DT, DP, kWaves, false><<<kParts, kWaves * kWave, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t out_rows = (int64_t)a.T * a.heads;
  if (out_rows <= kCus * 8) {
    join_kernel<DT, DP, ROWS, KEYS><<<(unsigned)out_rows, kJoinWaves * kWave, 0, s>>>(a);
  } else {
    const dim3 grid((unsigned)line_bound(a, ROWS), (ROWS + kSlice - 1) / kSlice);
    join_lines_kernel<DT, DP, ROWS, KEYS><<<grid, kWaves * kWave, 0, s>>>(a);
  }
  return hipGetLastError();
}

// Whether the table holds so few positions that a workgroup of eight waves takes
// each line whole: 509 positions, one token, 32 heads: 8.7 us and 3.9 us of the
// join's launch in parts.
bool short_lines(int64_t positions) { return positions <= kShortLine; }

// Waves of a workgroup that takes whole lines: what the registers allow.
constexpr int short_waves(int dp) { return dp == 256 ? 4 : 8; }

template <int DT, int DP>
hipError_t launch_short(const AttnArgs& a, hipStream_t s) {
  constexpr int W = short_waves(DP);
  attention_kernel<DT, DP, W, true><<<(unsigned)line_bound(a, 16), W * kWave, 0, s>>>(a);
  return hipGetLastError();
}

// Rows of a line, from what an average sequence has.  16 rows: the waves split
// the positions, which measured best there (64 sequences of one token, 8 rows
// each: 124 us against 173 us with 64).  Above, the waves split the rows: 64
// (two sequences of 32 rows on average over 120000 positions: 82 us against
// 122 us with two row tiles whose waves split the positions) or 128.
// 256-wide heads leave registers for 64 only.
int choose_rows(int64_t B, int64_t T, int group, int dp) {
  const int64_t rows = (T * group + B - 1) / B;
  return rows <= 16 ? 16 : rows <= 64 || dp == 256 ? 64 : 128;
}

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

template <int DT, int DP>
hipError_t launch_rows(const AttnArgs& a, int rows, hipStream_t s) {
  if (rows == 16)
    return short_lines((int64_t)a.max_pages * a.page_size) ? launch_short<DT, DP>(a, s) : launch<DT, DP, 16>(a, s);
  if constexpr (DP != 256) {
    if (rows == 128) return launch<DT, DP, 128>(a, s);
  }
  return launch<DT, DP, 64>(a, s);
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s) {
  const int dp = padded_dim(a.dim), rows = choose_rows(a.B, a.T, a.heads / a.kv_heads, dp);
  return dp == 64 ? launch_rows<DT, 64>(a, rows, s)
                  : dp == 128 ? launch_rows<DT, 128>(a, rows, s) : launch_rows<DT, 256>(a, rows, s);
}

}  // namespace

int64_t attention_threads(int32_t B, int32_t T, int32_t heads, int32_t kv_heads, int32_t dim, int64_t positions) {
  const int dp = padded_dim(dim), rows = choose_rows(B, T, heads / kv_heads, dp);
  const int waves = rows == 16 && short_lines(positions) ? short_waves(dp) : kWaves;
  return line_bound(B, T, heads, kv_heads, rows) * waves * kWave;
}

size_t attention_workspace(int32_t B, int32_t T, int32_t heads, int32_t kv_heads, int32_t dim) {
  const int dp = padded_dim(dim), rows = choose_rows(B, T, heads / kv_heads, dp);
  return (4 + ((size_t)B + 3) / 4 * 4 + (size_t)2 * kParts * rows * (dp + 2)) * 4;
}

hipError_t launch_attention(const AttnArgs& args, int dtype, hipStream_t s) {
  AttnArgs a = args;
  if (a.num_pages == 0) {  // nothing is there to be read: any legal address will do
    a.k = a.v = a.q;
    a.kv_head = 0;
  }
  a.page_mul = a.page_shift = 0;
  if (a.page_size > 1) {
    const int bits = 32 - __builtin_clz((uint32_t)(a.page_size - 1));
    a.page_mul = (uint32_t)(((1ull << (31 + bits)) + a.page_size - 1) / a.page_size);
    a.page_shift = bits - 1;
  }
  return dtype == 0 ? launch_dt<0>(a, s) : launch_dt<1>(a, s);
}

}  // namespace lora
