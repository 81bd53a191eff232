// Page operations of a paged key / value cache (lora_pages_*): allocation,
// reference counts, copies.
//
// Allocation is a scan of the reference counts for zeros by one workgroup:
// there is no free list whose order could depend on timing, and releasing a
// page is one atomic decrement.  Everything that moves cache rows runs as 16
// bytes per lane over many workgroups.
#include "decode_kernels.h"
#include "lora_device.h"

namespace lora {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanItems = 16;  // counts per thread and round: 64 KiB of counts a round
constexpr int kOk = 0, kNoSpace = 1, kBad = 2;

__device__ __forceinline__ bool in_range(int32_t v, int32_t n) { return (uint32_t)v < (uint32_t)n; }

// Whether entry i names the same id as an earlier entry.  Every thread of the
// block must call it.
__device__ __forceinline__ bool repeated(const int32_t* __restrict__ ids, int i) {
  bool same = false;
  const int32_t id = ids[i];
  for (int j = threadIdx.x; j < i; j += blockDim.x) same |= ids[j] == id;
  return __syncthreads_or(same);
}

// Calls give(rank, page) for the first `total` free pages in ascending order,
// rank 0 first.  Returns how many there were (at most total).  One block of
// kScanThreads; scratch: kScanThreads / 64 + 1 ints.
template <typename Give>
__device__ __forceinline__ int scan_free(const int32_t* __restrict__ refs, int32_t num_pages, int total,
                                         int* scratch, Give give) {
  int found = 0;
  for (int64_t base = 0; base < num_pages && found < total; base += kScanThreads * kScanItems) {
    const int64_t p0 = base + (int64_t)threadIdx.x * kScanItems;
    uint32_t zero = 0;
    int32_t count[kScanItems];
#pragma unroll
    for (int e = 0; e < kScanItems; ++e) count[e] = refs[min(p0 + e, (int64_t)num_pages - 1)];
#pragma unroll
    for (int e = 0; e < kScanItems; ++e)
      if (p0 + e < num_pages && count[e] == 0) zero |= 1u << e;
    int round;
    int rank = found + block_exclusive_sum<kScanThreads>(__popc(zero), scratch, &round);
    while (zero) {
      const int e = __ffs(zero) - 1;
      zero &= zero - 1;
      if (rank < total) give(rank, (int32_t)(p0 + e));
      ++rank;
    }
    found += round;
  }
  return found < total ? found : total;
}

// Number of leading entries >= 0 of a table row, by a whole wave: 64 probes a
// step.
__device__ __forceinline__ int row_pages(const int32_t* __restrict__ row, int max_pages) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, hi = max_pages;  // entries below lo are >= 0, the first < 0 is at or before hi
  while (lo < hi) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int at = lo + lane * step;
    const bool held = at < hi && row[at] >= 0;
    const uint64_t m = __ballot(held);
    const int leading = m == ~0ull ? kWave : __ffsll((unsigned long long)~m) - 1;
    if (leading == 0) return lo;
    const int last = lo + (leading - 1) * step;  // the last probe that was held
    hi = last + step < hi ? last + step : hi;
    lo = last + 1;
  }
  return lo;
}

// Pages of `tokens` tokens (tokens >= 0).
__device__ __forceinline__ int64_t pages_of(int64_t tokens, int page_size) {
  return (tokens + page_size - 1) / page_size;
}

// ---------------------------------------------------------------- copies
// Whole pages are moved 16 bytes a lane, past the caches' normal replacement:
// nothing here reads them again.  One block moves one piece of kPiece bytes with
// one load a lane.  That measured best: 200 pages of 32 KiB in 64 pools take
// 146 us (5.7 TB/s read and written) against 157 with 32 KiB a block and 167
// without the non-temporal hint; loads that are each in a condition of their
// own (a tail test for every load of a lane) wait for one another: 223 us.
constexpr int kPiece = 4096;

__device__ __forceinline__ u32x4 load_row(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}
__device__ __forceinline__ void store_row(uint8_t* p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
}

// Block (piece, entry, pool).
__global__ void __launch_bounds__(256) copy_kernel(PageView c, const int32_t* __restrict__ src,
                                                   const int32_t* __restrict__ dst, int64_t page_bytes) {
  const int32_t a = src[blockIdx.y], b = dst[blockIdx.y];
  const int64_t at = (int64_t)blockIdx.x * kPiece + threadIdx.x * 16;
  if (!in_range(a, c.num_pages) || !in_range(b, c.num_pages) || a == b || at >= page_bytes) return;
  uint8_t* pool = c.pool + blockIdx.z * c.pool_stride + at;
  store_row(pool + b * c.page_stride, load_row(pool + a * c.page_stride));
}

// ---------------------------------------------------------------- resize
// A page at or behind a sequence's new end that other sequences hold too (the
// row was forked and is cut now) is replaced by one of the sequence's own, so
// that no append reaches the others; the one that the end lies in keeps its
// filled rows.  Counts as they were before the call decide, so entries that cut
// the same page at once each get their own.  A fresh page that still has to
// receive rows is marked by its count, ~(page to copy from), until the second
// kernel has copied them; its last slot, which is not filled, holds a note.
// Calls in a row, with lengths and without (one launch less): 7.1 and 4.2 us for
// one entry, 8.8 and 5.2 for 48, 26 and 20 for 256.  48 branches cut inside a
// shared page, 101 MB read and written in 64 pools: 47 us.
struct CutNote {
  int32_t done;   // blocks that have copied their part
  int32_t entry;  // whose page it is
};

__device__ __forceinline__ CutNote* cut_note(const PageView& c, int32_t page) {
  return reinterpret_cast<CutNote*>(c.pool + page * c.page_stride + (c.page_size - 1) * c.row_bytes);
}

__global__ void __launch_bounds__(kScanThreads) resize_kernel(PageView c, const int32_t* __restrict__ seqs,
                                                              const int32_t* __restrict__ lens,
                                                              const int32_t* __restrict__ extra, int n,
                                                              int32_t* __restrict__ status) {
  __shared__ int scratch[kScanThreads / kWave + 1];
  __shared__ int32_t ids[kMaxPageEntries];
  __shared__ int end[kMaxPageEntries];    // inclusive prefix of the pages needed
  __shared__ int held[kMaxPageEntries];   // pages held before; -1: bad entry
  __shared__ int want[kMaxPageEntries];
  __shared__ int cut[kMaxPageEntries];    // first entry of the row that is replaced
  __shared__ int own[kMaxPageEntries];    // how many are
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int i = tid; i < n; i += kScanThreads) ids[i] = seqs[i];
  __syncthreads();
  for (int i = wave; i < n; i += kScanThreads / kWave) {
    const int32_t s = ids[i];
    bool same = false;
    for (int j = lane; j < i; j += kWave) same |= ids[j] == s;
    bool good = in_range(s, c.max_seqs) && !__any(same);
    int have = 0;
    int64_t need = 0;
    if (good) {
      const int32_t len = lens ? lens[i] : c.seq_len[s];
      const int32_t more = extra ? extra[i] : 0;
      need = pages_of((int64_t)len + more, c.page_size);
      good = len >= 0 && more >= 0 && need <= c.max_pages;
      if (good) have = row_pages(c.table + (int64_t)s * c.ld_table, c.max_pages);
    }
    if (lane == 0) {
      held[i] = good ? have : -1;
      want[i] = good ? (int)need : 0;
      own[i] = 0;
    }
  }
  __syncthreads();
  if (lens) {
    // A thread looks at an entry that keeps one such page, a wave at one that
    // keeps more (room for many tokens to come).
    auto kept = [&](int i) { return min(held[i], want[i]); };
    auto shared = [&](int i, int w) {
      const int32_t p = c.table[(int64_t)ids[i] * c.ld_table + w];
      return in_range(p, c.num_pages) && c.refs[p] > 1;
    };
    for (int i = tid; i < n; i += kScanThreads) {
      cut[i] = held[i] < 0 ? 0 : lens[i] / c.page_size;
      if (cut[i] + 1 == kept(i)) own[i] = shared(i, cut[i]);
    }
    __syncthreads();
    for (int i = wave; i < n; i += kScanThreads / kWave) {
      if (cut[i] + 1 >= kept(i)) continue;
      int last = cut[i] - 1;
      for (int w0 = cut[i]; w0 < kept(i); w0 += kWave) {
        const uint64_t m = __ballot(w0 + lane < kept(i) && shared(i, w0 + lane));
        if (m) last = w0 + kWave - 1 - __clzll((long long)m);
      }
      if (lane == 0) own[i] = last - cut[i] + 1;
    }
    __syncthreads();
  }
  auto needs = [&](int i) { return held[i] < 0 ? 0 : own[i] + max(want[i] - held[i], 0); };
  // Prefix sums of what each entry needs (a sum never passes 2^31: at most
  // kMaxPageEntries rows of max_pages entries, which the host has checked).
  int before = 0;
  for (int base = 0; base < n; base += kScanThreads) {
    const int i = base + tid;
    const int need = i < n ? needs(i) : 0;
    int sum;
    const int excl = block_exclusive_sum<kScanThreads>(need, scratch, &sum);
    if (i < n) end[i] = before + excl + need;
    before += sum;
  }
  __syncthreads();
  // Where the r-th page that entry i receives goes in its row.
  auto place = [&](int i, int r) { return r < own[i] ? cut[i] + r : held[i] + r - own[i]; };
  const int found = scan_free(c.refs, c.num_pages, before, scratch, [&](int rank, int32_t page) {
    // The entry whose range of ranks holds this one.  Entries that turn out
    // not to be served as a whole give their pages back below.
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (end[mid] > rank) hi = mid; else lo = mid + 1;
    }
    const int r = rank - (end[lo] - needs(lo));
    int32_t* at = c.table + (int64_t)ids[lo] * c.ld_table + place(lo, r);
    c.refs[page] = r < own[lo] ? ~*at : 1;
    *at = page;
  });
  __syncthreads();
  for (int i = wave; i < n; i += kScanThreads / kWave) {
    if (held[i] < 0) {
      if (status && lane == 0) status[i] = kBad;
      continue;
    }
    const int32_t s = ids[i];
    int32_t* row = c.table + (int64_t)s * c.ld_table;
    const int need = needs(i), got = min(max(found - (end[i] - need), 0), need);
    const bool fits = got == need;
    if (fits) {
      for (int r = lane; r < own[i]; r += kWave) {
        const int32_t page = row[cut[i] + r], old = ~c.refs[page];
        const bool there = in_range(old, c.num_pages);
        if (there) atomicSub(&c.refs[old], 1);
        if (r == 0 && there && lens[i] % c.page_size != 0)
          *cut_note(c, page) = CutNote{0, i};
        else
          c.refs[page] = 1;
      }
      for (int w = want[i] + lane; w < held[i]; w += kWave) {  // the tail of a shrinking row
        const int32_t p = row[w];
        if (in_range(p, c.num_pages)) atomicSub(&c.refs[p], 1);
        row[w] = -1;
      }
    } else {
      for (int r = lane; r < got; r += kWave) {  // what an unserved entry received
        int32_t* at = row + place(i, r);
        const int32_t page = *at;
        *at = r < own[i] ? ~c.refs[page] : -1;
        c.refs[page] = 0;
      }
    }
    if (lane == 0) {
      if (lens && fits) c.seq_len[s] = lens[i];
      if (status) status[i] = fits ? kOk : kNoSpace;
    }
  }
}

// Blocks (i, 0 .. kCutBlocks - 1), which deal out the pools: the filled rows of
// the page that entry i's sequence was cut in, from the page that it gave up.
// Most entries have none: four dependent look-ups, and few blocks to make them.
// The last block to finish clears the mark, which the others have read by then.
constexpr int kCutBlocks = 8;

__global__ void __launch_bounds__(256) resize_copy_kernel(PageView c, const int32_t* __restrict__ seqs) {
  const int i = blockIdx.x;
  const int32_t s = seqs[i];
  if (!in_range(s, c.max_seqs)) return;
  const int32_t len = c.seq_len[s];
  const int w = len / c.page_size, rest = len % c.page_size;
  if (rest <= 0 || w >= c.max_pages) return;
  const int32_t fresh = c.table[(int64_t)s * c.ld_table + w];
  if (!in_range(fresh, c.num_pages)) return;
  const int32_t old = ~c.refs[fresh];
  if (!in_range(old, c.num_pages)) return;
  CutNote* note = cut_note(c, fresh);
  if (note->entry != i) return;  // a later entry that repeats the sequence
  const int per_chunk = (int)(rest * c.row_bytes / 16);
  for (int pool = blockIdx.y; pool < c.num_pools; pool += gridDim.y)
    for (int e = threadIdx.x; e < per_chunk * c.chunks; e += 256) {
      uint8_t* at = c.pool + pool * c.pool_stride + e / per_chunk * (c.page_size * c.row_bytes) + (int64_t)(e % per_chunk) * 16;
      store_row(at + fresh * c.page_stride, load_row(at + old * c.page_stride));
    }
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(&note->done, 1) == (int)gridDim.y - 1) c.refs[fresh] = 1;
}

// ---------------------------------------------------------------- fork
// Workspace of a fork: the sources' rows as they were before the call, then
// their lengths and the page each entry was given.
struct ForkSpace {
  int32_t* rows;   // [n][max_pages]
  int32_t* len;    // [n]
  int32_t* fresh;  // [n]: a page, -1: none needed, -2: not served, -3: bad entry
};
constexpr int kNone = -1, kUnserved = -2, kBadEntry = -3;

__device__ __forceinline__ bool fork_entry_good(const PageView& c, int32_t s, int32_t d) {
  if (!in_range(s, c.max_seqs) || !in_range(d, c.max_seqs)) return false;
  const int32_t len = c.seq_len[s];
  return len >= 0 && pages_of(len, c.page_size) <= c.max_pages;
}

// 5 us for 3 entries, 7 us for 96: dependent look-ups (ids, lengths, counts).
// Block 0 gives out the pages; block 1 + i saves the row of src[i] and counts
// dst[i] as an owner of its full pages.  The counts that block 0 looks for are
// zeros, those that the other blocks raise are not.
__global__ void __launch_bounds__(kScanThreads) fork_plan_kernel(PageView c, const int32_t* __restrict__ src,
                                                                 const int32_t* __restrict__ dst, int n,
                                                                 ForkSpace ws, int32_t* __restrict__ status) {
  if (blockIdx.x > 0) {
    const int i = blockIdx.x - 1;
    if (repeated(dst, i) || !fork_entry_good(c, src[i], dst[i])) return;
    const int32_t s = src[i], len = c.seq_len[s];
    const int full = len / c.page_size, used = (int)pages_of(len, c.page_size);
    if (threadIdx.x == 0) ws.len[i] = len;
    for (int w = threadIdx.x; w < used; w += kScanThreads) {
      const int32_t p = c.table[(int64_t)s * c.ld_table + w];
      ws.rows[(int64_t)i * c.max_pages + w] = p;
      if (w < full && in_range(p, c.num_pages)) atomicAdd(&c.refs[p], 1);
    }
    return;
  }
  __shared__ int scratch[kScanThreads / kWave + 1];
  __shared__ int32_t ids[kMaxPageEntries];
  __shared__ int32_t who[kMaxPageEntries];  // entry of the rank-th page
  __shared__ uint8_t needs[kMaxPageEntries];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int i = tid; i < n; i += kScanThreads) {
    const int32_t d = dst[i], s = src[i];
    ids[i] = d;
    const bool good = fork_entry_good(c, s, d);
    needs[i] = !good ? 2 : c.seq_len[s] % c.page_size != 0;
  }
  __syncthreads();
  // A wave looks for each entry's destination among the earlier ones.
  for (int i = wave; i < n; i += kScanThreads / kWave) {
    bool same = false;
    for (int j = lane; j < i; j += kWave) same |= ids[j] == ids[i];
    if (__any(same) && lane == 0) needs[i] = 2;
  }
  __syncthreads();
  int total = 0;
  for (int base = 0; base < n; base += kScanThreads) {
    const int i = base + tid;
    const int state = i < n ? needs[i] : 0, need = state == 1;
    if (i < n && !need) {
      ws.fresh[i] = state == 0 ? kNone : kBadEntry;
      if (status) status[i] = state == 0 ? kOk : kBad;
    }
    int sum;
    const int excl = block_exclusive_sum<kScanThreads>(need, scratch, &sum);
    if (need) who[total + excl] = i;
    total += sum;
  }
  __syncthreads();
  const int found = scan_free(c.refs, c.num_pages, total, scratch, [&](int rank, int32_t page) {
    const int i = who[rank];
    ws.fresh[i] = page;
    c.refs[page] = 1;
    if (status) status[i] = kOk;
  });
  for (int r = found + tid; r < total; r += kScanThreads) {
    ws.fresh[who[r]] = kUnserved;
    if (status) status[who[r]] = kNoSpace;
  }
}

// Bound by memory: 96 sequences, 94 MB of filled rows in 64 pools: 40 to 48 us,
// 4.0 to 4.8 TB/s read and written.
// Blocks (0, i, 0) rewrite the row of dst[i]; blocks (piece, i, 1 + pool) copy a
// piece of the filled rows of the last page: piece p is piece p % per_chunk of
// chunk p / per_chunk.
__global__ void __launch_bounds__(256) fork_move_kernel(PageView c, const int32_t* __restrict__ dst, ForkSpace ws,
                                                        int per_chunk) {
  const int i = blockIdx.y;
  const int32_t fresh = ws.fresh[i];
  if (fresh == kBadEntry) return;
  const int32_t len = ws.len[i];
  const int full = len / c.page_size, rest = len % c.page_size;
  const int32_t* saved = ws.rows + (int64_t)i * c.max_pages;
  if (blockIdx.z == 0) {
    if (blockIdx.x > 0) return;
    int32_t* row = c.table + (int64_t)dst[i] * c.ld_table;
    if (fresh == kUnserved) {  // dst keeps its state: it is no owner of src's pages
      for (int w = threadIdx.x; w < full; w += 256)
        if (in_range(saved[w], c.num_pages)) atomicSub(&c.refs[saved[w]], 1);
      return;
    }
    for (int w = threadIdx.x; w < c.max_pages; w += 256) {
      const int32_t old = row[w];
      if (in_range(old, c.num_pages)) atomicSub(&c.refs[old], 1);
      row[w] = w < full ? saved[w] : w == full && fresh >= 0 ? fresh : -1;
    }
    if (threadIdx.x == 0) c.seq_len[dst[i]] = len;
    return;
  }
  if (fresh < 0) return;
  const int64_t in_chunk = (int64_t)(blockIdx.x % per_chunk) * kPiece + threadIdx.x * 16;
  if (in_chunk >= rest * c.row_bytes) return;
  const int32_t last = saved[full];
  if (!in_range(last, c.num_pages)) return;
  uint8_t* pool = c.pool + (int64_t)(blockIdx.z - 1) * c.pool_stride +
                  blockIdx.x / per_chunk * (c.page_size * c.row_bytes) + in_chunk;
  store_row(pool + fresh * c.page_stride, load_row(pool + last * c.page_stride));
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(256) free_kernel(PageView c, const int32_t* __restrict__ seqs) {
  const int i = blockIdx.x;
  const int32_t s = seqs[i];
  if (repeated(seqs, i) || !in_range(s, c.max_seqs)) return;
  int32_t* row = c.table + (int64_t)s * c.ld_table;
  for (int w = threadIdx.x; w < c.max_pages; w += 256) {
    const int32_t p = row[w];
    if (in_range(p, c.num_pages)) atomicSub(&c.refs[p], 1);
    row[w] = -1;
  }
  if (threadIdx.x == 0) c.seq_len[s] = 0;
}

// ---------------------------------------------------------------- append
// 192 tokens, 48 sequences, 3 MB read and written: 3.9 us, three dependent
// look-ups (sequence, length, page) before the copy.
__global__ void __launch_bounds__(256) append_kernel(PageView c, AppendArgs a) {
  const int t = blockIdx.x;
  // The sequence of token t: the last i with start[i] <= t.
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int32_t s = a.seqs[lo];
  if (!in_range(s, c.max_seqs)) return;
  const int64_t pos = (int64_t)c.seq_len[s] + t - a.start[lo];
  if (pos < 0 || t < a.start[lo] || t >= a.start[lo + 1]) return;
  const int64_t w = pos / c.page_size;
  if (w >= c.max_pages) return;
  const int32_t page = c.table[(int64_t)s * c.ld_table + w];
  if (!in_range(page, c.num_pages)) return;
  const int pieces = a.dim / 8;
  const int64_t slot = pos % c.page_size;
  const int64_t chunk_bytes = c.page_size * c.row_bytes;
  const int64_t at = page * c.page_stride + slot * c.row_bytes;
  for (int e = threadIdx.x; e < a.heads * pieces; e += 256) {
    const int h = e / pieces, d = e % pieces * 8;
    const int64_t in_page = c.chunks == 1 ? ((int64_t)h * a.dim + d) * 2 : h * chunk_bytes + d * 2;
    *reinterpret_cast<u32x4*>(c.pool + a.k_pool * c.pool_stride + at + in_page) =
        *reinterpret_cast<const u32x4*>(a.k + t * a.k_token + h * a.k_head + d);
    *reinterpret_cast<u32x4*>(c.pool + a.v_pool * c.pool_stride + at + in_page) =
        *reinterpret_cast<const u32x4*>(a.v + t * a.v_token + h * a.v_head + d);
  }
}

// ---------------------------------------------------------------- accept
// Block (i, pool).  A lane owns 16 bytes of a row and moves them for j = 0, 1,
// ... in order: row j is written after row path[j] >= j was read, and every
// later read is of a row above j, so no row is overwritten before it is read.
// 48 paths of 3 to 7 rows in 64 pools, 62 MB read and written: 12 us where the
// caches hold the rows, 20 where they do not (ten sets in turn), 3.1 TB/s.
constexpr int kAcceptUnroll = 4;

__global__ void __launch_bounds__(256) accept_kernel(PageView c, const int32_t* __restrict__ seqs,
                                                     const int32_t* __restrict__ drafted,
                                                     const int32_t* __restrict__ path, int64_t ld_path, int columns,
                                                     const int32_t* __restrict__ accepted,
                                                     int32_t* __restrict__ new_len) {
  __shared__ int64_t from[kMaxPath], to[kMaxPath];  // byte offsets in a pool of the rows that move, in order
  __shared__ int ends;
  const int i = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
  const int32_t s = seqs[i];
  if (!in_range(s, c.max_seqs)) {
    if (blockIdx.y == 0 && tid == 0) new_len[i] = 0;
    return;
  }
  const int32_t len = c.seq_len[s], bound = drafted[i];
  const int most = min(max(accepted[i], 0), columns);
  if (tid == 0) ends = most;
  __syncthreads();
  const int32_t* mine = path + (int64_t)i * ld_path;
  for (int j = tid; j < most; j += threads) {
    const int32_t p = mine[j], before = j ? mine[j - 1] : -1;
    if (p <= before || p >= bound) atomicMin(&ends, j);
  }
  __syncthreads();
  // The rows that move, by the first wave, up to the first row or place without a
  // page; the table is read for 64 of them at once (entries beyond the row look
  // at its first entry).
  if (tid < kWave) {
    int kept = ends, moves = 0;
    for (int j0 = 0; j0 < kept; j0 += kWave) {
      const int j = j0 + tid;
      const int32_t p = mine[min(j, kept - 1)];
      const int64_t fp = ((int64_t)len + p) / c.page_size, tp = ((int64_t)len + j) / c.page_size;
      const bool in = len >= 0 && fp < c.max_pages && tp < c.max_pages;
      const int32_t* row = c.table + (int64_t)s * c.ld_table;
      const int32_t a = row[in ? fp : 0], b = row[in ? tp : 0];
      const uint64_t none = __ballot(j < kept && !(in && in_range(a, c.num_pages) && in_range(b, c.num_pages)));
      if (none) kept = j0 + __ffsll((unsigned long long)none) - 1;
      const bool move = j < kept && p != j;
      const uint64_t m = __ballot(move);
      if (move) {
        const int at = moves + __popcll(m & ((1ull << tid) - 1ull));
        from[at] = a * c.page_stride + ((int64_t)len + p) % c.page_size * c.row_bytes;
        to[at] = b * c.page_stride + ((int64_t)len + j) % c.page_size * c.row_bytes;
      }
      moves += __popcll(m);
    }
    if (tid == 0) {
      if (blockIdx.y == 0) new_len[i] = len + kept;
      ends = moves;
    }
  }
  __syncthreads();
  const int moves = ends;
  uint8_t* pool = c.pool + (int64_t)blockIdx.y * c.pool_stride;
  const int64_t chunk = c.page_size * c.row_bytes;
  const int pieces = (int)(c.row_bytes / 16);
  for (int e = tid; e < pieces * c.chunks; e += threads) {
    uint8_t* at = pool + e / pieces * chunk + e % pieces * 16;
    // Through the caches, unlike the other copies: 12 us against 16 past them
    // where the caches still hold the drafted rows (a short step), 17.6 against
    // 17.8 for six sets in turn, 20 against 18 for ten (a step that moves more than
    // the last-level cache holds).  The last round repeats the last row.
    for (int j0 = 0; j0 < moves; j0 += kAcceptUnroll) {
      u32x4 v[kAcceptUnroll];
#pragma unroll
      for (int u = 0; u < kAcceptUnroll; ++u) v[u] = *reinterpret_cast<const u32x4*>(at + from[min(j0 + u, moves - 1)]);
#pragma unroll
      for (int u = 0; u < kAcceptUnroll; ++u) *reinterpret_cast<u32x4*>(at + to[min(j0 + u, moves - 1)]) = v[u];
    }
  }
}

// ---------------------------------------------------------------- compact
// Workspace: the pages that move and where to, their number, and the new id of
// every page.
struct CompactSpace {
  int32_t* from;   // [num_pages]
  int32_t* to;     // [num_pages]
  int32_t* now;    // [num_pages]
  int32_t* moves;  // [1]
};

__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(PageView c, CompactSpace ws,
                                                                    int32_t* __restrict__ live_out) {
  __shared__ int scratch[kScanThreads / kWave + 1];
  const int tid = threadIdx.x;
  int live = 0;
  for (int64_t base = 0; base < c.num_pages; base += kScanThreads) {
    const int64_t p = base + tid;
    int sum;
    block_exclusive_sum<kScanThreads>(p < c.num_pages && c.refs[p] != 0, scratch, &sum);
    live += sum;
  }
  // Free pages below `live` and live pages at or above it are equally many.
  int holes = 0, moving = 0;
  for (int64_t base = 0; base < c.num_pages; base += kScanThreads) {
    const int64_t p = base + tid;
    const bool in = p < c.num_pages;
    const bool used = in && c.refs[p] != 0;
    const bool hole = in && p < live && !used, moves = used && p >= live;
    int sum;
    int rank = block_exclusive_sum<kScanThreads>(hole, scratch, &sum);
    if (hole) ws.to[holes + rank] = (int32_t)p;
    holes += sum;
    rank = block_exclusive_sum<kScanThreads>(moves, scratch, &sum);
    if (moves) ws.from[moving + rank] = (int32_t)p;
    moving += sum;
    if (in) ws.now[p] = (int32_t)p;
  }
  __syncthreads();
  for (int i = tid; i < moving; i += kScanThreads) {
    const int32_t a = ws.from[i], b = ws.to[i];
    ws.now[a] = b;
    c.refs[b] = c.refs[a];
    c.refs[a] = 0;
  }
  if (tid == 0) {
    *ws.moves = moving;
    *live_out = live;
  }
}

// Bound by memory: 1000 pages of 16 KiB in 64 pools, 2.1 GB read and written: 428
// us, 4.9 TB/s, after 7.5 us of the plan for 4000 pages.
constexpr int kCompactBlocks = 256 * 8;

// Every block takes (move, pool, piece) items in turn: the number of moves is
// known on the device only.
__global__ void __launch_bounds__(256) compact_copy_kernel(PageView c, CompactSpace ws, int64_t page_bytes, int pieces) {
  const int64_t items = (int64_t)*ws.moves * c.num_pools * pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t at = it % pieces * kPiece + threadIdx.x * 16, i = it / pieces / c.num_pools;
    if (at >= page_bytes) continue;
    uint8_t* pool = c.pool + it / pieces % c.num_pools * c.pool_stride + at;
    store_row(pool + ws.to[i] * c.page_stride, load_row(pool + ws.from[i] * c.page_stride));
  }
}

__global__ void __launch_bounds__(256) compact_table_kernel(PageView c, CompactSpace ws) {
  int32_t* row = c.table + (int64_t)blockIdx.x * c.ld_table;
  for (int w = threadIdx.x; w < c.max_pages; w += 256) {
    const int32_t p = row[w];
    if (in_range(p, c.num_pages)) row[w] = ws.now[p];
  }
}

int64_t page_bytes_of(const PageView& c) { return (int64_t)c.chunks * c.page_size * c.row_bytes; }
int pieces_of(int64_t bytes) { return (int)((bytes + kPiece - 1) / kPiece); }

ForkSpace fork_space(void* ws, int32_t n, int32_t max_pages) {
  ForkSpace f;
  f.len = static_cast<int32_t*>(ws);
  f.fresh = f.len + n;
  f.rows = f.fresh + n;
  return f;
}

}  // namespace

size_t fork_workspace(int32_t n, int32_t max_pages) { return ((size_t)n * (size_t)max_pages + 2 * (size_t)n) * 4; }
size_t compact_workspace(int32_t num_pages) { return 3 * (size_t)num_pages * 4 + 16; }

hipError_t launch_pages_resize(const PageView& c, const int32_t* seqs, const int32_t* lens, const int32_t* extra,
                               int32_t n, int32_t* status, hipStream_t s) {
  resize_kernel<<<1, kScanThreads, 0, s>>>(c, seqs, lens, extra, n, status);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !lens) return e;  // a sequence that keeps its length is cut in no page
  resize_copy_kernel<<<dim3(n, c.num_pools < kCutBlocks ? c.num_pools : kCutBlocks), 256, 0, s>>>(c, seqs);
  return hipGetLastError();
}

hipError_t launch_pages_copy(const PageView& c, const int32_t* src, const int32_t* dst, int32_t n, hipStream_t s) {
  const int64_t bytes = page_bytes_of(c);
  copy_kernel<<<dim3(pieces_of(bytes), n, c.num_pools), 256, 0, s>>>(c, src, dst, bytes);
  return hipGetLastError();
}

hipError_t launch_pages_fork(const PageView& c, const int32_t* src, const int32_t* dst, int32_t n, int32_t* status,
                             void* workspace, hipStream_t s) {
  const ForkSpace ws = fork_space(workspace, n, c.max_pages);
  fork_plan_kernel<<<1 + n, kScanThreads, 0, s>>>(c, src, dst, n, ws, status);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int per_chunk = pieces_of(c.page_size * c.row_bytes);
  fork_move_kernel<<<dim3(per_chunk * c.chunks, n, 1 + c.num_pools), 256, 0, s>>>(c, dst, ws, per_chunk);
  return hipGetLastError();
}

hipError_t launch_pages_free(const PageView& c, const int32_t* seqs, int32_t n, hipStream_t s) {
  free_kernel<<<n, 256, 0, s>>>(c, seqs);
  return hipGetLastError();
}

hipError_t launch_pages_append(const PageView& c, const AppendArgs& a, int32_t T, hipStream_t s) {
  append_kernel<<<T, 256, 0, s>>>(c, a);
  return hipGetLastError();
}

hipError_t launch_pages_accept(const PageView& c, const int32_t* seqs, const int32_t* drafted, const int32_t* path,
                               int64_t ld_path, int32_t columns, const int32_t* accepted, int32_t n, int32_t* new_len,
                               hipStream_t s) {
  // A lane for each 16 bytes of a token, up to 256.
  const int64_t lanes = (c.row_bytes / 16 * c.chunks + kWave - 1) / kWave * kWave;
  accept_kernel<<<dim3(n, c.num_pools), (unsigned)(lanes < 256 ? lanes : 256), 0, s>>>(c, seqs, drafted, path, ld_path, columns, accepted, new_len);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const PageView& c, int32_t* live, void* workspace, hipStream_t s) {
  CompactSpace ws;
  ws.moves = static_cast<int32_t*>(workspace);
  ws.from = ws.moves + 4;
  ws.to = ws.from + c.num_pages;
  ws.now = ws.to + c.num_pages;
  compact_plan_kernel<<<1, kScanThreads, 0, s>>>(c, ws, live);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  compact_copy_kernel<<<kCompactBlocks, 256, 0, s>>>(c, ws, page_bytes_of(c), pieces_of(page_bytes_of(c)));
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  compact_table_kernel<<<c.max_seqs, 256, 0, s>>>(c, ws);
  return hipGetLastError();
}

}  // namespace lora
