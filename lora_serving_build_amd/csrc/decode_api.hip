// C-ABI of the decode-step operators (declared in include/lora_decode.h):
// argument validation and dispatch.  Nothing here allocates, copies between
// host and device or synchronises.
#include "decode_kernels.h"
#include "lora_decode.h"
#include "lora_kernels.h"

namespace {

using lora::fail;
using lora::hip_status;
using lora::ok;

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int check_workspace(const void* workspace, size_t given, size_t need, const char* fn) {
  if (need > 0 && (!workspace || given < need))
    return fail(LORA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? given : (size_t)0);
  if (need > 0 && !aligned(workspace, 16))
    return fail(LORA_ERR_WORKSPACE, "%s: workspace must be 16-byte aligned", fn);
  return LORA_OK;
}

// ---------------------------------------------------------------- 4-bit products
// A launch has at most 2^32 - 1 threads in x: this many workgroups of `threads`.
constexpr int64_t most_blocks(int threads) { return 0xffffffffll / threads; }

// Shape of a weight; LORA_OK if its packed form can exist.
int check_q4(int32_t n, int32_t k, int32_t group, int dtype, const char* fn) {
  if (dtype != LORA_F16 && dtype != LORA_BF16)
    return fail(LORA_ERR_INVALID_ARG, "%s: dtype %d is neither LORA_F16 nor LORA_BF16", fn, dtype);
  if (n < 1 || k < 1) return fail(LORA_ERR_INVALID_ARG, "%s: n %d and k %d must be at least 1", fn, n, k);
  if (group < 32 || group % 32 != 0)
    return fail(LORA_ERR_UNSUPPORTED, "%s: group %d is not a multiple of 32", fn, group);
  // The packing kernel has a workgroup of 256 for each (16 outputs, 128 inputs),
  // the products one of 512 for each 16 outputs at most.
  const int64_t tiles = ((int64_t)n + 15) / 16, units = tiles * (((int64_t)k + 127) / 128);
  if (units > most_blocks(256) || tiles > most_blocks(512) || k > 0x7fffffff - 128)
    return fail(LORA_ERR_UNSUPPORTED, "%s: n %d x k %d is too large", fn, n, k);
  return LORA_OK;
}

// ---------------------------------------------------------------- pages
int check_cache(const lora_page_cache* c, const char* fn, lora::PageView* v) {
  if (!c) return fail(LORA_ERR_INVALID_ARG, "%s: cache is NULL", fn);
  if (c->chunks < 1 || c->num_pools < 1 || c->num_pages < 1 || c->page_size < 1 || c->max_seqs < 1 || c->max_pages < 1)
    return fail(LORA_ERR_INVALID_ARG, "%s: chunks, num_pools, num_pages, page_size, max_seqs and max_pages must be at least 1", fn);
  if (c->row_bytes < 16 || c->row_bytes % 16 != 0)
    return fail(LORA_ERR_INVALID_ARG, "%s: row_bytes %lld is not a multiple of 16", fn, (long long)c->row_bytes);
  if (c->row_bytes > (1 << 24) || c->page_size > (1 << 16) || c->chunks > (1 << 16) || c->num_pools > 32768 ||
      c->max_pages > (1 << 20) || c->row_bytes * c->page_size * c->chunks > (1 << 30))
    return fail(LORA_ERR_UNSUPPORTED, "%s: a page of %d x %d rows of %lld bytes, %d pools or %d pages a row are too large", fn,
                c->chunks, c->page_size, (long long)c->row_bytes, c->num_pools, c->max_pages);
  const int64_t page = c->row_bytes * c->page_size * c->chunks;
  if (c->page_stride % 16 != 0 || c->pool_stride % 16 != 0 || c->page_stride < page ||
      (c->num_pools > 1 && c->pool_stride < page))
    return fail(LORA_ERR_INVALID_ARG, "%s: strides must be multiples of 16 and hold a page of %lld bytes", fn, (long long)page);
  if (c->ld_table < c->max_pages)
    return fail(LORA_ERR_INVALID_ARG, "%s: ld_table %lld < max_pages %d", fn, (long long)c->ld_table, c->max_pages);
  if (!c->pool || !c->refs || !c->table || !c->seq_len)
    return fail(LORA_ERR_INVALID_ARG, "%s: pool, refs, table and seq_len must not be NULL", fn);
  if (!aligned(c->pool, 16)) return fail(LORA_ERR_INVALID_ARG, "%s: pool must be 16-byte aligned", fn);
  *v = lora::PageView{static_cast<uint8_t*>(c->pool), c->pool_stride, c->page_stride, c->row_bytes, c->chunks,
                      c->num_pools, c->num_pages, c->page_size, c->refs, c->table, c->ld_table, c->max_seqs,
                      c->max_pages, c->seq_len};
  return LORA_OK;
}

int check_entries(int32_t n, const char* fn) {
  if (n < 0) return fail(LORA_ERR_INVALID_ARG, "%s: n %d < 0", fn, n);
  if (n > LORA_MAX_PAGE_ENTRIES)
    return fail(LORA_ERR_UNSUPPORTED, "%s: n %d above %d", fn, n, LORA_MAX_PAGE_ENTRIES);
  return LORA_OK;
}

static_assert(LORA_MAX_PAGE_ENTRIES == lora::kMaxPageEntries && LORA_MAX_PATH == lora::kMaxPath, "limits");

// ---------------------------------------------------------------- attention
int check_heads(int32_t heads, int32_t kv_heads, int32_t dim, const char* fn) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
    return fail(LORA_ERR_INVALID_ARG, "%s: heads %d is not a multiple of kv_heads %d", fn, heads, kv_heads);
  if (dim < 8 || dim > LORA_MAX_HEAD_DIM || dim % 8 != 0)
    return fail(LORA_ERR_UNSUPPORTED, "%s: dim %d is not a multiple of 8 in [8, %d]", fn, dim, LORA_MAX_HEAD_DIM);
  return LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_q4_packed_bytes(int32_t n, int32_t k, int32_t group, int has_zeros) {
  if (check_q4(n, k, group, LORA_F16, "lora_q4_packed_bytes")) return 0;
  return lora::q4_layout(n, k, group, has_zeros != 0).bytes;
}

int lora_q4_pack(const uint8_t* codes, int64_t ld_codes, const void* scales, int64_t ld_scales,
                 const uint8_t* zeros, int64_t ld_zeros, int32_t n, int32_t k, int32_t group, int dtype,
                 void* packed, size_t packed_bytes, lora_q4_weight* w, void* stream) {
  static const char* fn = "lora_q4_pack";
  if (int e = check_q4(n, k, group, dtype, fn)) return e;
  if (!codes || !scales || !w) return fail(LORA_ERR_INVALID_ARG, "%s: codes, scales and w must not be NULL", fn);
  if (ld_codes < ((int64_t)k + 1) / 2)
    return fail(LORA_ERR_INVALID_ARG, "%s: ld_codes %lld < ceil(k / 2)", fn, (long long)ld_codes);
  const int64_t groups = ((int64_t)k + group - 1) / group;
  if (ld_scales < groups)
    return fail(LORA_ERR_INVALID_ARG, "%s: ld_scales %lld < %lld groups", fn, (long long)ld_scales, (long long)groups);
  if (zeros && ld_zeros < groups)
    return fail(LORA_ERR_INVALID_ARG, "%s: ld_zeros %lld < %lld groups", fn, (long long)ld_zeros, (long long)groups);
  const size_t need = lora::q4_layout(n, k, group, zeros != nullptr).bytes;
  if (!packed || packed_bytes < need)
    return fail(LORA_ERR_WORKSPACE, "%s: packed buffer of %zu bytes needed, %zu given", fn, need,
                packed ? packed_bytes : (size_t)0);
  if (!aligned(packed, 16)) return fail(LORA_ERR_WORKSPACE, "%s: packed buffer must be 16-byte aligned", fn);
  w->n = n;
  w->k = k;
  w->group = group;
  w->has_zeros = zeros ? 1 : 0;
  w->dtype = dtype;
  w->packed = packed;
  return hip_status(lora::launch_q4_pack(codes, ld_codes, static_cast<const uint16_t*>(scales), ld_scales, zeros,
                                         ld_zeros, n, k, group, packed, static_cast<hipStream_t>(stream)),
                    fn);
}

size_t lora_q4_matmul_workspace_bytes(int32_t T, int32_t n, int32_t k, int32_t group) {
  if (T < 1 || check_q4(n, k, group, LORA_F16, "lora_q4_matmul_workspace_bytes")) return 0;
  return lora::q4_workspace(T, n, k, group);
}

int lora_q4_matmul(const void* x, int64_t ldx, const lora_q4_weight* w, int32_t T, void* y, int64_t ldy,
                   int add_inputs, void* workspace, size_t workspace_bytes, void* stream) {
  static const char* fn = "lora_q4_matmul";
  if (!w) return fail(LORA_ERR_INVALID_ARG, "%s: w is NULL", fn);
  if (int e = check_q4(w->n, w->k, w->group, w->dtype, fn)) return e;
  if (!w->packed || !aligned(w->packed, 16))
    return fail(LORA_ERR_INVALID_ARG, "%s: w was not filled by lora_q4_pack", fn);
  if (T < 0) return fail(LORA_ERR_INVALID_ARG, "%s: T %d < 0", fn, T);
  if (ldx < w->k) return fail(LORA_ERR_INVALID_ARG, "%s: ldx %lld < k %d", fn, (long long)ldx, w->k);
  if (ldy < w->n) return fail(LORA_ERR_INVALID_ARG, "%s: ldy %lld < n %d", fn, (long long)ldy, w->n);
  if (T == 0) return ok();
  if (!x || !y) return fail(LORA_ERR_INVALID_ARG, "%s: x and y must not be NULL", fn);
  if (T > 65535 * 16) return fail(LORA_ERR_UNSUPPORTED, "%s: T %d is too large", fn, T);
  if (int e = check_workspace(workspace, workspace_bytes, lora::q4_workspace(T, w->n, w->k, w->group), fn)) return e;
  const bool x_vec = aligned(x, 16) && ldx % 8 == 0 && w->k % 8 == 0;
  const bool y_vec = aligned(y, 8) && ldy % 4 == 0 && w->n % 4 == 0;
  return hip_status(lora::launch_q4_matmul(static_cast<const uint16_t*>(x), ldx, w->packed, w->n, w->k, w->group,
                                           w->has_zeros != 0, T, static_cast<uint16_t*>(y), ldy, add_inputs ? 1 : 0,
                                           w->dtype, x_vec, y_vec, workspace, static_cast<hipStream_t>(stream)),
                    fn);
}

int lora_pages_resize(const lora_page_cache* cache, const int32_t* seqs, const int32_t* lens, const int32_t* extra,
                      int32_t n, int32_t* status, void* stream) {
  static const char* fn = "lora_pages_resize";
  lora::PageView v;
  if (int e = check_cache(cache, fn, &v)) return e;
  if (int e = check_entries(n, fn)) return e;
  if (n == 0) return ok();
  if (!seqs) return fail(LORA_ERR_INVALID_ARG, "%s: seqs must not be NULL", fn);
  if ((int64_t)n * v.max_pages > 0x7fffffff)
    return fail(LORA_ERR_UNSUPPORTED, "%s: n %d x max_pages %d is too large", fn, n, v.max_pages);
  return hip_status(lora::launch_pages_resize(v, seqs, lens, extra, n, status, static_cast<hipStream_t>(stream)), fn);
}

int lora_pages_append(const lora_page_cache* cache, int32_t k_pool, int32_t v_pool, const void* k,
                      int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                      int64_t v_head_stride, int32_t heads, int32_t dim, const int32_t* seqs, const int32_t* start,
                      int32_t n, int32_t T, void* stream) {
  static const char* fn = "lora_pages_append";
  lora::PageView c;
  if (int e = check_cache(cache, fn, &c)) return e;
  if (int e = check_entries(n, fn)) return e;
  if (T < 0) return fail(LORA_ERR_INVALID_ARG, "%s: T %d < 0", fn, T);
  if (k_pool < 0 || k_pool >= c.num_pools || v_pool < 0 || v_pool >= c.num_pools)
    return fail(LORA_ERR_INVALID_ARG, "%s: pools %d and %d outside [0, %d)", fn, k_pool, v_pool, c.num_pools);
  if (heads < 1 || dim < 8 || dim % 8 != 0 || (int64_t)heads * dim * 2 != c.chunks * c.row_bytes ||
      (c.chunks != 1 && c.chunks != heads))
    return fail(LORA_ERR_INVALID_ARG, "%s: %d heads of %d do not fill a page's %d x %lld bytes a token", fn, heads, dim,
                c.chunks, (long long)c.row_bytes);
  if (k_token_stride % 8 != 0 || k_head_stride % 8 != 0 || v_token_stride % 8 != 0 || v_head_stride % 8 != 0 ||
      !aligned(k, 16) || !aligned(v, 16))
    return fail(LORA_ERR_INVALID_ARG, "%s: k and v must be 16-byte aligned with strides that are multiples of 8", fn);
  if (n == 0 || T == 0) return ok();
  if (T > most_blocks(256)) return fail(LORA_ERR_UNSUPPORTED, "%s: T %d is too large", fn, T);
  if (!k || !v || !seqs || !start) return fail(LORA_ERR_INVALID_ARG, "%s: k, v, seqs and start must not be NULL", fn);
  const lora::AppendArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_token_stride,
                           k_head_stride, v_token_stride, v_head_stride, k_pool, v_pool, heads, dim, seqs, start, n};
  return hip_status(lora::launch_pages_append(c, a, T, static_cast<hipStream_t>(stream)), fn);
}

int lora_pages_copy(const lora_page_cache* cache, const int32_t* src_pages, const int32_t* dst_pages, int32_t n,
                    void* stream) {
  static const char* fn = "lora_pages_copy";
  lora::PageView v;
  if (int e = check_cache(cache, fn, &v)) return e;
  if (int e = check_entries(n, fn)) return e;
  if (n == 0) return ok();
  if (!src_pages || !dst_pages) return fail(LORA_ERR_INVALID_ARG, "%s: src_pages and dst_pages must not be NULL", fn);
  return hip_status(lora::launch_pages_copy(v, src_pages, dst_pages, n, static_cast<hipStream_t>(stream)), fn);
}

size_t lora_pages_fork_workspace_bytes(int32_t n, int32_t max_pages) {
  return n < 1 || max_pages < 1 ? 0 : lora::fork_workspace(n, max_pages);
}

int lora_pages_fork(const lora_page_cache* cache, const int32_t* src, const int32_t* dst, int32_t n, int32_t* status,
                    void* workspace, size_t workspace_bytes, void* stream) {
  static const char* fn = "lora_pages_fork";
  lora::PageView v;
  if (int e = check_cache(cache, fn, &v)) return e;
  if (int e = check_entries(n, fn)) return e;
  if (n == 0) return ok();
  if (!src || !dst) return fail(LORA_ERR_INVALID_ARG, "%s: src and dst must not be NULL", fn);
  if (int e = check_workspace(workspace, workspace_bytes, lora::fork_workspace(n, v.max_pages), fn)) return e;
  return hip_status(lora::launch_pages_fork(v, src, dst, n, status, workspace, static_cast<hipStream_t>(stream)), fn);
}

int lora_pages_accept(const lora_page_cache* cache, const int32_t* seqs, const int32_t* drafted, const int32_t* path,
                      int64_t ld_path, int32_t columns, const int32_t* accepted, int32_t n, int32_t* new_len,
                      void* stream) {
  static const char* fn = "lora_pages_accept";
  lora::PageView v;
  if (int e = check_cache(cache, fn, &v)) return e;
  if (int e = check_entries(n, fn)) return e;
  if (columns < 0 || ld_path < columns)
    return fail(LORA_ERR_INVALID_ARG, "%s: columns %d and ld_path %lld", fn, columns, (long long)ld_path);
  if (columns > LORA_MAX_PATH) return fail(LORA_ERR_UNSUPPORTED, "%s: columns %d above %d", fn, columns, LORA_MAX_PATH);
  if (n == 0) return ok();
  if (!seqs || !drafted || !accepted || !new_len || (!path && columns > 0))
    return fail(LORA_ERR_INVALID_ARG, "%s: seqs, drafted, path, accepted and new_len must not be NULL", fn);
  return hip_status(lora::launch_pages_accept(v, seqs, drafted, path, ld_path, columns, accepted, n, new_len,
                                              static_cast<hipStream_t>(stream)),
                    fn);
}

int lora_pages_free(const lora_page_cache* cache, const int32_t* seqs, int32_t n, void* stream) {
  static const char* fn = "lora_pages_free";
  lora::PageView v;
  if (int e = check_cache(cache, fn, &v)) return e;
  if (int e = check_entries(n, fn)) return e;
  if (n == 0) return ok();
  if (!seqs) return fail(LORA_ERR_INVALID_ARG, "%s: seqs must not be NULL", fn);
  return hip_status(lora::launch_pages_free(v, seqs, n, static_cast<hipStream_t>(stream)), fn);
}

size_t lora_pages_compact_workspace_bytes(int32_t num_pages) {
  return num_pages < 1 ? 0 : lora::compact_workspace(num_pages);
}

int lora_pages_compact(const lora_page_cache* cache, int32_t* live, void* workspace, size_t workspace_bytes,
                       void* stream) {
  static const char* fn = "lora_pages_compact";
  lora::PageView v;
  if (int e = check_cache(cache, fn, &v)) return e;
  if (v.max_seqs > most_blocks(256))
    return fail(LORA_ERR_UNSUPPORTED, "%s: %d rows of the table are too many", fn, v.max_seqs);
  if (!live) return fail(LORA_ERR_INVALID_ARG, "%s: live must not be NULL", fn);
  if (int e = check_workspace(workspace, workspace_bytes, lora::compact_workspace(v.num_pages), fn)) return e;
  return hip_status(lora::launch_pages_compact(v, live, workspace, static_cast<hipStream_t>(stream)), fn);
}

size_t lora_tree_attention_workspace_bytes(int32_t B, int32_t T, int32_t heads, int32_t kv_heads, int32_t dim) {
  if (B < 1 || T < 1 || check_heads(heads, kv_heads, dim, "lora_tree_attention_workspace_bytes")) return 0;
  return lora::attention_workspace(B, T, heads, kv_heads, dim);
}

int lora_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const lora_kv_layer* cache,
                        const lora_tree_batch* batch, int32_t heads, int32_t kv_heads, int32_t dim, float scale,
                        void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse, void* workspace,
                        size_t workspace_bytes, int dtype, void* stream) {
  static const char* fn = "lora_tree_attention";
  if (!cache || !batch) return fail(LORA_ERR_INVALID_ARG, "%s: cache and batch must not be NULL", fn);
  if (dtype != LORA_F16 && dtype != LORA_BF16)
    return fail(LORA_ERR_INVALID_ARG, "%s: dtype %d is neither LORA_F16 nor LORA_BF16", fn, dtype);
  if (int e = check_heads(heads, kv_heads, dim, fn)) return e;
  const lora_tree_batch& b = *batch;
  const lora_kv_layer& c = *cache;
  if (b.B < 0 || b.T < 0) return fail(LORA_ERR_INVALID_ARG, "%s: B %d or T %d < 0", fn, b.B, b.T);
  if (c.num_pages < 0 || c.page_size < 1 || b.max_pages < 0 || b.ld_table < b.max_pages)
    return fail(LORA_ERR_INVALID_ARG, "%s: num_pages %d, page_size %d, max_pages %d, ld_table %lld", fn, c.num_pages,
                c.page_size, b.max_pages, (long long)b.ld_table);
  if ((int64_t)b.max_pages * c.page_size > 0x7fffff00)
    return fail(LORA_ERR_UNSUPPORTED, "%s: %d pages of %d positions are too many", fn, b.max_pages, c.page_size);
  if (b.mask_words < 0 || (b.mask && b.ld_mask < b.mask_words))
    return fail(LORA_ERR_INVALID_ARG, "%s: mask_words %d and ld_mask %lld", fn, b.mask_words, (long long)b.ld_mask);
  if (q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || out_token_stride % 4 != 0 || out_head_stride % 4 != 0 ||
      c.page_stride % 8 != 0 || c.token_stride % 8 != 0 || c.head_stride % 8 != 0)
    return fail(LORA_ERR_INVALID_ARG, "%s: strides must be multiples of 8 (of out: of 4) elements", fn);
  if (!aligned(q, 16) || !aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(out, 8))
    return fail(LORA_ERR_INVALID_ARG, "%s: q, k and v must be 16-byte aligned, out 8-byte", fn);
  if ((int64_t)b.T * heads > 0x3fffffff) return fail(LORA_ERR_UNSUPPORTED, "%s: T %d x heads %d is too large", fn, b.T, heads);
  // The kernels count (row tile, key head, tile of positions) units in 32 bits.
  const int64_t rows = (int64_t)b.T * (heads / kv_heads), tiles = rows / 16 + (b.B < rows ? b.B : rows);
  const int64_t units = (int64_t)b.max_pages * c.page_size / 32 + 8;
  if (tiles * kv_heads > 0x7fffffff / units)
    return fail(LORA_ERR_UNSUPPORTED, "%s: %lld row tiles of up to %lld positions are too many", fn,
                (long long)(tiles * kv_heads), (long long)b.max_pages * c.page_size);
  if (b.B == 0 || b.T == 0) return ok();
  if (!q || !out || !b.start || !b.ctx_len || (b.max_pages > 0 && !b.table) || (c.num_pages > 0 && (!c.k || !c.v)))
    return fail(LORA_ERR_INVALID_ARG, "%s: q, out, start, ctx_len, table, k and v must not be NULL", fn);
  if (lora::attention_threads(b.B, b.T, heads, kv_heads, dim, (int64_t)b.max_pages * c.page_size) > 0xffffffffll)
    return fail(LORA_ERR_UNSUPPORTED, "%s: %lld row tiles are too many", fn, (long long)(tiles * kv_heads));
  if (int e = check_workspace(workspace, workspace_bytes,
                              lora::attention_workspace(b.B, b.T, heads, kv_heads, dim), fn))
    return e;
  lora::AttnArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.k = static_cast<const uint16_t*>(c.k);
  a.v = static_cast<const uint16_t*>(c.v);
  a.kv_page = c.page_stride;
  a.kv_token = c.token_stride;
  a.kv_head = c.head_stride;
  a.num_pages = c.num_pages;
  a.page_size = c.page_size;
  a.table = b.table;
  a.ld_table = b.ld_table;
  a.max_pages = b.max_pages;
  a.ctx = b.ctx_len;
  a.start = b.start;
  a.mask = b.mask;
  a.ld_mask = b.ld_mask;
  a.mask_words = b.mask_words;
  a.out = static_cast<uint16_t*>(out);
  a.out_token = out_token_stride;
  a.out_head = out_head_stride;
  a.lse = lse;
  a.B = b.B;
  a.T = b.T;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.dim = dim;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.partial = static_cast<float*>(workspace);
  return hip_status(lora::launch_attention(a, dtype, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
