/*
 * liblora_mi355x: the operators of a decode step around the adapters, for AMD
 * Instinct MI355X (gfx950):
 *   - lora_q4_*: the base projection under an expand, with 4-bit weights;
 *   - lora_tree_attention: attention of a step's drafted tokens (a tree for
 *     each sequence; one token, or a chain, in the simple cases) over a paged
 *     key / value cache;
 *   - lora_pages_*: the cache's page operations (resize, append, copy, fork,
 *     accept, free, compact).
 *
 * The conventions are those of lora.h: pointers are DEVICE memory unless
 * marked host, the library allocates nothing, keeps no pointer past a call,
 * never synchronises and copies nothing between host and device, so every
 * call can be captured in a HIP graph.  Host-checkable errors return a
 * negative status before any launch and lora_last_error() describes them.
 * Data-dependent problems never read or write out of range; each call says
 * what becomes of them.
 */
#ifndef LORA_DECODE_H
#define LORA_DECODE_H

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ 4-bit products
 * y[t, c] = (add_inputs ? y[t, c] : 0) + sum_{h<k} x[t, h] W[c, h],
 * W[c, h] = scale[c, h / group] * (q[c, h] - zero[c, h / group]),
 * with 4-bit codes q in [0, 15].  Without zeros, zero = 8.  The products are
 * exact (16-bit x times a small whole number), sums and scales are fp32, and y
 * is rounded once.  Infinities and NaN in x give what the definition gives. */

/* A weight as lora_q4_pack lays it out.  A host struct whose pointer is a
 * caller-owned device buffer. */
typedef struct lora_q4_weight {
  int32_t n;           /* output columns                                    */
  int32_t k;           /* inputs                                            */
  int32_t group;       /* inputs that share a scale: a multiple of 32       */
  int32_t has_zeros;   /* 0: every zero is 8                                */
  int32_t dtype;       /* LORA_F16 / LORA_BF16: type of the scales, x and y */
  const void *packed;  /* device, lora_q4_packed_bytes(...) bytes           */
} lora_q4_weight;

/* Bytes of the packed form (0 for arguments out of range).  n is padded to 16
 * and k to 128. */
size_t lora_q4_packed_bytes(int32_t n, int32_t k, int32_t group, int has_zeros);

/* Lays a weight out for lora_q4_matmul (once, when it is loaded).
 *   codes   [n][ld_codes] bytes, ld_codes >= ceil(k / 2): input 2 i in the low
 *           half of byte i, input 2 i + 1 in the high half
 *   scales  [n][ld_scales] of dtype, ld_scales >= ceil(k / group)
 *   zeros   [n][ld_zeros] bytes (the low four bits count), or NULL
 *   w       host; filled by the call
 *   packed  16-byte aligned, packed_bytes >= lora_q4_packed_bytes
 * Errors: INVALID_ARG (NULL, n or k < 1, strides, dtype), UNSUPPORTED (group
 * not a multiple of 32, n above 2^27 - 16, more than 2^24 - 1 blocks of 16 outputs
 * x 128 inputs), WORKSPACE (packed_bytes too small or unaligned), HIP. */
int lora_q4_pack(const uint8_t *codes, int64_t ld_codes, const void *scales, int64_t ld_scales,
                 const uint8_t *zeros, int64_t ld_zeros, int32_t n, int32_t k, int32_t group,
                 int dtype, void *packed, size_t packed_bytes, lora_q4_weight *w, void *stream);

/* The product for T tokens.  Meant for decode and verification batches: tokens
 * are taken in passes of 16 to 128, whichever form is cheapest for the shape, and
 * every pass reads the weight.
 *   x  [T][ldx], ldx >= k;  y  [T][ldy], ldy >= n; both of the weight's dtype;
 *   x and y must not overlap
 *   workspace  lora_q4_matmul_workspace_bytes(T, n, k, group) bytes (0 for most
 *              batches of up to 16 tokens, then NULL will do), 16-byte aligned, needs no
 *              initialisation; calls that run concurrently must not share it
 * Same inputs give the same bits.
 * Errors: INVALID_ARG (NULL, T < 0, strides, a weight struct that no
 * lora_q4_pack filled), UNSUPPORTED (T above 65535 x 16), WORKSPACE, HIP. */
size_t lora_q4_matmul_workspace_bytes(int32_t T, int32_t n, int32_t k, int32_t group);
int lora_q4_matmul(const void *x, int64_t ldx, const lora_q4_weight *w, int32_t T, void *y,
                   int64_t ldy, int add_inputs, void *workspace, size_t workspace_bytes,
                   void *stream);

/* ------------------------------------------------------------------ tree attention
 * A step's tokens are grouped by sequence: sequence b owns rows [start[b],
 * start[b + 1]) of q, its nodes 0, 1, ... in order.  Their keys and values are
 * already in the cache, at positions ctx_len[b] + node, behind the ctx_len[b]
 * tokens of the context (lora_pages_append puts them there).  Node i sees every
 * position of the context and those nodes whose bit is set in its mask row (a
 * tree: itself and its ancestors):
 *   o[i, h] = sum_p w_p v[p, h / G] / sum_p w_p,
 *   w_p = exp(scale q[i, h] . k[p, h / G]),  G = heads / kv_heads,
 * over the positions p that node i sees.  A row that sees nothing is 0 and its
 * lse is -inf.  What a row does not see never reaches it, NaN and infinities
 * among it.  Scores, the softmax and the sums are fp32; o is rounded once.  The
 * matrix cores take the weights in 16 bits: as a sum of two parts, which adds
 * little to o's own rounding, for dims up to 128 and up to 64 rows (nodes times
 * G) a sequence on average; beyond that rounded once to the cache's type.  In
 * f16 a weight below 2^-23 of the row's heaviest keeps fewer bits, 2^-33 of that
 * one being the last. */
typedef struct lora_tree_batch {
  int32_t B;                 /* sequences                                           */
  int32_t T;                 /* rows of q; start[B] = T                             */
  const int32_t *start;      /* [B + 1] ascending from 0; where it does not ascend, */
                             /* what out and lse hold afterwards is undefined       */
  const int32_t *ctx_len;    /* [B] tokens of the context                           */
  const int32_t *table;      /* [B][ld_table] page ids; positions of pages outside  */
  int64_t ld_table;          /* [0, num_pages) are not seen                         */
  int32_t max_pages;         /* entries of a row; positions beyond are not seen     */
  const uint64_t *mask;      /* [T][ld_mask]: bit j % 64 of word j / 64 is node j;  */
  int64_t ld_mask;           /* NULL: node i sees nodes 0..i (a chain)              */
  int32_t mask_words;        /* words of a row; nodes beyond them are not seen      */
} lora_tree_batch;

/* One layer's cache: page p, slot s, head h at p page_stride + s token_stride +
 * h head_stride (elements, multiples of 8; the bases 16-byte aligned). */
typedef struct lora_kv_layer {
  const void *k;
  const void *v;
  int64_t page_stride, token_stride, head_stride;
  int32_t num_pages;
  int32_t page_size;
} lora_kv_layer;

#define LORA_MAX_HEAD_DIM 256

/* q, out [T] tokens with strides in elements; lse fp32 [T][heads] or NULL.
 * dim: a multiple of 8, at most LORA_MAX_HEAD_DIM.  heads: a multiple of
 * kv_heads.  workspace: lora_tree_attention_workspace_bytes, 16-byte aligned,
 * needs no initialisation.  Calls that run concurrently must not share it.
 * Same inputs give the same bits.
 * Errors: INVALID_ARG (NULL, sizes, strides, alignment, dtype), UNSUPPORTED
 * (dim; a table row of more than 2^31 - 256 positions; 2^31 or more units of 16
 * rows, a key head and 32 positions of the table; launches of 2^32 threads),
 * WORKSPACE, HIP. */
size_t lora_tree_attention_workspace_bytes(int32_t B, int32_t T, int32_t heads, int32_t kv_heads,
                                           int32_t dim);
int lora_tree_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                        const lora_kv_layer *cache, const lora_tree_batch *batch, int32_t heads,
                        int32_t kv_heads, int32_t dim, float scale, void *out,
                        int64_t out_token_stride, int64_t out_head_stride, float *lse,
                        void *workspace, size_t workspace_bytes, int dtype, void *stream);

/* ------------------------------------------------------------------ pages of a cache
 * The keys and values of every layer live in equal pools of equal pages (a
 * layer's keys are one pool, its values another); page p of a sequence holds
 * its positions [p page_size, (p + 1) page_size) in every pool.  A page is
 * free while its reference count is 0; it may belong to several sequences.
 * Only full pages are ever shared: a fork copies the last, partly filled one,
 * and a resize that cuts a sequence inside a shared page gives it its own.
 * Slots of a page behind a sequence's tokens hold no defined bytes.
 *
 * A host struct whose pointers are caller-owned device buffers.  A table row
 * holds a sequence's page ids in its leading entries and -1 after them. */
typedef struct lora_page_cache {
  void *pool;           /* [num_pools][num_pages] pages, 16-byte aligned       */
  int64_t pool_stride;  /* bytes from pool to pool, a multiple of 16           */
  int64_t page_stride;  /* bytes from page to page, a multiple of 16           */
  int64_t row_bytes;    /* a page is [chunks][page_size][row_bytes]; row_bytes */
  int32_t chunks;       /* is a multiple of 16.  Token-major pages have one    */
                        /* chunk (all heads of a token), head-major pages one  */
                        /* chunk for each head                                 */
  int32_t num_pools;
  int32_t num_pages;
  int32_t page_size;    /* tokens of a page                                    */
  int32_t *refs;        /* [num_pages] reference counts, 0 = free              */
  int32_t *table;       /* [max_seqs][ld_table] page ids                       */
  int64_t ld_table;     /* >= max_pages                                        */
  int32_t max_seqs;
  int32_t max_pages;    /* entries of a row that belong to the sequence        */
  int32_t *seq_len;     /* [max_seqs] cached tokens                            */
} lora_page_cache;

/* Entries of one call, and path columns of lora_pages_accept. */
#define LORA_MAX_PAGE_ENTRIES 2048
#define LORA_MAX_PATH 256

/* Per-entry results (int32, device). */
#define LORA_PAGES_OK 0
#define LORA_PAGES_NO_SPACE 1  /* no page left for this entry; it is unchanged      */
#define LORA_PAGES_BAD 2       /* sequence out of range or named by an earlier entry */
                               /* (as a destination), or more than max_pages needed; */
                               /* the entry is unchanged                             */

/* Common rules of the calls below: n entries, 0 <= n <= LORA_MAX_PAGE_ENTRIES
 * (n = 0 launches nothing); seqs, src, dst are int32 device arrays of n
 * sequence ids.  Free pages are given out lowest id first, in entry order, so
 * results do not depend on timing; once an entry finds no page, no later entry
 * that needs one is served.  Pages released by a call are given out by later
 * calls only.  Table entries outside [0, num_pages) are never followed.
 * Errors of each: INVALID_ARG (NULL, sizes, strides, alignment), UNSUPPORTED
 * (n or another size above its limit; T of an append or max_seqs of a compaction
 * above 2^24 - 1), WORKSPACE, HIP. */

/* Sets sequence lengths and makes every row hold exactly the pages of its
 * length plus `extra` tokens to come: allocates what is missing, releases what
 * is too much.  With lens, a page at or behind the new end that another
 * sequence holds as well (by the counts before the call) is replaced by one of
 * the sequence's own, with a copy of the rows that stay filled; an entry that
 * needs such a page and finds none is NO_SPACE like any other.  lens [n] (NULL:
 * lengths stay), extra [n] (NULL: 0), status [n] (or NULL). */
int lora_pages_resize(const lora_page_cache *cache, const int32_t *seqs, const int32_t *lens,
                      const int32_t *extra, int32_t n, int32_t *status, void *stream);

/* Stores the keys and values of new tokens: token t in [start[i], start[i + 1])
 * goes to position seq_len[seqs[i]] + t - start[i] of sequence i, in pools
 * k_pool and v_pool.  16-bit elements, heads x dim of them for each token
 * (heads dim 2 = chunks row_bytes), dim a multiple of 8; k and v 16-byte
 * aligned with strides (elements) that are multiples of 8.  start is [n + 1],
 * ascending from 0 to T.  Positions without a page are dropped. */
int lora_pages_append(const lora_page_cache *cache, int32_t k_pool, int32_t v_pool, const void *k,
                      int64_t k_token_stride, int64_t k_head_stride, const void *v,
                      int64_t v_token_stride, int64_t v_head_stride, int32_t heads, int32_t dim,
                      const int32_t *seqs, const int32_t *start, int32_t n, int32_t T, void *stream);

/* Copies page src_pages[i] to dst_pages[i] in every pool.  Entries with an id
 * outside [0, num_pages) are skipped.  A page that one entry writes must not
 * be named by another. */
int lora_pages_copy(const lora_page_cache *cache, const int32_t *src_pages, const int32_t *dst_pages,
                    int32_t n, void *stream);

/* Every dst[i] takes the state that src[i] had before the call (a beam step,
 * a shared prefix): it refers to src's full pages, owns a copy of the filled
 * rows of its last page, and what it held is released.  src may repeat and
 * may be a destination too; destinations are distinct.  status [n] or NULL.
 * workspace: lora_pages_fork_workspace_bytes(n, max_pages), 16-byte aligned,
 * needs no initialisation. */
size_t lora_pages_fork_workspace_bytes(int32_t n, int32_t max_pages);
int lora_pages_fork(const lora_page_cache *cache, const int32_t *src, const int32_t *dst, int32_t n,
                    int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/* Keeps the accepted path of drafted trees: sequence i holds drafted[i] rows
 * from position seq_len on; row path[i][j] moves to row j, j < accepted[i], in
 * every pool, and new_len[i] = seq_len + the rows kept (seq_len itself is set
 * by a resize).  path is [n][ld_path], columns <= LORA_MAX_PATH; a path ends at
 * its first entry that is not above the one before it, not below drafted[i], or
 * whose row or place has no page (a draft that found no space); what is behind
 * it is not kept.  seqs are distinct; new_len of one out of range is 0.  new_len
 * must not overlap seq_len. */
int lora_pages_accept(const lora_page_cache *cache, const int32_t *seqs, const int32_t *drafted,
                      const int32_t *path, int64_t ld_path, int32_t columns, const int32_t *accepted,
                      int32_t n, int32_t *new_len, void *stream);

/* Releases every page of the sequences: rows become -1, lengths 0.  Ids out of
 * range and repeated ids are skipped. */
int lora_pages_free(const lora_page_cache *cache, const int32_t *seqs, int32_t n, void *stream);

/* Moves the live pages to the lowest ids, in every pool and every table: the
 * i-th free page below `live` takes the i-th live page at or above it, live
 * being the number of live pages, which is also written to *live (device).
 * workspace: lora_pages_compact_workspace_bytes(num_pages), 16-byte aligned,
 * needs no initialisation. */
size_t lora_pages_compact_workspace_bytes(int32_t num_pages);
int lora_pages_compact(const lora_page_cache *cache, int32_t *live, void *workspace,
                       size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_DECODE_H */
