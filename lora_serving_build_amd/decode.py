"""Python binding of the decode-step operators of liblora_mi355x
(``include/lora_decode.h``): 4-bit base products, attention of drafted tokens
over a paged cache, and the cache's page operations.

Argument marshalling only, as in the package's ``__init__``: shapes, strides,
dtype codes and the current stream of torch tensors.

Calls that need a workspace take ``workspace``, or use one that is kept for the
current stream.  Captured in a graph they take it from the graph's memory.
"""
from __future__ import annotations

import ctypes
import struct

import torch

import lora_serving_build_amd as _base

__all__ = [
    "Q4Weight", "lora_q4_packed_bytes", "lora_q4_pack", "lora_q4_matmul",
    "lora_q4_matmul_workspace_bytes",
    "lora_tree_attention", "lora_tree_attention_workspace_bytes",
    "PageCache", "lora_pages_resize", "lora_pages_append", "lora_pages_copy", "lora_pages_fork",
    "lora_pages_fork_workspace_bytes", "lora_pages_accept", "lora_pages_free", "lora_pages_compact",
    "lora_pages_compact_workspace_bytes", "PAGES_OK", "PAGES_NO_SPACE", "PAGES_BAD",
    "LORA_MAX_PAGE_ENTRIES", "LORA_MAX_PATH", "LORA_MAX_HEAD_DIM",
]

PAGES_OK, PAGES_NO_SPACE, PAGES_BAD = 0, 1, 2
LORA_MAX_PAGE_ENTRIES, LORA_MAX_PATH, LORA_MAX_HEAD_DIM = 2048, 256, 256

_DTYPE = {torch.float16: 0, torch.bfloat16: 1}


class _CQ4Weight(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("has_zeros", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("packed", ctypes.c_void_p),
    ]


class _CTreeBatch(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32),
        ("T", ctypes.c_int32),
        ("start", ctypes.c_void_p),
        ("ctx_len", ctypes.c_void_p),
        ("table", ctypes.c_void_p),
        ("ld_table", ctypes.c_int64),
        ("max_pages", ctypes.c_int32),
        ("mask", ctypes.c_void_p),
        ("ld_mask", ctypes.c_int64),
        ("mask_words", ctypes.c_int32),
    ]


class _CKvLayer(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
    ]


class _CPageCache(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p),
        ("pool_stride", ctypes.c_int64),
        ("page_stride", ctypes.c_int64),
        ("row_bytes", ctypes.c_int64),
        ("chunks", ctypes.c_int32),
        ("num_pools", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("refs", ctypes.c_void_p),
        ("table", ctypes.c_void_p),
        ("ld_table", ctypes.c_int64),
        ("max_seqs", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("seq_len", ctypes.c_void_p),
    ]


# The same two structs packed at once.
_BATCH = struct.Struct("@iiPPPqi4xPqi4x").pack
_LAYER = struct.Struct("@PPqqqii").pack


def _declare(L) -> None:
    p, i32, i64, sz, ci = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    L.lora_q4_packed_bytes.argtypes = [i32, i32, i32, ci]
    L.lora_q4_packed_bytes.restype = sz
    L.lora_q4_pack.argtypes = [p, i64, p, i64, p, i64, i32, i32, i32, ci, p, sz, p, p]
    L.lora_q4_matmul_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.lora_q4_matmul_workspace_bytes.restype = sz
    L.lora_q4_matmul.argtypes = [p, i64, p, i32, p, i64, ci, p, sz, p]
    L.lora_tree_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.lora_tree_attention_workspace_bytes.restype = sz
    L.lora_tree_attention.argtypes = [p, i64, i64, p, p, i32, i32, i32, ctypes.c_float, p, i64, i64, p, p, sz, ci, p]
    L.lora_pages_resize.argtypes = [p, p, p, p, i32, p, p]
    L.lora_pages_append.argtypes = [p, i32, i32, p, i64, i64, p, i64, i64, i32, i32, p, p, i32, i32, p]
    L.lora_pages_copy.argtypes = [p, p, p, i32, p]
    L.lora_pages_fork_workspace_bytes.argtypes = [i32, i32]
    L.lora_pages_fork_workspace_bytes.restype = sz
    L.lora_pages_fork.argtypes = [p, p, p, i32, p, p, sz, p]
    L.lora_pages_accept.argtypes = [p, p, p, p, i64, i32, p, i32, p, p]
    L.lora_pages_free.argtypes = [p, p, i32, p]
    L.lora_pages_compact_workspace_bytes.argtypes = [i32]
    L.lora_pages_compact_workspace_bytes.restype = sz
    L.lora_pages_compact.argtypes = [p, p, p, sz, p]
    for f in ("lora_q4_pack", "lora_q4_matmul", "lora_tree_attention", "lora_pages_resize", "lora_pages_append",
              "lora_pages_copy", "lora_pages_fork", "lora_pages_accept", "lora_pages_free", "lora_pages_compact"):
        getattr(L, f).restype = ci


def _run(rc: int) -> None:
    if rc:
        raise _base.LoraError(rc, _base.lora_last_error())


# The calls below are made many times in a decoding step, some of them shorter
# on the GPU than here on the host: checks take the cheapest accessors
# (get_device, identity of dtypes), structs are packed in one go.
_raw_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing
_I32, _U8, _F32, _I64 = torch.int32, torch.uint8, torch.float32, torch.int64


def _code(t: torch.Tensor, name: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}: {name} must be float16 or bfloat16")
    return code


def _rows(t: torch.Tensor, name: str) -> int:
    """Row stride of a 2-D device tensor with contiguous rows."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _ld(rows: int, stride: int, width: int) -> int:
    """Row stride as the library takes it: that of a lone row means nothing.
    Rows that overlap keep theirs, which the library refuses."""
    return stride if rows > 1 else max(stride, width)


def _gpu(*tensors) -> int:
    """Index of the GPU that holds all of the tensors (None: not given)."""
    at = tensors[0].get_device()
    if at >= 0:
        for t in tensors:
            if t is not None and t.get_device() != at:
                break
        else:
            return at
    raise ValueError("every tensor must be on the same GPU")


def _int32(t: torch.Tensor, name: str, n: int) -> int:
    """Address of a contiguous int32 vector of (at least) n entries."""
    if t.dtype is not _I32 or t.dim() != 1 or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be a contiguous int32 vector of {n} entries")
    return t.data_ptr()


def _count(t: torch.Tensor, name: str) -> int:
    """Entries of a vector that sets how many a call has."""
    if t.dim() != 1:
        raise ValueError(f"{name} must be a vector")
    return t.numel()


def _workspace(at: int, stream: int, nbytes: int, given: torch.Tensor | None):
    """A call's workspace, its address and size: the one given, or the stream's
    (in a captured call: one of its own, from the graph's memory)."""
    if given is None:
        if nbytes == 0:
            return None, None, 0
        if not _capturing():
            given = _base._ws_cache.get((at, stream))
        if given is None or given.numel() < nbytes:
            given = _base._workspace(torch.device("cuda", at), nbytes)
    return given, given.data_ptr(), given.numel() * given.element_size()


# ---------------------------------------------------------------- 4-bit products
class Q4Weight:
    """A weight in the kernel's layout: the packed device buffer and the C
    struct that points at it."""

    def __init__(self, packed: torch.Tensor, n: int, k: int, group: int, has_zeros: bool, dtype: torch.dtype):
        self.packed, self.n, self.k, self.group, self.has_zeros, self.dtype = packed, n, k, group, has_zeros, dtype
        self.c = _CQ4Weight(n, k, group, int(has_zeros), _DTYPE[dtype], packed.data_ptr())
        self._ref = ctypes.addressof(self.c)


def lora_q4_packed_bytes(n: int, k: int, group: int, has_zeros: bool) -> int:
    return int(_base.lib().lora_q4_packed_bytes(int(n), int(k), int(group), int(bool(has_zeros))))


def lora_q4_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None, k: int,
                 group: int) -> Q4Weight:
    """Lays a weight out for lora_q4_matmul.  codes: uint8 [n][ceil(k / 2)],
    input 2 i in the low half of byte i; scales: float16 or bfloat16
    [n][ceil(k / group)]; zeros: uint8 of the scales' shape, or None (8)."""
    code = _code(scales, "scales")
    if codes.dtype != torch.uint8 or (zeros is not None and zeros.dtype != torch.uint8):
        raise TypeError("codes and zeros must be uint8")
    ldc, lds = _rows(codes, "codes"), _rows(scales, "scales")
    ldz = _rows(zeros, "zeros") if zeros is not None else 0
    n, k, group = codes.shape[0], int(k), int(group)
    groups = -(-k // group) if group > 0 else 0
    if codes.shape[1] < (k + 1) // 2 or scales.shape[0] != n or scales.shape[1] < groups:
        raise ValueError("codes must be [n][ceil(k / 2)] and scales [n][ceil(k / group)]")
    if zeros is not None and (zeros.shape[0] != n or zeros.shape[1] < groups):
        raise ValueError("zeros must have the scales' shape")
    need = lora_q4_packed_bytes(n, k, group, zeros is not None)
    packed = torch.empty(max(need, 16), dtype=torch.uint8, device=codes.device)
    w = Q4Weight(packed, n, k, group, zeros is not None, scales.dtype)
    # A shape without a packed form is refused below, before any launch.
    stream = _raw_stream(_gpu(codes, scales, zeros)) if need else 0
    _run(_base.lib().lora_q4_pack(codes.data_ptr(), ldc, scales.data_ptr(), lds,
                                  zeros.data_ptr() if zeros is not None else None, ldz, n, k, group, code,
                                  packed.data_ptr(), packed.numel(), w._ref, stream))
    return w


def lora_q4_matmul_workspace_bytes(T: int, n: int, k: int, group: int) -> int:
    return int(_base.lib().lora_q4_matmul_workspace_bytes(int(T), int(n), int(k), int(group)))


def lora_q4_matmul(x: torch.Tensor, w: Q4Weight, y: torch.Tensor, add_inputs: bool = False,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[t, :n] (+)= x[t, :k] . W for every row t of x (decode and
    verification batches); y is [T][n] in the weight's dtype, and is returned."""
    if x.dtype is not w.dtype or y.dtype is not w.dtype:
        raise TypeError("x and y must have the weight's dtype")
    if x.dim() != 2 or y.dim() != 2:
        raise ValueError("x and y must be 2-D tensors with contiguous rows")
    (T, k), (rows, n), (ldx, x_in), (ldy, y_in) = x.shape, y.shape, x.stride(), y.stride()
    if (x_in != 1 and k > 1) or (y_in != 1 and n > 1):
        raise ValueError("x and y must be 2-D tensors with contiguous rows")
    if k != w.k or n != w.n or rows < T:
        raise ValueError(f"x must be [T][{w.k}] and y [T][{w.n}]")
    if T <= 1:  # the stride of a lone row means nothing
        ldx, ldy = max(ldx, k), max(ldy, n)
    at = _gpu(w.packed, x, y, workspace)
    stream = _raw_stream(at)
    L = _base.lib()
    held, ws, ws_bytes = _workspace(at, stream, L.lora_q4_matmul_workspace_bytes(T, n, k, w.group), workspace)
    _run(L.lora_q4_matmul(x.data_ptr(), ldx, w._ref, T, y.data_ptr(), ldy, 1 if add_inputs else 0, ws, ws_bytes, stream))
    return y


# ---------------------------------------------------------------- tree attention
def lora_tree_attention_workspace_bytes(B: int, T: int, heads: int, kv_heads: int, dim: int) -> int:
    return int(_base.lib().lora_tree_attention_workspace_bytes(B, T, heads, kv_heads, dim))


def lora_tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                        ctx_len: torch.Tensor, start: torch.Tensor, out: torch.Tensor, scale: float,
                        mask: torch.Tensor | None = None, lse: torch.Tensor | None = None, head_major: bool = False,
                        workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of each sequence's drafted tokens over its cached positions.

    q, out [T][heads][dim]; k_cache, v_cache [num_pages][page_size][kv_heads][dim]
    (head_major: [num_pages][kv_heads][page_size][dim]) with the drafted tokens'
    keys and values already in place; table int32 [B][max_pages]; ctx_len int32
    [B]; start int32 [B + 1]; mask int64 [T][words], bit j of a row: the row sees
    node j of its sequence (None: node i sees nodes 0..i); lse float32
    [T][heads].  Returns out."""
    code = _code(q, "q")
    dt = q.dtype
    if k_cache.dtype is not dt or v_cache.dtype is not dt or out.dtype is not dt:
        raise TypeError("q, k_cache, v_cache and out must share a dtype")
    shape, cache_shape, strides = q.shape, k_cache.shape, k_cache.stride()
    if len(shape) != 3 or len(cache_shape) != 4 or out.shape != shape or v_cache.shape != cache_shape:
        raise ValueError("q and out must be [T][heads][dim], k_cache and v_cache four-dimensional and alike")
    T, heads, dim = shape
    num_pages, page_size, kv_heads, kdim = cache_shape
    page_st, token_st, head_st, one = strides
    if head_major:
        page_size, kv_heads, token_st, head_st = kv_heads, page_size, head_st, token_st
    (q_token, q_head, q_one), (o_token, o_head, o_one) = q.stride(), out.stride()
    if kdim != dim or one != 1 or v_cache.stride() != strides or q_one != 1 or o_one != 1:
        raise ValueError("head dims must agree and be contiguous, k_cache and v_cache must have the same strides")
    if table.dtype is not _I32 or table.dim() != 2:
        raise ValueError("table must be an int32 [B][max_pages] tensor with contiguous rows")
    (B, max_pages), (ld_table, table_in) = table.shape, table.stride()
    if table_in != 1 and max_pages > 1:
        raise ValueError("table must be an int32 [B][max_pages] tensor with contiguous rows")
    if lse is not None and (lse.dtype is not _F32 or lse.shape != (T, heads) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [T][heads] tensor")
    words, ld_mask, mask_ptr = 0, 0, 0
    if mask is not None:
        if mask.dtype is not _I64 or mask.dim() != 2:
            raise ValueError("mask must be an int64 [T][words] tensor with contiguous rows")
        (mask_rows, words), (ld_mask, mask_in) = mask.shape, mask.stride()
        if mask_rows < T or (mask_in != 1 and words > 1):
            raise ValueError("mask must be an int64 [T][words] tensor with contiguous rows")
        mask_ptr, ld_mask = mask.data_ptr(), _ld(mask_rows, ld_mask, words)
    at = _gpu(q, k_cache, v_cache, table, ctx_len, start, out, mask, lse, workspace)
    batch = _BATCH(B, T, _int32(start, "start", B + 1), _int32(ctx_len, "ctx_len", B), table.data_ptr(),
                   _ld(B, ld_table, max_pages), max_pages, mask_ptr, ld_mask, words)
    layer = _LAYER(k_cache.data_ptr(), v_cache.data_ptr(), page_st, token_st, head_st, num_pages, page_size)
    stream = _raw_stream(at)
    L = _base.lib()
    held, ws, ws_bytes = _workspace(at, stream, L.lora_tree_attention_workspace_bytes(B, T, heads, kv_heads, dim), workspace)
    _run(L.lora_tree_attention(q.data_ptr(), q_token, q_head, layer, batch, heads, kv_heads, dim, scale,
                               out.data_ptr(), o_token, o_head, lse.data_ptr() if lse is not None else None, ws,
                               ws_bytes, code, stream))
    return out


# ---------------------------------------------------------------- pages
class PageCache:
    """A paged cache: its device buffers and the C struct that points at them.

    pool     [num_pools][num_pages][page_size][heads][dim] of a 16-bit type
             (head_major: [num_pools][num_pages][heads][page_size][dim]), pages
             contiguous; one pool for each layer's keys and one for its values
    refs     int32 [num_pages] reference counts, 0 = free
    table    int32 [max_seqs][max_pages] page ids, -1 behind a row's last page
    seq_len  int32 [max_seqs] cached tokens

    A new cache has zeros in refs and seq_len and -1 throughout table."""

    def __init__(self, pool: torch.Tensor, refs: torch.Tensor, table: torch.Tensor, seq_len: torch.Tensor,
                 head_major: bool = False):
        if pool.dim() != 5 or pool.element_size() != 2 or not pool[0, 0].is_contiguous():
            raise ValueError("pool must be a five-dimensional tensor of a 16-bit type with contiguous pages")
        if table.dtype != torch.int32 or table.dim() != 2 or (table.stride(1) != 1 and table.shape[1] > 1):
            raise ValueError("table must be an int32 [max_seqs][max_pages] tensor with contiguous rows")
        pools, pages, a, b, dim = pool.shape
        self.page_size, self.heads, self.dim, self.head_major = (b, a, dim, True) if head_major else (a, b, dim, False)
        max_seqs, max_pages = table.shape
        refs_ptr, len_ptr = _int32(refs, "refs", pages), _int32(seq_len, "seq_len", max_seqs)
        _gpu(pool, refs, table, seq_len)
        self.pool, self.refs, self.table, self.seq_len = pool, refs, table, seq_len
        self.num_pages, self.max_pages = pages, max_pages
        self.c = _CPageCache(pool.data_ptr(), pool.stride(0) * 2, pool.stride(1) * 2,
                             dim * 2 if head_major else b * dim * 2, a if head_major else 1, pools, pages,
                             self.page_size, refs_ptr, table.data_ptr(), _ld(max_seqs, table.stride(0), max_pages), max_seqs,
                             max_pages, len_ptr)
        self._ref = ctypes.addressof(self.c)

    def layer(self, i: int):
        """Keys and values of layer i (pools 2 i and 2 i + 1), as
        lora_tree_attention takes them."""
        return self.pool[2 * i], self.pool[2 * i + 1]


def lora_pages_resize(cache: PageCache, seqs: torch.Tensor, lens: torch.Tensor | None = None,
                      extra: torch.Tensor | None = None, status: torch.Tensor | None = None) -> None:
    """Sets the sequences' lengths (lens; None: as they are) and makes their
    rows hold exactly the pages of length + extra tokens.  A sequence that lens
    cuts inside a page which others hold too gets its own copy of it.  status
    (optional): PAGES_OK, PAGES_NO_SPACE or PAGES_BAD for each."""
    n = _count(seqs, "seqs")
    at = _gpu(cache.pool, seqs, lens, extra, status)
    _run(_base.lib().lora_pages_resize(cache._ref, _int32(seqs, "seqs", n),
                                       _int32(lens, "lens", n) if lens is not None else None,
                                       _int32(extra, "extra", n) if extra is not None else None, n,
                                       _int32(status, "status", n) if status is not None else None, _raw_stream(at)))


def lora_pages_append(cache: PageCache, layer: int, k: torch.Tensor, v: torch.Tensor, seqs: torch.Tensor,
                      start: torch.Tensor) -> None:
    """Stores new tokens' keys and values ([T][heads][dim] each) of one layer
    behind the sequences' cached tokens: rows start[i] .. start[i + 1] - 1 go to
    positions seq_len[seqs[i]] and on."""
    dt = cache.pool.dtype
    if k.dtype is not dt or v.dtype is not dt:
        raise TypeError("k and v must have the cache's dtype")
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or shape[1] != cache.heads or shape[2] != cache.dim:
        raise ValueError("k and v must be [T][heads][dim], as in the cache")
    (k_token, k_head, k_one), (v_token, v_head, v_one) = k.stride(), v.stride()
    if k_one != 1 or v_one != 1:
        raise ValueError("k and v must have contiguous head dims")
    n = _count(seqs, "seqs")
    at = _gpu(cache.pool, k, v, seqs, start)
    _run(_base.lib().lora_pages_append(cache._ref, 2 * layer, 2 * layer + 1, k.data_ptr(), k_token, k_head,
                                       v.data_ptr(), v_token, v_head, cache.heads, cache.dim, _int32(seqs, "seqs", n),
                                       _int32(start, "start", n + 1), n, shape[0], _raw_stream(at)))


def lora_pages_copy(cache: PageCache, src_pages: torch.Tensor, dst_pages: torch.Tensor) -> None:
    """Copies page src_pages[i] to page dst_pages[i] in every pool."""
    n = _count(src_pages, "src_pages")
    at = _gpu(cache.pool, src_pages, dst_pages)
    _run(_base.lib().lora_pages_copy(cache._ref, _int32(src_pages, "src_pages", n), _int32(dst_pages, "dst_pages", n),
                                     n, _raw_stream(at)))


def lora_pages_fork_workspace_bytes(n: int, max_pages: int) -> int:
    return int(_base.lib().lora_pages_fork_workspace_bytes(n, max_pages))


def lora_pages_fork(cache: PageCache, src: torch.Tensor, dst: torch.Tensor, status: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> None:
    """Gives every sequence dst[i] the state that src[i] had before the call:
    full pages are shared, the last, partly filled one is copied, and what
    dst[i] held is released."""
    n = _count(src, "src")
    at = _gpu(cache.pool, src, dst, status, workspace)
    stream = _raw_stream(at)
    L = _base.lib()
    held, ws, ws_bytes = _workspace(at, stream, L.lora_pages_fork_workspace_bytes(n, cache.max_pages), workspace)
    _run(L.lora_pages_fork(cache._ref, _int32(src, "src", n), _int32(dst, "dst", n), n,
                           _int32(status, "status", n) if status is not None else None, ws, ws_bytes, stream))


def lora_pages_accept(cache: PageCache, seqs: torch.Tensor, drafted: torch.Tensor, path: torch.Tensor,
                      accepted: torch.Tensor, new_len: torch.Tensor) -> torch.Tensor:
    """Moves the accepted nodes' rows (path int32 [n][columns], accepted[i] of
    them) to the front of each sequence's drafted rows, in every pool, up to the
    first that has no page.  new_len receives seq_len + the rows kept; a resize
    with it makes that the length."""
    n = _count(seqs, "seqs")
    if path.dtype is not _I32 or path.dim() != 2:
        raise ValueError("path must be an int32 [n][columns] tensor with contiguous rows")
    (rows, columns), (ld_path, path_in) = path.shape, path.stride()
    if rows < n or (path_in != 1 and columns > 1):
        raise ValueError("path must be an int32 [n][columns] tensor with contiguous rows")
    at = _gpu(cache.pool, seqs, drafted, path, accepted, new_len)
    _run(_base.lib().lora_pages_accept(cache._ref, _int32(seqs, "seqs", n), _int32(drafted, "drafted", n),
                                       path.data_ptr(), _ld(rows, ld_path, columns), columns,
                                       _int32(accepted, "accepted", n), n, _int32(new_len, "new_len", n),
                                       _raw_stream(at)))
    return new_len


def lora_pages_free(cache: PageCache, seqs: torch.Tensor) -> None:
    """Releases every page of the sequences."""
    n = _count(seqs, "seqs")
    at = _gpu(cache.pool, seqs)
    _run(_base.lib().lora_pages_free(cache._ref, _int32(seqs, "seqs", n), n, _raw_stream(at)))


def lora_pages_compact_workspace_bytes(num_pages: int) -> int:
    return int(_base.lib().lora_pages_compact_workspace_bytes(num_pages))


def lora_pages_compact(cache: PageCache, live: torch.Tensor, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Moves the live pages to the lowest ids, in every pool and table row;
    live[0] receives their number."""
    at = _gpu(cache.pool, live, workspace)
    stream = _raw_stream(at)
    L = _base.lib()
    held, ws, ws_bytes = _workspace(at, stream, L.lora_pages_compact_workspace_bytes(cache.num_pages), workspace)
    _run(L.lora_pages_compact(cache._ref, _int32(live, "live", 1), ws, ws_bytes, stream))
    return live
