"""The decode-step entry points (include/lora_decode.h) refuse what the host
can check before anything is launched.  CPU only: every call here returns from
argument validation or has nothing to do."""
import ctypes

import pytest
import torch

import lora_serving_build_amd as lsb
from lora_serving_build_amd import decode as D

FAKE = 0x100000  # never dereferenced


def _expect(rc, code, text):
    assert rc == code, (rc, lsb.lora_last_error())
    assert text in lsb.lora_last_error()


BAD, UNS, WS = lsb.LORA_ERR_INVALID_ARG, lsb.LORA_ERR_UNSUPPORTED, lsb.LORA_ERR_WORKSPACE


# ---------------------------------------------------------------- 4-bit products
@pytest.mark.parametrize("n,k,group,zeros,want", [
    (16, 128, 128, False, 1024 + 32),
    (16, 128, 128, True, 1024 + 32 + 16),
    (17, 129, 64, False, 4 * (1024 + 64)),      # two row tiles, two blocks, two sub-groups
    (1, 1, 32, True, 1024 + 128 + 64),
    (16, 384, 96, False, 3 * (1024 + 128)),     # 96 divides neither 128 nor 64: one scale for 32 inputs
    (16, 256, 256, False, 2 * (1024 + 32)),
])
def test_q4_packed_bytes(n, k, group, zeros, want):
    assert lsb.lora_q4_packed_bytes(n, k, group, zeros) == want


@pytest.mark.parametrize("n,k,group", [(0, 128, 32), (16, 0, 32), (16, 128, 16), (16, 128, 40), (16, 128, 0),
                                       (-1, 128, 32), (16, 128, -32)])
def test_q4_packed_bytes_out_of_range(n, k, group):
    assert lsb.lora_q4_packed_bytes(n, k, group, False) == 0


def test_q4_pack_refusals():
    lib = lsb.lib()
    w = D._CQ4Weight()

    def call(**a):
        return lib.lora_q4_pack(a.get("codes", FAKE), a.get("ldc", 64), a.get("scales", FAKE), a.get("lds", 1),
                                a.get("zeros", None), a.get("ldz", 0), a.get("n", 16), a.get("k", 128),
                                a.get("group", 128), a.get("dtype", 0), a.get("packed", FAKE),
                                a.get("bytes", 1 << 20), a.get("w", ctypes.addressof(w)), None)

    _expect(call(dtype=2), BAD, "dtype")
    _expect(call(n=0), BAD, "n 0")
    _expect(call(group=48), UNS, "group 48")
    _expect(call(codes=None), BAD, "must not be NULL")
    _expect(call(w=None), BAD, "must not be NULL")
    _expect(call(ldc=63), BAD, "ld_codes")
    _expect(call(lds=0), BAD, "ld_scales")
    _expect(call(zeros=FAKE, ldz=0), BAD, "ld_zeros")
    _expect(call(bytes=1055), WS, "1056 bytes")
    _expect(call(packed=None), WS, "needed")
    _expect(call(packed=FAKE + 8), WS, "aligned")
    _expect(call(n=1 << 30, k=1 << 30, lds=1 << 24, ldc=1 << 30), UNS, "too large")


def test_q4_matmul_refusals():
    lib = lsb.lib()

    def call(**a):
        w = D._CQ4Weight(a.get("n", 16), a.get("k", 128), a.get("group", 128), 0, a.get("dtype", 0),
                         a.get("packed", FAKE))
        return lib.lora_q4_matmul(a.get("x", FAKE), a.get("ldx", a.get("k", 128)), ctypes.addressof(w), a.get("T", 4),
                                  a.get("y", FAKE), a.get("ldy", 16), 0, a.get("ws", None), a.get("ws_bytes", 0), None)

    _expect(lib.lora_q4_matmul(FAKE, 128, None, 4, FAKE, 16, 0, None, 0, None), BAD, "w is NULL")
    _expect(call(packed=None), BAD, "lora_q4_pack")
    _expect(call(packed=FAKE + 4), BAD, "lora_q4_pack")
    _expect(call(dtype=7), BAD, "dtype")
    _expect(call(n=0), BAD, "n 0")
    _expect(call(T=-1), BAD, "T -1")
    _expect(call(ldx=127), BAD, "ldx")
    _expect(call(ldy=15), BAD, "ldy")
    _expect(call(x=None), BAD, "must not be NULL")
    _expect(call(T=65535 * 16 + 1), UNS, "too large")
    size = dict(T=64, n=28672, k=8192, ldx=8192, ldy=28672)
    need = lsb.lora_q4_matmul_workspace_bytes(64, 28672, 8192, 128)
    assert need > 0 and lsb.lora_q4_matmul_workspace_bytes(1, 16, 4096, 128) == 0
    _expect(call(ws=FAKE, ws_bytes=need - 1, **size), WS, "workspace")
    _expect(call(**size), WS, "workspace")
    _expect(call(ws=FAKE + 8, ws_bytes=need, **size), WS, "aligned")
    assert call(T=0) == lsb.LORA_OK
    for sizes in ((0, 16, 128, 32), (4, 0, 128, 32), (4, 16, 0, 32), (4, 16, 128, 40)):
        assert lsb.lora_q4_matmul_workspace_bytes(*sizes) == 0


def test_q4_binding_refusals():
    codes = torch.zeros(16, 64, dtype=torch.uint8)
    scales = torch.zeros(16, 1, dtype=torch.float16)
    with pytest.raises(TypeError):
        lsb.lora_q4_pack(codes, scales.float(), None, 128, 128)
    with pytest.raises(TypeError):
        lsb.lora_q4_pack(codes.int(), scales, None, 128, 128)
    with pytest.raises(ValueError):
        lsb.lora_q4_pack(codes, scales, None, 130, 128)
    with pytest.raises(ValueError):
        lsb.lora_q4_pack(codes, scales, torch.zeros(15, 1, dtype=torch.uint8), 128, 128)
    with pytest.raises(ValueError):
        lsb.lora_q4_pack(codes, scales, None, 128, 128)          # not on a GPU
    with pytest.raises(lsb.LoraError, match="group"):
        lsb.lora_q4_pack(codes, torch.zeros(16, 8, dtype=torch.float16), None, 128, 16)


# ---------------------------------------------------------------- tree attention
def _attention(lib, **a):
    layer = D._CKvLayer(a.get("k", FAKE), a.get("v", FAKE), a.get("page_stride", 16 * 2 * 64), a.get("token_stride", 128),
                        a.get("head_stride", 64), a.get("num_pages", 8), a.get("page_size", 16))
    batch = D._CTreeBatch(a.get("B", 2), a.get("T", 3), a.get("start", FAKE), a.get("ctx", FAKE), a.get("table", FAKE),
                          a.get("ld_table", 4), a.get("max_pages", 4), a.get("mask", FAKE), a.get("ld_mask", 1),
                          a.get("words", 1))
    return lib.lora_tree_attention(a.get("q", FAKE), a.get("qt", 256), a.get("qh", 64),
                                   ctypes.addressof(layer) if a.get("layer", True) else None, ctypes.addressof(batch),
                                   a.get("heads", 4), a.get("kv_heads", 2), a.get("dim", 64), 0.125, a.get("out", FAKE),
                                   256, a.get("oh", 64), None, a.get("ws", FAKE), a.get("ws_bytes", 1 << 30),
                                   a.get("dtype", 1), None)


def test_attention_refusals():
    lib = lsb.lib()
    call = lambda **a: _attention(lib, **a)  # noqa: E731
    _expect(call(layer=False), BAD, "cache and batch")
    _expect(call(dtype=2), BAD, "dtype")
    _expect(call(heads=3), BAD, "multiple of kv_heads")
    _expect(call(kv_heads=0), BAD, "multiple of kv_heads")
    for dim in (0, 4, 12, 264):
        _expect(call(dim=dim), UNS, "dim")
    _expect(call(B=-1), BAD, "B -1")
    _expect(call(T=-1), BAD, "T -1")
    _expect(call(page_size=0), BAD, "page_size")
    _expect(call(ld_table=3), BAD, "ld_table")
    _expect(call(max_pages=1 << 28, ld_table=1 << 28), UNS, "too many")
    _expect(call(T=1 << 20, B=1 << 20, max_pages=1 << 16, ld_table=1 << 16), UNS, "row tiles")
    _expect(call(words=2), BAD, "ld_mask")
    _expect(call(qh=60), BAD, "strides")
    _expect(call(oh=62), BAD, "strides")
    _expect(call(token_stride=68), BAD, "strides")
    _expect(call(q=FAKE + 8), BAD, "aligned")
    _expect(call(v=FAKE + 2), BAD, "aligned")
    _expect(call(out=FAKE + 4), BAD, "aligned")
    _expect(call(q=None), BAD, "must not be NULL")
    _expect(call(k=None), BAD, "must not be NULL")
    _expect(call(table=None), BAD, "must not be NULL")
    need = lsb.lora_tree_attention_workspace_bytes(2, 3, 4, 2, 64)
    assert need > 0
    _expect(call(ws_bytes=need - 1), WS, "workspace")
    _expect(call(ws=None), WS, "workspace")
    _expect(call(ws=FAKE + 8), WS, "aligned")
    assert call(T=0) == lsb.LORA_OK and call(B=0) == lsb.LORA_OK
    assert lsb.lora_tree_attention_workspace_bytes(0, 3, 4, 2, 64) == 0
    assert lsb.lora_tree_attention_workspace_bytes(2, 3, 4, 3, 64) == 0


def test_attention_binding_refusals():
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    kv = torch.zeros(8, 16, 2, 64, dtype=torch.float16)
    table, ctx, start = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)

    def call(q=q, k=kv, v=kv, table=table, ctx=ctx, start=start, out=None, mask=None, lse=None):
        return lsb.lora_tree_attention(q, k, v, table, ctx, start, torch.empty_like(q) if out is None else out, 0.1,
                                       mask=mask, lse=lse)

    with pytest.raises(TypeError):
        call(q=q.float())
    with pytest.raises(TypeError):
        call(k=kv.bfloat16())
    with pytest.raises(ValueError):
        call(out=torch.zeros(3, 4, 32, dtype=torch.float16))
    with pytest.raises(ValueError):
        call(v=kv[:4])
    with pytest.raises(ValueError):
        call(v=kv.transpose(1, 2).contiguous().transpose(1, 2))   # other strides than k's
    with pytest.raises(ValueError):
        call(table=table.long())
    with pytest.raises(ValueError):
        call(start=start[:2])
    with pytest.raises(ValueError):
        call(mask=torch.zeros(3, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        call(lse=torch.zeros(3, 3))
    with pytest.raises(ValueError):
        call()                                                     # not on a GPU


# ---------------------------------------------------------------- pages
def _cache(**a):
    row = a.get("row_bytes", 256)
    page = row * a.get("page_size", 16) * a.get("chunks", 1)
    return D._CPageCache(a.get("pool", FAKE), a.get("pool_stride", page * 8), a.get("page_stride", page), row,
                         a.get("chunks", 1), a.get("num_pools", 2), a.get("num_pages", 8), a.get("page_size", 16),
                         a.get("refs", FAKE), a.get("table", FAKE), a.get("ld_table", 4), a.get("max_seqs", 4),
                         a.get("max_pages", 4), a.get("seq_len", FAKE))


def test_page_cache_refusals():
    """Every page operation checks the cache the same way."""
    lib = lsb.lib()
    for text, code, change in (("must be at least 1", BAD, {"num_pools": 0}), ("must be at least 1", BAD, {"page_size": 0}),
                               ("must be at least 1", BAD, {"max_pages": 0}), ("row_bytes", BAD, {"row_bytes": 24}),
                               ("too large", UNS, {"row_bytes": 1 << 25}), ("too large", UNS, {"max_pages": 1 << 21, "ld_table": 1 << 21}),
                               ("strides", BAD, {"page_stride": 4095}), ("strides", BAD, {"pool_stride": 4080}),
                               ("ld_table", BAD, {"ld_table": 3}), ("must not be NULL", BAD, {"refs": None}),
                               ("must not be NULL", BAD, {"pool": None}), ("aligned", BAD, {"pool": FAKE + 8})):
        c = _cache(**change)
        r = ctypes.addressof(c)
        for rc in (lib.lora_pages_resize(r, FAKE, None, None, 1, None, None),
                   lib.lora_pages_append(r, 0, 1, FAKE, 128, 64, FAKE, 128, 64, 2, 64, FAKE, FAKE, 1, 1, None),
                   lib.lora_pages_copy(r, FAKE, FAKE, 1, None),
                   lib.lora_pages_fork(r, FAKE, FAKE, 1, None, FAKE, 1 << 20, None),
                   lib.lora_pages_accept(r, FAKE, FAKE, FAKE, 1, 1, FAKE, 1, FAKE, None),
                   lib.lora_pages_free(r, FAKE, 1, None),
                   lib.lora_pages_compact(r, FAKE, FAKE, 1 << 20, None)):
            _expect(rc, code, text)
    _expect(lib.lora_pages_free(None, FAKE, 1, None), BAD, "cache is NULL")


def test_page_call_refusals():
    lib = lsb.lib()
    c = _cache()
    r = ctypes.addressof(c)
    many = lsb.LORA_MAX_PAGE_ENTRIES + 1
    for n, code, text in ((-1, BAD, "n -1"), (many, UNS, "above")):
        _expect(lib.lora_pages_resize(r, FAKE, None, None, n, None, None), code, text)
        _expect(lib.lora_pages_copy(r, FAKE, FAKE, n, None), code, text)
        _expect(lib.lora_pages_fork(r, FAKE, FAKE, n, None, FAKE, 1 << 30, None), code, text)
        _expect(lib.lora_pages_accept(r, FAKE, FAKE, FAKE, 1, 1, FAKE, n, FAKE, None), code, text)
        _expect(lib.lora_pages_free(r, FAKE, n, None), code, text)
    # Nothing to do: no launch, no pointer needed.
    assert lib.lora_pages_resize(r, None, None, None, 0, None, None) == lsb.LORA_OK
    assert lib.lora_pages_copy(r, None, None, 0, None) == lsb.LORA_OK
    assert lib.lora_pages_fork(r, None, None, 0, None, None, 0, None) == lsb.LORA_OK
    assert lib.lora_pages_accept(r, None, None, None, 0, 0, None, 0, None, None) == lsb.LORA_OK
    assert lib.lora_pages_free(r, None, 0, None) == lsb.LORA_OK
    _expect(lib.lora_pages_resize(r, None, None, None, 1, None, None), BAD, "seqs")
    _expect(lib.lora_pages_copy(r, FAKE, None, 1, None), BAD, "dst_pages")
    _expect(lib.lora_pages_fork(r, None, FAKE, 1, None, FAKE, 1 << 20, None), BAD, "src")
    need = lsb.lora_pages_fork_workspace_bytes(3, 4)
    assert need == (3 * 4 + 2 * 3) * 4 and lsb.lora_pages_fork_workspace_bytes(0, 4) == 0
    _expect(lib.lora_pages_fork(r, FAKE, FAKE, 3, None, FAKE, need - 1, None), WS, "workspace")
    _expect(lib.lora_pages_fork(r, FAKE, FAKE, 3, None, FAKE + 4, need, None), WS, "aligned")
    _expect(lib.lora_pages_accept(r, FAKE, FAKE, FAKE, 4, 5, FAKE, 1, FAKE, None), BAD, "ld_path")
    _expect(lib.lora_pages_accept(r, FAKE, FAKE, FAKE, 300, 257, FAKE, 1, FAKE, None), UNS, "columns")
    _expect(lib.lora_pages_accept(r, FAKE, FAKE, FAKE, 4, 4, None, 1, FAKE, None), BAD, "accepted")
    _expect(lib.lora_pages_compact(r, None, FAKE, 1 << 20, None), BAD, "live")
    _expect(lib.lora_pages_compact(r, FAKE, FAKE, 8, None), WS, "workspace")

    def append(**a):
        return lib.lora_pages_append(r, a.get("kp", 0), a.get("vp", 1), a.get("k", FAKE), a.get("kt", 128), 64,
                                     a.get("v", FAKE), 128, 64, a.get("heads", 2), a.get("dim", 64), FAKE,
                                     a.get("start", FAKE), a.get("n", 1), a.get("T", 1), None)

    _expect(append(T=-1), BAD, "T -1")
    _expect(append(kp=2), BAD, "pools")
    _expect(append(vp=-1), BAD, "pools")
    _expect(append(heads=3), BAD, "do not fill")
    _expect(append(dim=128), BAD, "do not fill")
    _expect(append(kt=130), BAD, "strides")
    _expect(append(k=FAKE + 2), BAD, "aligned")
    _expect(append(start=None), BAD, "must not be NULL")
    assert append(T=0) == lsb.LORA_OK and append(n=0) == lsb.LORA_OK


def test_page_cache_binding_refusals():
    pool = torch.zeros(2, 8, 16, 2, 64, dtype=torch.float16)
    refs, table, lens = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        lsb.PageCache(pool.float(), refs, table, lens)
    with pytest.raises(ValueError):
        lsb.PageCache(pool.transpose(2, 3), refs, table, lens)
    with pytest.raises(ValueError):
        lsb.PageCache(pool, refs[:7], table, lens)
    with pytest.raises(ValueError):
        lsb.PageCache(pool, refs, table.long(), lens)
    with pytest.raises(ValueError):
        lsb.PageCache(pool, refs, table, lens)                     # not on a GPU


def test_packed_structs_match_the_header():
    """The binding packs two structs in one go: their layout is that of C."""
    import struct
    assert struct.calcsize("@iiPPPqi4xPqi4x") == ctypes.sizeof(D._CTreeBatch)
    assert struct.calcsize("@PPqqqii") == ctypes.sizeof(D._CKvLayer)
    b = D._CTreeBatch.from_buffer_copy(D._BATCH(1, 2, 3, 4, 5, 6, 7, 8, 9, 10))
    assert [getattr(b, f) for f, _ in b._fields_] == list(range(1, 11))
    k = D._CKvLayer.from_buffer_copy(D._LAYER(1, 2, 3, 4, 5, 6, 7))
    assert [getattr(k, f) for f, _ in k._fields_] == list(range(1, 8))
