"""What the binding of the decode-step operators hands to the library (CPU: the
calls are stopped before, or refused by, the library's checks)."""
import pytest
import torch

import lora_serving_build_amd as lsb
from lora_serving_build_amd import decode as D


@pytest.fixture
def no_gpu(monkeypatch):
    """Tensors in host memory pass for a GPU's: only for calls that the library
    refuses before any launch, or that a stub takes."""
    monkeypatch.setattr(D, "_gpu", lambda *tensors: 0)
    monkeypatch.setattr(D, "_raw_stream", lambda at: 0)


def attention(table=None, mask=None, T=3, B=2):
    q = torch.zeros(T, 4, 64, dtype=torch.float16)
    kv = torch.zeros(8, 16, 2, 64, dtype=torch.float16)
    table = torch.zeros(B, 4, dtype=torch.int32) if table is None else table
    return lsb.lora_tree_attention(q, kv, kv, table, torch.zeros(B, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32),
                                   torch.empty_like(q), 0.1, mask=mask, workspace=torch.empty(1 << 24, dtype=torch.uint8))


def test_broadcast_rows_are_refused(no_gpu):
    """Rows that overlap (one row expanded to all) have a stride below their
    width: the library is told, and refuses, instead of reading beyond them."""
    with pytest.raises(lsb.LoraError, match="ld_table 0"):
        attention(table=torch.zeros(1, 4, dtype=torch.int32).expand(2, 4))
    with pytest.raises(lsb.LoraError, match="ld_table 3"):
        attention(table=torch.zeros(16, dtype=torch.int32).as_strided((2, 4), (3, 1)))
    with pytest.raises(lsb.LoraError, match="ld_mask 0"):
        attention(mask=torch.zeros(1, 2, dtype=torch.int64).expand(3, 2))
    pool = torch.zeros(2, 8, 16, 2, 64, dtype=torch.float16)
    ints = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    cache = lsb.PageCache(pool, ints(8), torch.full((1, 4), -1, dtype=torch.int32).expand(3, 4), ints(3))
    with pytest.raises(lsb.LoraError, match="ld_table 0"):
        lsb.lora_pages_free(cache, ints(1))
    cache = lsb.PageCache(pool, ints(8), torch.full((3, 4), -1, dtype=torch.int32), ints(3))
    with pytest.raises(lsb.LoraError, match="ld_path 0"):
        lsb.lora_pages_accept(cache, ints(2), ints(2), torch.zeros(1, 3, dtype=torch.int32).expand(2, 3), ints(2), ints(2))
    x = torch.zeros(1, 128, dtype=torch.float16).expand(4, 128)
    w = lsb.Q4Weight(torch.zeros(2048, dtype=torch.uint8), 16, 128, 128, False, torch.float16)
    with pytest.raises(lsb.LoraError, match="ldx 0"):
        lsb.lora_q4_matmul(x, w, torch.zeros(4, 16, dtype=torch.float16))


def test_lone_rows_may_have_any_stride(no_gpu, monkeypatch):
    """The stride of a single row means nothing: it passes as the width."""
    got = []

    class Stub:
        def lora_tree_attention_workspace_bytes(self, *a):
            return 0

        def lora_tree_attention(self, *a):
            got.append((D._CKvLayer.from_buffer_copy(a[3]), D._CTreeBatch.from_buffer_copy(a[4])))
            return 0

        def lora_pages_accept(self, *a):
            got.append(a[4:6])
            return 0

    monkeypatch.setattr(lsb, "lib", lambda: Stub())
    monkeypatch.setattr(D._base, "lib", lambda: Stub())
    attention(table=torch.zeros(16, dtype=torch.int32).as_strided((1, 4), (1, 1)),
              mask=torch.zeros(16, dtype=torch.int64).as_strided((1, 2), (0, 1)), T=1, B=1)
    assert got[0][1].ld_table == 4 and got[0][1].ld_mask == 2
    ints = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    cache = lsb.PageCache(torch.zeros(2, 8, 16, 2, 64, dtype=torch.float16), ints(8),
                          torch.zeros(8, dtype=torch.int32).as_strided((1, 4), (2, 1)), ints(1))
    assert cache.c.ld_table == 4
    lsb.lora_pages_accept(cache, ints(1), ints(1), torch.zeros(8, dtype=torch.int32).as_strided((1, 3), (1, 1)), ints(1), ints(1))
    assert got[1] == (3, 3)
