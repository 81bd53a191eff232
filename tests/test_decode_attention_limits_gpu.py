"""Tree attention at the ends of what its arguments can say."""
import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb
from test_decode_attention_gpu import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,B,kv,pages", [(4096, 4096, 16, 40), (4096, 4096, 16, 100), (64, 3000, 4, 40), (8, 3, 2, 2)])
def test_starts_that_do_not_ascend(T, B, kv, pages):
    """0, T, 0, T, ...: far more rows than there are, tiles of which 32 bits lose
    count.  Nothing is written behind the outputs, and the next call is right."""
    dim, page = 64, 1024
    q = torch.zeros(T + 2, kv, dim, dtype=torch.float16, device="cuda")
    k = torch.zeros(1, page, kv, dim, dtype=torch.float16, device="cuda")
    table = torch.zeros(B, pages, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, T] * (B // 2) + [0] * (1 + B % 2), dtype=torch.int32, device="cuda")[:B + 1]
    ctx = torch.full((B,), pages * page - T, dtype=torch.int32, device="cuda")
    out = torch.full((T + 2, kv, dim), 9.0, dtype=torch.float16, device="cuda")
    need = lsb.lora_tree_attention_workspace_bytes(B, T, kv, kv, dim)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    lsb.lora_tree_attention(q[1:-1], k, k, table, ctx, start, out[1:-1], 1.0, workspace=ws[256:-256])
    torch.cuda.synchronize()
    assert bool((out[0] == 9).all()) and bool((out[-1] == 9).all())
    assert bool((ws[:256] == 77).all()) and bool((ws[-256:] == 77).all())
    b = Batch([3, 2], [1500, 90], 8, 2, 64, 16, "f16", seed=1)
    b.check(b.run())


def test_starts_out_of_range():
    """Values below 0 or above T count as 0 and T."""
    b = Batch([3, 2], [1500, 90], 8, 2, 64, 16, "f16", seed=2)
    assert torch.equal(b.run(start=b.ints([-7, 3, 2 ** 31 - 1])), b.run())


def test_many_sequences_without_rows():
    """Empty sequences between the others, in parts and in whole lines."""
    for ctx in (1300, 40):
        nodes = [0] * 70 + [2] + [0] * 130 + [1, 0, 3] + [0] * 70
        b = Batch(nodes, [ctx] * len(nodes), 4, 2, 64, 16, "bf16", seed=3)
        b.check(b.run())
