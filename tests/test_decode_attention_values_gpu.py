"""Tree attention where values are not finite beside missing pages
(lora_tree_attention), against the definition in 64 bits.  The tolerance is that
of test_decode_attention_gpu."""
import numpy as np
import pytest
import torch

from test_decode_attention_gpu import Batch

pytestmark = pytest.mark.gpu


def position(b, seq, p):
    return b.table[seq, p // b.page], p % b.page


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nodes,heads,kv,dim", [(1, 16, 8, 128), (3, 64, 8, 128), (9, 64, 8, 64), (3, 32, 4, 256), (4, 24, 4, 80)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_missing_pages_and_values_that_are_not_finite(nodes, heads, kv, dim, dtype, value):
    """Pages of the context are missing, and seen values beside them are not
    finite in one column: that column of their head is spoilt, the others are
    the definition's.  Twelve sequences, so that a workgroup takes several tiles
    of positions one after the other."""
    B = 12
    b = Batch([nodes] * B, [1400 - 7 * i for i in range(B)], heads, kv, dim, 16, dtype, seed=nodes + dim)
    hit = [37, 390, 70, 1000]                          # beside a missing page, three times; beside none
    for s in range(B):
        b.table[s, [3, 25, 61]] = [-1, -7, 10 ** 6]
        for p in hit:
            b.v[position(b, s, p)][0, 5] = value
    got = b.run()
    spoilt = got[:, :heads // kv, 5].double().cpu().numpy()
    assert not np.isfinite(spoilt).any()
    if value == float("inf"):
        assert (spoilt > 0).all()
    for s in range(B):
        for p in hit:
            b.v[position(b, s, p)][0, 5] = 0.0         # the definition's other columns
    got[:, :heads // kv, 5] = torch.from_numpy(b.expect()[0][:, :heads // kv, 5]).to(got)
    b.check(got)
