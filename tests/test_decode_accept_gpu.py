"""lora_pages_accept where drafted rows have no page: the path ends there and
new_len counts what is kept.  Results are compared bit for bit with a model."""
import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb
from test_decode_pages_gpu import NO_SPACE, OK, Model, grow, ints, status_of

pytestmark = pytest.mark.gpu


class Ending(Model):
    """The model, with paths that end at the first row without a page."""

    def accept(self, seqs, drafted, path, accepted):
        out = []
        for s, d, row, n in zip(seqs, drafted, path, accepted):
            if not 0 <= s < len(self.lens):
                out.append(0)
                continue
            base = int(self.lens[s])

            def spot(x):
                w = (base + x) // self.page
                p = int(self.table[s, w]) if base >= 0 and w < self.table.shape[1] else -1
                return (p, (base + x) % self.page) if 0 <= p < len(self.refs) else None

            kept = []
            for j, p in enumerate(row[:max(n, 0)]):
                if p <= (kept[-1] if kept else -1) or p >= d or spot(p) is None or spot(j) is None:
                    break
                kept.append(int(p))
            rows = [self.pool[:, spot(p)[0], spot(p)[1]].copy() for p in kept]
            for j, r in enumerate(rows):
                self.pool[:, spot(j)[0], spot(j)[1]] = r
            out.append(base + len(kept))
        return out


def accept(m, c, seqs, drafted, path, kept):
    new = status_of(len(seqs))
    lsb.lora_pages_accept(c, ints(seqs), ints(drafted), ints(path), ints(kept), new)
    want = m.accept(seqs, drafted, path, kept)
    assert new.tolist() == want
    m.same(c)
    return want


@pytest.mark.parametrize("head_major", [False, True])
def test_draft_without_space(head_major):
    """A draft that found no page, appended and accepted all the same."""
    m = Ending(pages=6, page=4, seqs=4, width=6, seed=1)
    c = m.device(head_major)
    grow(m, c, [0, 1], [10, 7])                        # five pages: one is left
    st = status_of(2)
    lsb.lora_pages_resize(c, ints([0, 1]), extra=ints([9, 6]), status=st)
    assert st.tolist() == m.resize([0, 1], extra=[9, 6]) == [NO_SPACE, NO_SPACE]
    k = m.rs.randint(-9000, 9000, (15, 2, 8)).astype(np.int16)
    tk = torch.from_numpy(k).cuda().view(torch.float16)
    lsb.lora_pages_append(c, 0, tk, tk, ints([0, 1]), ints([0, 9, 15]))
    m.append(0, k, k, [0, 1], [0, 9, 15])
    m.same(c)
    # Slots 10 and 11 have a page, 12 and on have none; slot 7 has, 8 has not.
    want = accept(m, c, [0, 1], [9, 6], [[0, 1, 2, 3], [0, 1, 2, 3]], [4, 4])
    assert want == [12, 8]
    want = accept(m, c, [0, 1], [9, 6], [[1, 2, 3, 4], [1, 2, 3, 4]], [4, 4])
    assert want == [11, 7]
    st = status_of(2)
    lsb.lora_pages_resize(c, ints([0, 1]), lens=ints(want), status=st)
    assert st.tolist() == m.resize([0, 1], want) == [OK, OK]
    m.same(c)
    m.sound()


def test_holes_and_ends_of_rows():
    """Missing pages inside a row, ids out of range, lengths beyond the row."""
    m = Ending(pages=30, page=2, seqs=5, width=8, seed=2)
    c = m.device()
    grow(m, c, [0, 1, 2, 3], [3, 3, 3, 15])
    lsb.lora_pages_resize(c, ints([0, 1, 2]), extra=ints([9, 9, 9]))
    m.resize([0, 1, 2], extra=[9, 9, 9])
    for s, w, p in ((0, 3, -1), (1, 2, 30), (2, 1, 10 ** 6)):
        m.table[s, w] = p
        c.table[s, w] = p
    path = [[0, 2, 4, 5, 6], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4]]
    want = accept(m, c, [0, 1, 2, 3, 4], [9, 9, 9, 9, 9], path, [5] * 5)
    assert want == [5, 4, 3, 16, 0]


@pytest.mark.parametrize("length", [-5, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 3])
def test_lengths_out_of_range(length):
    m = Ending(seed=3)
    c = m.device()
    grow(m, c, [1], [6])
    m.lens[1] = length
    c.seq_len[1] = length
    assert accept(m, c, [1], [4], [[0, 1, 2]], [3]) == [length]


@pytest.mark.parametrize("missing", [63, 64, 65, 130, 200])
def test_long_path_ends(missing):
    """Paths of more entries than a wave has lanes, ending anywhere."""
    m = Ending(pools=2, pages=300, page=1, heads=1, seqs=2, width=270, seed=4)
    c = m.device()
    grow(m, c, [0], [3])
    lsb.lora_pages_resize(c, ints([0]), extra=ints([260]))
    m.resize([0], extra=[260])
    m.table[0, 3 + missing] = -1
    c.table[0, 3 + missing] = -1
    kept = list(range(2, 252))
    assert accept(m, c, [0], [260], [kept], [250]) == [3 + missing - 2]
