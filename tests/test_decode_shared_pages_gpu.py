"""Pages that several sequences hold are never written through one of them: a
sequence cut inside such a page (lora_pages_resize with a shorter length) gets
a page of its own with its filled rows, before an append or an accept can
reach it.  Results are compared bit for bit with a model on the host."""
import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb
from test_decode_pages_gpu import BAD, NO_SPACE, OK, Model, ints, status_of

pytestmark = pytest.mark.gpu


class Owning(Model):
    """The model, with a resize that leaves no sequence a shared page at or
    behind its end."""

    def __init__(self, **a):
        super().__init__(**a)
        self.taken = []  # pages that were copied into: the last slot of the first pool holds notes

    def resize(self, seqs, lens=None, extra=None):
        counts = self.refs.copy()
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        dry, status, done, drop = False, [], set(), []
        for i, s in enumerate(seqs):
            length = None if not 0 <= s < len(self.lens) else int(self.lens[s] if lens is None else lens[i])
            more = 0 if extra is None else int(extra[i])
            if length is None or s in done or length < 0 or more < 0 or self.pages_of(length + more) > self.table.shape[1]:
                status.append(BAD)
                done.add(s)
                continue
            done.add(s)
            want, row = self.pages_of(length + more), self.table[s]
            have = int(np.argmax(np.append(row, -1) < 0))
            first, rest = divmod(length, self.page)
            shared = [w for w in range(first, min(have, want)) if counts[row[w]] > 1] if lens is not None else []
            own = shared[-1] - first + 1 if shared else 0
            need = own + max(want - have, 0)
            if need and (dry or need > len(free)):
                dry = True
                status.append(NO_SPACE)
                continue
            for w in range(first, first + own):
                old, row[w] = row[w], free.pop(0)
                self.refs[row[w]] = 1
                if w == first and rest:
                    self.pool[:, row[w], :rest] = self.pool[:, old, :rest]
                    self.taken.append(int(row[w]))
                drop.append(old)
            for w in range(have, want):
                row[w] = free.pop(0)
                self.refs[row[w]] = 1
            drop += [p for p in row[want:have]]
            row[want:] = -1
            if lens is not None:
                self.lens[s] = length
            status.append(OK)
        for p in drop:
            self.refs[p] -= 1
        return status

    def same(self, cache):
        pool = cache.pool.view(torch.int16).cpu().numpy()
        if cache.head_major:
            pool = pool.transpose(0, 1, 3, 2, 4)
        for p in self.taken:
            self.pool[0, p, -1] = pool[0, p, -1]
        self.taken = []
        super().same(cache)

    def tokens(self, s):
        """What sequence s sees, in every pool."""
        at = np.arange(self.lens[s])
        return self.pool[:, self.table[s, at // self.page], at % self.page].copy()

    def private(self):
        """No page at or behind a sequence's end is anybody else's."""
        for s, n in enumerate(self.lens):
            tail = self.table[s, n // self.page:]
            assert (self.refs[tail[tail >= 0]] == 1).all(), s


def resize(m, c, seqs, lens=None, extra=None):
    st = status_of(len(seqs))
    lsb.lora_pages_resize(c, ints(seqs), lens=None if lens is None else ints(lens),
                          extra=None if extra is None else ints(extra), status=st)
    want = m.resize(seqs, lens, extra)
    assert st.tolist() == want
    m.same(c)
    m.sound()
    return want


def fork(m, c, src, dst):
    st = status_of(len(src))
    lsb.lora_pages_fork(c, ints(src), ints(dst), st)
    want = m.fork(src, dst)
    assert st.tolist() == want
    m.same(c)
    return want


def append(m, c, layer, seqs, counts):
    T = int(np.sum(counts))
    k, v = (m.rs.randint(-9000, 9000, (T, m.heads, m.dim)).astype(np.int16) for _ in range(2))
    start = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    tk, tv = (torch.from_numpy(x).cuda().view(torch.float16) for x in (k, v))
    lsb.lora_pages_append(c, layer, tk, tv, ints(seqs), ints(start))
    m.append(layer, k, v, seqs, start)


@pytest.mark.parametrize("head_major", [False, True])
def test_branch_cut_to_a_prefix(head_major):
    """A prompt of two full pages, a branch cut inside the second one: what is
    appended to the branch does not reach the prompt."""
    m = Owning(page=16, seed=1)
    c = m.device(head_major)
    resize(m, c, [0], [32])
    fork(m, c, [0], [1])
    prompt = m.tokens(0)
    assert resize(m, c, [1], [20], [9]) == [OK]
    assert m.table[1, 0] == m.table[0, 0] and m.table[1, 1] != m.table[0, 1]
    append(m, c, 0, [1], [9])
    append(m, c, 1, [1], [9])
    m.same(c)
    np.testing.assert_array_equal(m.tokens(0), prompt)
    np.testing.assert_array_equal(m.tokens(1), prompt[:, :20])
    new = status_of(1)
    lsb.lora_pages_accept(c, ints([1]), ints([9]), ints([[1, 4, 8]]), ints([3]), new)
    assert new.tolist() == m.accept([1], [9], [[1, 4, 8]], [3]) == [23]
    m.same(c)
    np.testing.assert_array_equal(m.tokens(0), prompt)


def test_every_page_behind_the_cut():
    """Shared pages that stay for tokens to come are replaced too, and a cut at
    a page's end copies nothing."""
    m = Owning(pages=40, seqs=6, width=8, seed=2)
    c = m.device()
    resize(m, c, [0], [30])
    fork(m, c, [0] * 4, [1, 2, 3, 4])
    prompt = m.tokens(0)
    assert resize(m, c, [1, 2, 3, 4], [5, 8, 0, 27], [20, 3, 13, 1]) == [OK] * 4
    m.private()
    for layer in range(2):
        append(m, c, layer, [1, 2, 3, 4], [20, 3, 13, 1])
    m.same(c)
    np.testing.assert_array_equal(m.tokens(0), prompt)
    for s, n in ((1, 5), (2, 8), (4, 27)):
        np.testing.assert_array_equal(m.tokens(s), prompt[:, :n])


def test_all_holders_cut_at_once():
    """Every holder of a page is cut in one call: counts before the call decide,
    so each gets a page of its own and the old one is free afterwards."""
    m = Owning(pages=20, seed=3)
    c = m.device()
    resize(m, c, [0], [8])
    fork(m, c, [0, 0], [1, 2])
    old = int(m.table[0, 1])
    assert resize(m, c, [0, 1, 2, 1], [6, 7, 5, 3]) == [OK, OK, OK, BAD]
    m.private()
    assert m.refs[old] == 0


def test_no_page_left_for_a_cut():
    """Without a free page the entry is unchanged, and so is every later one
    that needs a page; entries that need none are served."""
    m = Owning(pages=5, seqs=4, width=5, seed=4)
    c = m.device()
    resize(m, c, [0, 3], [16, 3])
    fork(m, c, [0, 0], [1, 2])
    assert resize(m, c, [1, 2, 0, 3], [5, 8, 15, 6], [4, 0, 0, 0]) == [NO_SPACE, OK, NO_SPACE, NO_SPACE]
    lsb.lora_pages_free(c, ints([2]))
    m.free([2])
    m.same(c)
    assert resize(m, c, [3, 1], [0, 13], [0, 3]) == [OK, NO_SPACE]  # pages released by a call serve later calls
    assert resize(m, c, [1], [13], [3]) == [OK]
    m.private()


@pytest.mark.parametrize("page,heads,dim,pools,head_major", [(16, 8, 128, 6, False), (24, 3, 80, 2, True),
                                                             (2, 1, 8, 2, False), (64, 4, 64, 10, True), (1, 2, 8, 2, False)])
def test_page_shapes(page, heads, dim, pools, head_major):
    m = Owning(pools=pools, pages=30, page=page, heads=heads, dim=dim, width=4, seed=5)
    c = m.device(head_major)
    n = 3 * page
    resize(m, c, [0], [n])
    fork(m, c, [0, 0, 0], [1, 2, 3])
    prompt = m.tokens(0)
    cuts = [n - 1, n // 2, max(1, page - 1)]
    assert resize(m, c, [1, 2, 3], cuts, [1, 1, 1]) == [OK] * 3
    append(m, c, 0, [1, 2, 3], [1, 1, 1])
    m.same(c)
    m.private()
    np.testing.assert_array_equal(m.tokens(0), prompt)
    for s, k in zip((1, 2, 3), cuts):
        np.testing.assert_array_equal(m.tokens(s), prompt[:, :k])


def test_many_cuts():
    n = 700
    m = Owning(pools=2, pages=6 * n, page=4, heads=1, dim=8, seqs=n, width=6, seed=6)
    c = m.device()
    resize(m, c, [0], [20])
    fork(m, c, [0] * (n - 1), list(range(1, n)))
    prompt = m.tokens(0)
    lens = m.rs.randint(0, 21, n - 1).tolist()
    extra = m.rs.randint(0, 4, n - 1).tolist()
    assert resize(m, c, list(range(1, n)), lens, extra) == [OK] * (n - 1)
    m.private()
    append(m, c, 0, list(range(1, n)), extra)
    m.same(c)
    np.testing.assert_array_equal(m.tokens(0), prompt)


@pytest.mark.parametrize("seed", [7, 8])
def test_random_life(seed):
    """Mixed calls with appends and accepts: after each the device holds what
    the model holds, and no sequence's tokens change unless it was named."""
    m = Owning(pools=2, pages=41, page=3, heads=1, dim=8, seqs=9, width=9, seed=seed)
    c = m.device()
    rs = np.random.RandomState(seed)
    cuts = 0
    for step in range(80):
        before = [m.tokens(s) for s in range(9)]
        op, n = rs.randint(5), rs.randint(1, 6)
        if op == 0:
            touched, lens = rs.randint(-1, 10, n).tolist(), rs.randint(0, 26, n).tolist()
            held = m.taken[:]
            st = status_of(n)
            lsb.lora_pages_resize(c, ints(touched), lens=ints(lens), status=st)
            assert st.tolist() == m.resize(touched, lens), step
            cuts += len(m.taken) - len(held)
        elif op == 1:
            src, touched = rs.randint(-1, 10, n).tolist(), rs.randint(0, 9, n).tolist()
            st = status_of(n)
            lsb.lora_pages_fork(c, ints(src), ints(touched), st)
            assert st.tolist() == m.fork(src, touched), step
        elif op == 2 and rs.rand() < 0.4:
            touched = rs.randint(-2, 11, n).tolist()
            lsb.lora_pages_free(c, ints(touched))
            m.free(touched)
        elif op == 4 and rs.rand() < 0.4:
            touched, live = [], status_of(1)
            lsb.lora_pages_compact(c, live)
            assert live.tolist() == [m.compact()]
        else:  # a drafted step of distinct sequences
            touched = rs.permutation(9)[:n].tolist()
            counts = rs.randint(1, 5, n).tolist()
            st = status_of(n)
            lsb.lora_pages_resize(c, ints(touched), extra=ints(counts), status=st)
            want = m.resize(touched, extra=counts)
            assert st.tolist() == want, step
            fits = [i for i in range(n) if want[i] == OK]
            touched, counts = [touched[i] for i in fits], [counts[i] for i in fits]
            if touched:
                append(m, c, 0, touched, counts)
                path = [np.sort(rs.permutation(k)[:3]).tolist() + [0] * max(0, 3 - k) for k in counts]
                kept = [int(rs.randint(0, min(k, 3) + 1)) for k in counts]
                new = status_of(len(touched))
                lsb.lora_pages_accept(c, ints(touched), ints(counts), ints(path), ints(kept), new)
                lens = m.accept(touched, counts, path, kept)
                assert new.tolist() == lens
                lsb.lora_pages_resize(c, ints(touched), lens=new)
                assert m.resize(touched, lens) == [OK] * len(touched)
        m.same(c)
        m.sound()
        m.private()
        for s in set(range(9)) - set(touched):
            np.testing.assert_array_equal(m.tokens(s), before[s])
    assert cuts


def test_random_steps():
    """The run of test_decode_pages_gpu's test of the same name."""
    m = Owning(pools=2, pages=37, page=3, heads=1, dim=8, seqs=9, width=8, seed=2)
    c = m.device()
    rs = np.random.RandomState(3)
    for step in range(60):
        op = rs.randint(5)
        n = rs.randint(1, 6)
        if op == 0:
            seqs, lens = rs.randint(-1, 10, n).tolist(), rs.randint(0, 26, n).tolist()
            resize(m, c, seqs, lens)
        elif op == 1:
            fork(m, c, rs.randint(-1, 10, n).tolist(), rs.randint(0, 9, n).tolist())
        elif op == 2:
            seqs = rs.randint(-2, 11, n).tolist()
            lsb.lora_pages_free(c, ints(seqs))
            m.free(seqs)
        elif op == 3:
            resize(m, c, rs.randint(0, 9, n).tolist(), extra=rs.randint(-1, 6, n).tolist())
        else:
            live = status_of(1)
            lsb.lora_pages_compact(c, live)
            assert live.tolist() == [m.compact()]
        m.same(c)
        m.sound()
        m.private()


def test_graph_replays():
    """A captured cut, draft and fork, replayed between eager work."""
    m = Owning(pages=60, width=8, seed=9)
    c = m.device()
    resize(m, c, [0], [20])
    src, dst, cut, more, start = ints([0, 0]), ints([1, 2]), ints([10, 17]), ints([3, 5]), ints([0, 3, 8])
    k = torch.zeros(8, 2, 8, dtype=torch.float16, device="cuda")
    ws = torch.empty(lsb.lora_pages_fork_workspace_bytes(2, 8), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lsb.lora_pages_fork(c, src, dst, workspace=ws)
        lsb.lora_pages_resize(c, dst, lens=cut, extra=more)
        lsb.lora_pages_append(c, 0, k, k, dst, start)
    prompt = m.tokens(0)
    for lens in ([10, 17], [3, 20], [16, 0], [19, 1]):
        cut.copy_(ints(lens))
        data = m.rs.randint(-9000, 9000, (8, 2, 8)).astype(np.int16)
        k.view(torch.int16).copy_(torch.from_numpy(data))
        graph.replay()
        torch.cuda.synchronize()
        m.fork([0, 0], [1, 2])
        assert m.resize([1, 2], lens, [3, 5]) == [OK, OK]
        m.append(0, data, data, [1, 2], [0, 3, 8])
        m.same(c)
        m.sound()
        np.testing.assert_array_equal(m.tokens(0), prompt)
