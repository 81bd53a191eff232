"""Page operations (lora_pages_*) against a model of the cache on the host.
Everything here moves whole values: results are compared bit for bit."""
import numpy as np
import pytest
import torch

import lora_serving_build_amd as lsb

pytestmark = pytest.mark.gpu

OK, NO_SPACE, BAD = lsb.PAGES_OK, lsb.PAGES_NO_SPACE, lsb.PAGES_BAD


class Model:
    """The cache as plain arrays; a device cache is made from it."""

    def __init__(self, pools=4, pages=24, page=4, heads=2, dim=8, seqs=6, width=6, seed=0):
        self.rs = np.random.RandomState(seed)
        self.page, self.heads, self.dim = page, heads, dim
        self.pool = self.rs.randint(-30000, 30000, (pools, pages, page, heads, dim)).astype(np.int16)
        self.refs = np.zeros(pages, np.int32)
        self.table = np.full((seqs, width), -1, np.int32)
        self.lens = np.zeros(seqs, np.int32)

    def device(self, head_major=False, dtype=torch.float16):
        pool = self.pool.transpose(0, 1, 3, 2, 4) if head_major else self.pool
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        return lsb.PageCache(t(pool).view(dtype), t(self.refs), t(self.table), t(self.lens), head_major=head_major)

    def same(self, cache):
        pool = cache.pool.view(torch.int16).cpu().numpy()
        if cache.head_major:
            pool = pool.transpose(0, 1, 3, 2, 4)
        np.testing.assert_array_equal(cache.refs.cpu().numpy(), self.refs)
        np.testing.assert_array_equal(cache.table.cpu().numpy(), self.table)
        np.testing.assert_array_equal(cache.seq_len.cpu().numpy(), self.lens)
        np.testing.assert_array_equal(pool, self.pool)

    def sound(self):
        """Every live page is counted as often as rows name it."""
        named = np.bincount(self.table[self.table >= 0], minlength=len(self.refs))
        np.testing.assert_array_equal(named, self.refs)

    def pages_of(self, tokens):
        return -(-int(tokens) // self.page)

    # -- the operations, one entry after the other
    def resize(self, seqs, lens=None, extra=None):
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        dry, status, done, drop = False, [], set(), []
        for i, s in enumerate(seqs):
            length = None if not 0 <= s < len(self.lens) else self.lens[s] if lens is None else lens[i]
            more = 0 if extra is None else extra[i]
            if length is None or s in done or length < 0 or more < 0 or self.pages_of(int(length) + int(more)) > self.table.shape[1]:
                status.append(BAD)
                done.add(s)
                continue
            done.add(s)
            want, row = self.pages_of(int(length) + int(more)), self.table[s]
            have = int(np.argmax(np.append(row, -1) < 0))
            if want > have and (dry or want - have > len(free)):
                dry = True
                status.append(NO_SPACE)
                continue
            for w in range(have, want):
                row[w] = free.pop(0)
                self.refs[row[w]] = 1
            drop += [(s, w) for w in range(want, have)]
            if lens is not None:
                self.lens[s] = length
            status.append(OK)
        for s, w in drop:
            self.refs[self.table[s, w]] -= 1
            self.table[s, w] = -1
        return status

    def fork(self, src, dst):
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        before, lens = self.table.copy(), self.lens.copy()
        status, done, dry, drop = [], set(), False, []
        for a, b in zip(src, dst):
            repeated = b in done
            done.add(b)
            if repeated or not (0 <= a < len(lens) and 0 <= b < len(lens)):
                status.append(BAD)
                continue
            full, rest = divmod(int(lens[a]), self.page)
            if rest and (dry or not free):
                dry = True
                status.append(NO_SPACE)
                continue
            new = np.full(self.table.shape[1], -1, np.int32)
            new[:full] = before[a, :full]
            for p in new[:full]:
                self.refs[p] += 1
            if rest:
                new[full] = free.pop(0)
                self.refs[new[full]] = 1
                self.pool[:, new[full], :rest] = self.pool[:, before[a, full], :rest]
            drop += [p for p in before[b] if p >= 0]
            self.table[b], self.lens[b] = new, lens[a]
            status.append(OK)
        for p in drop:
            self.refs[p] -= 1
        return status

    def free(self, seqs):
        for s in dict.fromkeys(seqs):
            if 0 <= s < len(self.lens):
                for p in self.table[s][self.table[s] >= 0]:
                    self.refs[p] -= 1
                self.table[s], self.lens[s] = -1, 0

    def append(self, layer, k, v, seqs, start):
        for i, s in enumerate(seqs):
            for t in range(start[i], start[i + 1]):
                pos = int(self.lens[s]) + t - start[i] if 0 <= s < len(self.lens) else -1
                if pos >= 0 and pos // self.page < self.table.shape[1]:
                    p = self.table[s, pos // self.page]
                    if p >= 0:
                        self.pool[2 * layer, p, pos % self.page] = k[t]
                        self.pool[2 * layer + 1, p, pos % self.page] = v[t]

    def accept(self, seqs, drafted, path, accepted):
        out = []
        for s, d, row, n in zip(seqs, drafted, path, accepted):
            if not 0 <= s < len(self.lens):
                out.append(0)
                continue
            kept = []
            for p in row[:max(n, 0)]:
                if p <= (kept[-1] if kept else -1) or p >= d:
                    break
                kept.append(int(p))
            base = int(self.lens[s])
            spot = lambda x: (self.table[s, x // self.page], x % self.page)  # noqa: E731
            rows = [self.pool[:, spot(base + p)[0], spot(base + p)[1]].copy() for p in kept]
            for j, r in enumerate(rows):
                self.pool[:, spot(base + j)[0], spot(base + j)[1]] = r
            out.append(base + len(kept))
        return out

    def compact(self):
        live = int((self.refs != 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        moves = [p for p in range(live, len(self.refs)) if self.refs[p] != 0]
        for a, b in zip(moves, holes):
            self.pool[:, b] = self.pool[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
        return live


def ints(v):
    return torch.tensor(np.asarray(v, np.int32).reshape(np.shape(v)), device="cuda")


def status_of(n):
    return torch.full((n,), 77, dtype=torch.int32, device="cuda")


def grow(m, c, seqs, lens):
    st = status_of(len(seqs))
    lsb.lora_pages_resize(c, ints(seqs), lens=ints(lens), status=st)
    want = m.resize(seqs, lens)
    assert st.tolist() == want
    return want


@pytest.mark.parametrize("head_major", [False, True])
def test_life_of_a_cache(head_major):
    """Prompts, forks, drafted tokens, an accepted path, freeing, compaction:
    after each call the device holds what the model holds."""
    m = Model(seed=1)
    c = m.device(head_major)
    assert grow(m, c, [0, 2, 3], [9, 0, 4]) == [OK] * 3
    m.same(c)
    m.sound()
    st = status_of(3)
    lsb.lora_pages_fork(c, ints([0, 3, 0]), ints([1, 4, 5]), st)
    assert st.tolist() == m.fork([0, 3, 0], [1, 4, 5]) == [OK] * 3
    m.same(c)
    m.sound()
    # drafted tokens of three sequences
    seqs, drafts = [1, 4, 0], [5, 3, 0]
    st = status_of(3)
    lsb.lora_pages_resize(c, ints(seqs), extra=ints(drafts), status=st)
    assert st.tolist() == m.resize(seqs, extra=drafts) == [OK] * 3
    k, v = (m.rs.randint(-9000, 9000, (8, 2, 8)).astype(np.int16) for _ in range(2))
    tk, tv = (torch.from_numpy(x).cuda().view(torch.float16) for x in (k, v))
    lsb.lora_pages_append(c, 1, tk, tv, ints(seqs), ints([0, 5, 8, 8]))
    m.append(1, k, v, seqs, [0, 5, 8, 8])
    m.same(c)
    path, kept = [[0, 2, 4], [1, 2, 0], [0, 0, 0]], [3, 2, 0]
    new = status_of(3)
    lsb.lora_pages_accept(c, ints(seqs), ints(drafts), ints(path), ints(kept), new)
    want = m.accept(seqs, drafts, path, kept)
    assert new.tolist() == want == [12, 6, 9]
    m.same(c)
    grow(m, c, seqs, want)                               # the lengths, and back to the pages they need
    m.same(c)
    m.sound()
    lsb.lora_pages_free(c, ints([0, 3, 0, -1, 6]))
    m.free([0, 3, 0, -1, 6])
    m.same(c)
    m.sound()
    live = status_of(1)
    lsb.lora_pages_compact(c, live)
    assert live.tolist() == [m.compact()]
    m.same(c)
    m.sound()


def test_random_steps():
    """Long runs of mixed calls on a tight pool."""
    m = Model(pools=2, pages=37, page=3, heads=1, dim=8, seqs=9, width=8, seed=2)
    c = m.device()
    rs = np.random.RandomState(3)
    for step in range(60):
        op = rs.randint(5)
        n = rs.randint(1, 6)
        if op == 0:
            seqs, lens = rs.randint(-1, 10, n).tolist(), rs.randint(0, 26, n).tolist()
            grow(m, c, seqs, lens)
        elif op == 1:
            src, dst = rs.randint(-1, 10, n).tolist(), rs.randint(0, 9, n).tolist()
            st = status_of(n)
            lsb.lora_pages_fork(c, ints(src), ints(dst), st)
            assert st.tolist() == m.fork(src, dst), step
        elif op == 2:
            seqs = rs.randint(-2, 11, n).tolist()
            lsb.lora_pages_free(c, ints(seqs))
            m.free(seqs)
        elif op == 3:
            seqs, extra = rs.randint(0, 9, n).tolist(), rs.randint(-1, 6, n).tolist()
            st = status_of(n)
            lsb.lora_pages_resize(c, ints(seqs), extra=ints(extra), status=st)
            assert st.tolist() == m.resize(seqs, extra=extra), step
        else:
            live = status_of(1)
            lsb.lora_pages_compact(c, live)
            assert live.tolist() == [m.compact()]
        m.same(c)
        m.sound()


def test_reorder_with_chains_and_cycles():
    """Destinations that are sources: every entry sees the state before the call."""
    m = Model(pages=40, seed=4)
    c = m.device()
    grow(m, c, [0, 1, 2, 3, 4, 5], [5, 8, 3, 0, 11, 1])
    for src, dst in (([1, 0, 2, 2, 5, 4], [0, 1, 2, 3, 4, 5]), ([0, 0, 0], [1, 2, 0]), ([3], [3])):
        st = status_of(len(src))
        lsb.lora_pages_fork(c, ints(src), ints(dst), st)
        assert st.tolist() == m.fork(src, dst)
        m.same(c)
        m.sound()


def test_pool_runs_dry():
    m = Model(pages=5, seqs=6, width=6, seed=5)
    c = m.device()
    assert grow(m, c, [0, 1, 2, 3], [6, 20, 4, 0]) == [OK, NO_SPACE, NO_SPACE, OK]
    m.same(c)
    m.sound()
    assert grow(m, c, [1, 2], [9, 1]) == [OK, NO_SPACE]
    st = status_of(4)
    lsb.lora_pages_fork(c, ints([1, 0, 3, 0]), ints([4, 5, 2, 2]), st)
    assert st.tolist() == m.fork([1, 0, 3, 0], [4, 5, 2, 2]) == [NO_SPACE, NO_SPACE, OK, BAD]
    m.same(c)
    m.sound()


def test_entries_that_are_refused():
    m = Model(seed=6)
    c = m.device()
    assert grow(m, c, [0, 0, 6, -1, 1, 2], [4, 8, 4, 4, 25, -1]) == [OK, BAD, BAD, BAD, BAD, BAD]
    m.same(c)
    st = status_of(4)
    lsb.lora_pages_fork(c, ints([0, 0, 9, 0]), ints([1, 1, 2, -3]), st)
    assert st.tolist() == m.fork([0, 0, 9, 0], [1, 1, 2, -3]) == [OK, BAD, BAD, BAD]
    m.same(c)


@pytest.mark.parametrize("row,drafted,kept", [([0, 1, 2], 4, 3), ([3, 2, 1], 4, 3), ([1, 1, 2], 4, 3), ([0, 4, 5], 5, 3),
                                              ([-1, 0, 1], 4, 3), ([2, 3, 3], 4, 9), ([1, 2, 3], 4, -2), ([1, 2, 3], 0, 3)])
def test_path_ends_at_its_first_bad_entry(row, drafted, kept):
    m = Model(seed=7)
    c = m.device()
    grow(m, c, [2], [3])
    lsb.lora_pages_resize(c, ints([2]), extra=ints([6]))
    m.resize([2], extra=[6])
    new = status_of(2)
    lsb.lora_pages_accept(c, ints([2, 99]), ints([drafted, 4]), ints([row, row]), ints([kept, 2]), new)
    assert new.tolist() == m.accept([2, 99], [drafted, 4], [row, row], [kept, 2])
    m.same(c)


def test_long_path_overlaps_itself():
    """A path whose rows move by one place, many pages long."""
    m = Model(pages=80, page=4, seqs=2, width=70, pools=2, seed=8)
    c = m.device()
    grow(m, c, [1], [5])
    lsb.lora_pages_resize(c, ints([1]), extra=ints([257]))
    m.resize([1], extra=[257])
    path = [list(range(1, 257))]
    new = status_of(1)
    lsb.lora_pages_accept(c, ints([1]), ints([257]), ints(path), ints([256]), new)
    assert new.tolist() == m.accept([1], [257], path, [256]) == [261]
    m.same(c)


@pytest.mark.parametrize("page,heads,dim,head_major", [(16, 8, 128, False), (24, 3, 80, True), (1, 1, 8, False), (64, 4, 64, True)])
def test_copy_whole_pages(page, heads, dim, head_major):
    m = Model(pools=3, pages=12, page=page, heads=heads, dim=dim, seed=9)
    c = m.device(head_major, torch.bfloat16)
    src, dst = [0, 11, 4, 4, 7, -1, 3, 12, 9], [1, 2, 3, 5, 7, 6, 99, 8, 9]
    lsb.lora_pages_copy(c, ints(src), ints(dst))
    for a, b in zip(src, dst):
        if 0 <= a < 12 and 0 <= b < 12:
            m.pool[:, b] = m.pool[:, a]
    m.same(c)


def test_large_rounds_of_the_scan():
    """More pages than one round of the allocation scan, most of them taken."""
    m = Model(pools=1, pages=40000, page=1, heads=1, dim=8, seqs=40, width=600, seed=10)
    m.refs[m.rs.permutation(40000)[:35000]] = 1
    m.refs[39999] = 0
    held = np.flatnonzero(m.refs)
    c = m.device()
    seqs = list(range(40))
    lens = m.rs.randint(0, 250, 40).tolist()
    grow(m, c, seqs, lens)
    m.same(c)
    st = status_of(40)
    more = [100] * 40
    lsb.lora_pages_resize(c, ints(seqs), extra=ints(more), status=st)
    assert st.tolist() == m.resize(seqs, extra=more)
    m.same(c)
    assert len(held) and m.table.max() > 20000
    lsb.lora_pages_free(c, ints(seqs))
    m.free(seqs)
    m.same(c)


def test_many_entries():
    n = lsb.LORA_MAX_PAGE_ENTRIES
    m = Model(pools=1, pages=3 * n, page=2, heads=1, dim=8, seqs=n, width=3, seed=11)
    c = m.device()
    seqs = list(range(n))
    grow(m, c, seqs, (m.rs.randint(0, 7, n)).tolist())
    perm = m.rs.permutation(n).tolist()
    src = m.rs.randint(0, n, n).tolist()
    st = status_of(n)
    lsb.lora_pages_fork(c, ints(src), ints(perm), st)
    assert st.tolist() == m.fork(src, perm)
    m.same(c)
    m.sound()


def test_padded_strides():
    """Pools and pages with room between them, rows of a wider table."""
    m = Model(seed=12)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    room = torch.zeros(4, 30, 6, 2, 8, dtype=torch.int16, device="cuda")
    flat = room.view(4, 30, -1)
    pool = flat.as_strided((4, 24, 4, 2, 8), (30 * 96, 96, 16, 8, 1)).view(torch.float16)
    pool.view(torch.int16).copy_(t(m.pool))
    table = torch.full((6, 9), -5, dtype=torch.int32, device="cuda")
    table[:, :6] = -1
    c = lsb.PageCache(pool, t(m.refs), table[:, :6], t(m.lens))
    grow(m, c, [0, 1, 5], [9, 3, 24])
    lsb.lora_pages_fork(c, ints([0, 5]), ints([2, 3]))
    m.fork([0, 5], [2, 3])
    m.same(c)
    assert bool((table[:, 6:] == -5).all()) and bool((room.view(4, 30, 96)[:, 24:] == 0).all())
    assert bool((room.view(4, 30, 96)[:, :, 64:] == 0).all())


def test_append_drops_what_has_no_page():
    m = Model(seed=13)
    c = m.device()
    grow(m, c, [0, 3], [7, 22])
    k = m.rs.randint(-9000, 9000, (9, 2, 8)).astype(np.int16)
    tk = torch.from_numpy(k).cuda().view(torch.float16)
    seqs, start = [0, 3, 8, 1], [0, 3, 6, 7, 9]
    lsb.lora_pages_append(c, 0, tk, tk, ints(seqs), ints(start))
    m.append(0, k, k, seqs, start)
    m.same(c)


def test_graph_replays():
    """A captured step (grow, append, accept, fork, free) replayed with other
    data between eager work."""
    m = Model(pages=60, seed=14)
    c = m.device()
    grow(m, c, [0, 1], [6, 9])
    seqs, extra, start = ints([0, 1]), ints([4, 3]), ints([0, 4, 7])
    path, kept, new = ints([[0, 2], [1, 2]]), ints([2, 2]), status_of(2)
    src, dst, gone = ints([0, 1]), ints([2, 3]), ints([2])
    k = torch.zeros(7, 2, 8, dtype=torch.float16, device="cuda")
    ws = torch.empty(lsb.lora_pages_fork_workspace_bytes(2, 6), dtype=torch.uint8, device="cuda")

    def step():
        lsb.lora_pages_resize(c, seqs, extra=extra)
        lsb.lora_pages_append(c, 0, k, k, seqs, start)
        lsb.lora_pages_accept(c, seqs, extra, path, kept, new)
        lsb.lora_pages_resize(c, seqs, lens=new)
        lsb.lora_pages_fork(c, src, dst, workspace=ws)
        lsb.lora_pages_free(c, gone)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        data = m.rs.randint(-9000, 9000, (7, 2, 8)).astype(np.int16)
        k.view(torch.int16).copy_(torch.from_numpy(data))
        graph.replay()
        torch.cuda.synchronize()
        m.resize([0, 1], extra=[4, 3])
        m.append(0, data, data, [0, 1], [0, 4, 7])
        lens = m.accept([0, 1], [4, 3], [[0, 2], [1, 2]], [2, 2])
        assert new.tolist() == lens
        m.resize([0, 1], lens)
        m.fork([0, 1], [2, 3])
        m.free([2])
        m.same(c)
        m.sound()
