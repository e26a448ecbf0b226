"""The pages' life (mla_pages_free, _extend, _fork, _compact) through the C ABI, against a plain
sequential model: whole numbers and copied bytes have to be equal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 64
OUT_OF_RANGE, NO_PAGES = 4, 7


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def pages_of(n):
    return -(-n // PAGE)


class Model:
    """One entry after the other, as the header says."""

    def __init__(self, pages, rows, most, pools):
        self.refs = np.zeros(pages, np.int32)
        self.table = np.full((rows, most), -1, np.int32)
        self.lens = np.zeros(rows, np.int32)
        self.pools = pools
        self.most = most

    def free(self, rows):
        for r in rows:
            for k in range(pages_of(self.lens[r])):
                self.refs[self.table[r, k]] -= 1
                self.table[r, k] = -1
            self.lens[r] = 0

    def _take(self, wants):
        """Lowest free pages in the list's order; None from the first that does not fit on."""
        free = list(np.flatnonzero(self.refs == 0))
        got, failed = [], False
        for n in wants:
            failed = failed or (n > len(free))
            if n and failed:
                got.append(None)
            else:
                got.append(free[:n])
                free = free[n:]
        return got

    def extend(self, rows, lens):
        wants, seen = [], set()
        for r, n in zip(rows, lens):
            ok = 0 <= r < len(self.lens) and r not in seen and self.lens[r] <= n <= PAGE * self.most
            seen.add(r)
            wants.append(pages_of(n) - pages_of(self.lens[r]) if ok else -1)
        got = self._take([max(w, 0) for w in wants])
        for r, n, w, g in zip(rows, lens, wants, got):
            if w < 0 or g is None:
                continue
            at = pages_of(self.lens[r])
            self.table[r, at:at + w] = g
            self.refs[g] = 1
            self.lens[r] = n

    def fork(self, parents, children):
        wants, seen, rows = [], set(), len(self.lens)
        for p, c in zip(parents, children):
            ok = 0 <= p < rows and 0 <= c < rows and c not in seen and self.lens[c] == 0
            seen.add(c)
            wants.append(int(self.lens[p] % PAGE > 0) if ok else -1)
        got = self._take([max(w, 0) for w in wants])
        lens = self.lens.copy()
        for p, c, w, g in zip(parents, children, wants, got):
            if w < 0 or g is None:
                continue
            full = lens[p] // PAGE
            self.table[c, :full] = self.table[p, :full]
            self.refs[self.table[p, :full]] += 1
            if w:
                self.table[c, full] = g[0]
                self.refs[g] = 1
                for q in self.pools:
                    q[:, g[0]] = q[:, self.table[p, full]]
            self.lens[c] = lens[p]

    def compact(self):
        live = np.flatnonzero(self.refs > 0)
        n = len(live)
        movers = live[live >= n]
        holes = np.flatnonzero(self.refs[:n] == 0)
        to = np.arange(len(self.refs))
        to[movers] = holes
        for q in self.pools:
            q[:, holes] = q[:, movers]
        self.refs[holes] = self.refs[movers]
        self.refs[movers] = 0
        for r, length in enumerate(self.lens):
            k = pages_of(length)
            self.table[r, :k] = to[self.table[r, :k]]
        return n


class Device:
    def __init__(self, mla, m):
        self.mla = mla
        self.refs, self.table, self.lens = (torch.from_numpy(a.copy()).cuda()
                                            for a in (m.refs, m.table, m.lens))
        self.pools = [torch.from_numpy(p.copy()).cuda() for p in m.pools]
        self.ws = mla.alloc_workspace(mla.pages_workspace_size(len(m.refs), len(m.lens)))

    def _list(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def free(self, rows):
        self.mla.pages_free(self.refs, self.table, self.lens, self._list(rows), self.ws)

    def extend(self, rows, lens):
        self.mla.pages_extend(self.refs, self.table, self.lens, self._list(rows),
                              self._list(lens), self.ws)

    def fork(self, parents, children):
        self.mla.pages_fork(self.refs, self.table, self.lens, self._list(parents),
                            self._list(children), self.pools, self.ws)

    def compact(self, **kw):
        return self.mla.pages_compact(self.refs, self.table, self.lens, self.pools,
                                      workspace=self.ws, **kw)

    def status(self):
        return self.mla.check_device_status(self.ws)


def same(m, d, pools=True):
    assert np.array_equal(d.refs.cpu().numpy(), m.refs)
    assert np.array_equal(d.lens.cpu().numpy(), m.lens)
    assert np.array_equal(d.table.cpu().numpy(), m.table)
    for a, b in zip(d.pools if pools else [], m.pools):
        assert np.array_equal(a.cpu().numpy(), b)


def both(mla, pages, rows, most, layers=2, seed=0, fp8=False):
    rng = np.random.default_rng(seed)
    shapes = [(PAGE * 576, np.uint8), (PAGE, np.int8)] if fp8 else [(PAGE * 576, np.int16)]
    pools = [rng.integers(0, 100, (layers, pages, n)).astype(t) for n, t in shapes]
    m = Model(pages, rows, most, pools)
    return m, Device(mla, m), rng


@pytest.mark.parametrize("pages,rows,seed,fp8", [(7, 3, 0, False), (40, 9, 1, True),
                                                 (130, 30, 2, False), (300, 50, 3, True)])
def test_long_run(mla, pages, rows, seed, fp8):
    """Many random calls of every kind, some of which run out of pages."""
    m, d, rng = both(mla, pages, rows, 8, layers=1 + seed % 2, seed=seed, fp8=fp8)
    for step in range(40):
        kind = rng.integers(0, 4)
        n = int(rng.integers(1, rows + 1))
        if kind == 0:
            pick = [int(r) for r in rng.integers(0, rows, max(1, n // 3))]
            m.free(pick)
            d.free(pick)
            assert d.status() == 0
        elif kind == 1:
            pick = [int(r) for r in rng.permutation(rows)[:n]]
            lens = [int(min(8 * PAGE, m.lens[r] + rng.integers(0, 150))) for r in pick]
            m.extend(pick, lens)
            d.extend(pick, lens)
            assert d.status() in (0, NO_PAGES)
        elif kind == 2:
            empty = [int(r) for r in np.flatnonzero(m.lens == 0)][:n]
            if empty:
                par = [int(r) for r in rng.integers(0, rows, len(empty))]
                m.fork(par, empty)
                d.fork(par, empty)
                assert d.status() in (0, NO_PAGES)
        else:
            n = m.compact()
            _, _, live, _ = d.compact()
            assert live.item() == n and d.status() == 0
        same(m, d)


@pytest.mark.parametrize("pages", [1, 2, 4097, 16383, 16384, 16385, 33000, 70000])
def test_pool_sizes(mla, pages):
    """Pools around and past one pass of the scans; sizes of the copies stay small."""
    rng = np.random.default_rng(pages)
    pools = [rng.integers(0, 100, (1, pages, 16)).astype(np.uint8)]
    rows, most = 6, max(2, min(3000, pages))
    m = Model(pages, rows, most, pools)
    # pages held at random by rows 0 and 1
    held = rng.permutation(pages)[: max(1, min(pages // 2, 2 * most - 1))]
    for r, ids in enumerate(np.array_split(held, 2)):
        m.table[r, :len(ids)] = ids
        m.lens[r] = PAGE * len(ids)
        m.refs[ids] += 1
    d = Device(mla, m)
    lens = [max(1, PAGE * min(most, max(1, pages // 8)) - 3)] * 2
    m.extend([4, 2], lens)
    d.extend([4, 2], lens)
    assert d.status() in (0, NO_PAGES)
    same(m, d)
    n = m.compact()
    _, _, live, _ = d.compact()
    assert live.item() == n and d.status() == 0
    same(m, d)


def test_compact_into_other_arrays_leaves_the_old_ones(mla):
    m, d, rng = both(mla, 50, 5, 8)
    for r, n in enumerate([300, 64, 130, 500, 1]):
        m.extend([r], [n])
    m.free([0, 2])
    d = Device(mla, m)
    old = [t.clone() for t in (d.refs, d.table, d.lens)]
    refs, table = torch.full_like(d.refs, 9), torch.full_like(d.table, 9)
    _, _, live, _ = d.compact(refs_out=refs, table_out=table)
    assert all(torch.equal(a, b) for a, b in zip(old, (d.refs, d.table, d.lens)))
    n = m.compact()
    d.refs, d.table = refs, table
    assert live.item() == n and d.status() == 0
    same(m, d)


def test_strided_layers(mla):
    m, _, rng = both(mla, 20, 4, 4, layers=3)
    m.extend([0, 1], [100, 30])
    wide = torch.zeros((3, 25, PAGE * 576), dtype=torch.int16, device="cuda")
    wide[:, :20] = torch.from_numpy(m.pools[0]).cuda()
    d = Device(mla, m)
    d.pools = [wide[:, :20]]
    m.fork([0, 1, 0], [2, 3, 1])  # row 1 is not empty: refused
    d.fork([0, 1, 0], [2, 3, 1])
    assert d.status() == OUT_OF_RANGE
    same(m, d)


def test_rows_listed_twice(mla):
    m, d, _ = both(mla, 30, 6, 8)
    m.extend([1, 2], [200, 64])
    d.extend([1, 2], [200, 64])
    m.free([1])
    d.free([1, 1, 1])
    assert d.status() == 0
    same(m, d)
    m.extend([3, 3, 0], [100, 300, 5])
    d.extend([3, 3, 0], [100, 300, 5])
    assert d.status() == OUT_OF_RANGE
    same(m, d)
    m.fork([2, 3, 2], [4, 4, 5])
    d.fork([2, 3, 2], [4, 4, 5])
    assert d.status() == OUT_OF_RANGE
    same(m, d)


def test_entries_out_of_range_are_skipped(mla):
    m, d, _ = both(mla, 30, 4, 4)
    args = ([0, -1, 1, 4, 2, 3], [70, 5, 257, 5, -1, 256])
    m.extend(*args)
    d.extend(*args)
    assert d.status() == OUT_OF_RANGE
    same(m, d)
    m.extend([0], [69])  # shorter than it is
    d.extend([0], [69])
    assert d.status() == OUT_OF_RANGE
    same(m, d)
    d.fork([9, -1, 0], [1, 2, 7])
    assert d.status() == OUT_OF_RANGE
    same(m, d)
    d.free([-1, 4])
    assert d.status() == OUT_OF_RANGE
    same(m, d)


def test_bad_page_ids(mla):
    """A row with a page id outside the pool: released except for it, and not forked."""
    m, d, _ = both(mla, 10, 3, 4)
    m.extend([0], [130])
    d.extend([0], [130])
    d.table[0, 1] = 10
    d.fork([0], [1])
    assert d.status() == OUT_OF_RANGE
    assert d.lens.tolist() == [130, 0, 0] and d.refs.tolist() == [1, 1, 1] + [0] * 7
    d.free([0])
    assert d.status() == OUT_OF_RANGE
    assert d.refs.tolist() == [0, 1, 0] + [0] * 7 and d.lens.tolist() == [0, 0, 0]
    # a page that nobody holds is not released below 0
    d.table[2, 0], d.lens[2] = 5, 10
    d.free([2])
    assert d.status() == OUT_OF_RANGE
    assert d.refs.tolist() == [0, 1, 0] + [0] * 7


def test_full_list_and_empty_lists(mla):
    rows = 4096
    m, d, rng = both(mla, 5000, rows, 2, layers=1)
    order = [int(r) for r in rng.permutation(rows)]
    lens = [int(n) for n in rng.integers(0, 100, rows)]
    m.extend(order, lens)
    d.extend(order, lens)
    assert d.status() == NO_PAGES
    same(m, d, pools=False)
    d.extend([], [])
    d.free([])
    d.fork([], [])
    assert d.status() == 0
    same(m, d)


def test_captured_and_replayed(mla):
    """A turnover in a graph: every replay does it anew on the state it finds."""
    m, d, _ = both(mla, 60, 8, 6)
    m.extend([0, 1], [100, 300])
    d.extend([0, 1], [100, 300])
    rows, lens = d._list([0, 2, 3]), d._list([200])
    par, child, new = d._list([0, 0]), d._list([2, 3]), d._list([0])
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())

    def turn():
        mla.pages_free(d.refs, d.table, d.lens, rows, d.ws)
        mla.pages_extend(d.refs, d.table, d.lens, new, lens, d.ws)
        mla.pages_fork(d.refs, d.table, d.lens, par, child, d.pools, d.ws)

    with torch.cuda.graph(g, stream=s):
        turn()
    for _ in range(3):
        g.replay()
        m.free([0, 2, 3])
        m.extend([0], [200])
        m.fork([0, 0], [2, 3])
        torch.cuda.synchronize()
        assert d.status() == 0
        same(m, d)


@pytest.mark.parametrize("pages", [1, 64, 16383, 16384, 16385, 32768])
def test_compact_of_a_full_pool(mla, pages):
    """Every page held (as many as one CTA counts, and one page to either side): nothing moves,
    whatever an uncleared workspace holds."""
    m = Model(pages, 1, pages, [np.arange(8 * pages).astype(np.int16).reshape(1, pages, 8)])
    d = Device(mla, m)
    m.extend([0], [PAGE * pages])
    d.extend([0], [PAGE * pages])
    d.ws[256:] = 1  # (behind the header)
    live = d.compact()[2]
    assert live.item() == m.compact() == pages
    assert d.status() == 0
    same(m, d)


def test_fork_of_a_free_page_is_refused(mla):
    """A parent whose table names a page that nobody holds, which the same call hands out to many
    other children: refused, whichever is seen first."""
    rows = 66
    m, d, _ = both(mla, 80, rows, 2, layers=1)
    m.extend([0], [70])
    d.extend([0], [70])
    d.table[1, 0], d.lens[1] = 2, 64  # the lowest free page: handed to child 2
    for _ in range(20):
        m.fork([0] * 63, range(2, 65))
        d.fork([0] * 63 + [1], range(2, rows))
        assert d.status() == OUT_OF_RANGE
        m.table[1, 0], m.lens[1] = 2, 64
        same(m, d)
        m.table[1, 0], m.lens[1] = -1, 0
        m.free(range(2, 65))
        d.free(range(2, 65))
        assert d.status() == 0


def test_binding_on_the_device(mla):
    """Shapes, types and numbers that the compiled binding refuses with tensors on the device."""
    m, d, _ = both(mla, 10, 3, 4)
    rows = d._list([0])
    for wrong in (d.refs[::2], d.refs.float(), d.refs[None]):
        with pytest.raises((TypeError, ValueError)):
            mla.pages_free(wrong, d.table, d.lens, rows, d.ws)
    with pytest.raises(ValueError):
        mla.pages_extend(d.refs, d.table, d.lens, rows, d._list([1, 2]), d.ws)
    with pytest.raises(ValueError):
        mla.pages_extend(d.refs, d.table.t(), d.lens, rows, d._list([1]), d.ws)
    with pytest.raises(ValueError, match="pools"):
        mla.pages_compact(d.refs, d.table, d.lens, [d.pools[0][:, :9]], workspace=d.ws)
    with pytest.raises(ValueError, match="pools"):
        mla.pages_fork(d.refs, d.table, d.lens, rows, rows, [d.pools[0].transpose(1, 2)], d.ws)
    with pytest.raises(mla.MLAError):
        mla.pages_free(d.refs, d.table, d.lens, rows, d.ws[:256])
    assert d.status() == 0
    same(m, d)
    # an empty list of pools, and streams by object
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mla.pages_extend(d.refs, d.table, d.lens, rows, d._list([70]), d.ws, stream=s)
    mla.pages_compact(d.refs, d.table, d.lens, (), workspace=d.ws, stream=s)
    s.synchronize()
    m.extend([0], [70])
    assert d.status() == 0
    same(m, d)


@pytest.mark.parametrize("n", [1, 2, 31, 33, 64, 65, 1023, 1025, 2048, 2050, 4095, 4096])
def test_list_lengths(mla, n):
    """Lists of every shape of the plan, rows named twice among them, with rows up to the last that
    there can be and more pages wanted than there are."""
    rng = np.random.default_rng(n)
    rows = 1 << 20 if n in (33, 4096) else 5000
    pages = 3 * n // 2 + 1
    m = Model(pages, rows, 2, [np.arange(8 * pages).astype(np.int16).reshape(1, pages, 8)])
    d = Device(mla, m)
    pick = rng.permutation(rows)[:n]
    pick[n // 2] = rows - 1
    if n > 3:
        pick[n // 3] = pick[n // 5]
        pick[-1] = rows - 1  # index 4095 and row 2^20 - 1 in the longest
    lens = rng.integers(0, 129, n)
    m.extend(pick.tolist(), lens.tolist())
    d.extend(pick.tolist(), lens.tolist())
    assert d.status() in (0, OUT_OF_RANGE, NO_PAGES)
    same(m, d)
    # the last row alone at the last index
    if n == 4096:
        m.free([rows - 1])
        d.free([rows - 1])
        order = [0] * 4095 + [rows - 1]
        m.extend(order, [m.lens[0]] * 4095 + [1])
        d.extend(order, [int(m.lens[0])] * 4095 + [1])
        d.status()
        same(m, d)
        assert m.lens[rows - 1] == 1
    full = [int(r) for r in pick if m.lens[r]][: max(1, n // 4)]
    empty = [int(r) for r in range(rows - 2, -1, -1) if not m.lens[r]][: len(full)]
    m.fork(full[:len(empty)], empty)
    d.fork(full[:len(empty)], empty)
    assert d.status() in (0, NO_PAGES)
    same(m, d)


def test_extend_past_the_first_pass(mla):
    """The free pages lie behind the first 16384, in several passes of the scan."""
    pages, most = 60000, 12000
    m = Model(pages, 6, most, [np.zeros((1, pages, 8), np.int16)])
    held = np.r_[0:16300, 16390:30000]
    for r, ids in enumerate(np.array_split(held, 3)):
        m.table[r, :len(ids)] = ids
        m.lens[r] = PAGE * len(ids)
        m.refs[ids] += 1
    d = Device(mla, m)
    for rows, lens in (([3, 4], [PAGE * 60, PAGE * 11000 - 1]), ([5], [PAGE * 12000]), ([3], [PAGE * 12000])):
        m.extend(rows, lens)
        d.extend(rows, lens)
        assert d.status() in (0, NO_PAGES)
        same(m, d)
