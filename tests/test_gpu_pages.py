"""GPU: page bookkeeping of the paged cache (rq_pages_*) against a plain Python model.

The model states rq.h's rules one entry at a time; tables, counts, pool bytes
and status words have to be equal."""
import numpy as np
import pytest
import torch

from rq_harness import Case, GpuCache, rotation32

pytestmark = pytest.mark.gpu


class Model:
    """pool [planes, pages, bytes], table [rows, tiles], refs [pages] as rq.h describes them."""

    def __init__(self, pool, table, refs, nmax):
        self.pool, self.table, self.refs, self.nmax = pool, table, refs, nmax
        self.status = [0, 0, 0, 0]

    @property
    def pages(self):
        return len(self.refs)

    def named(self, e):
        return 0 <= e < self.pages

    def copy(self, src, dst):
        n, old = len(src), self.pool.copy()
        for i in range(n):
            bad = not (self.named(src[i]) and self.named(dst[i]))
            bad |= any(j != i and src[j] == dst[i] for j in range(n)) or any(dst[j] == dst[i] for j in range(i))
            if bad:
                self.status[2] = 1
            else:
                self.pool[:, dst[i]] = old[:, src[i]]

    def fork(self, src, dst):
        rows, old = len(self.table), self.table.copy()
        ok = [0 <= s < rows and 0 <= t < rows for s, t in zip(src, dst)]
        if not all(ok):
            self.status[1] = 1
        target = {t: s for s, t, o in zip(src, dst, ok) if o}
        for t, s in target.items():
            for col in range(old.shape[1]):
                if self.named(old[s, col]):
                    self.refs[old[s, col]] += 1
                if self.named(old[t, col]):
                    self.refs[old[t, col]] -= 1
            self.table[t] = old[s]

    def free(self, rows, keep):
        for r, k in zip(rows, keep if keep is not None else [0] * len(rows)):
            if not 0 <= r < len(self.table):
                self.status[1] = 1
                continue
            for col in range(-(-max(k, 0) // 64), self.table.shape[1]):
                if self.named(self.table[r, col]):
                    self.refs[self.table[r, col]] -= 1
                self.table[r, col] = -1

    def reserve(self, lens, n):
        """One request after the other, each taking the lowest page that was free when the call began."""
        free = [p for p in range(self.pages) if self.refs[p] <= 0]
        for b, ln in enumerate(lens):
            if ln < 0 or ln + n > self.nmax:
                self.status[1] = 1
                continue
            for t in range(ln // 64, (ln + n - 1) // 64 + 1):
                e = self.table[b, t]
                shared = self.named(e) and self.refs[e] > 1
                if self.named(e) and not shared:
                    continue
                if not free:
                    self.status[3] = 1
                    continue
                p = free.pop(0)
                if shared:
                    if t == ln // 64 and ln % 64:
                        self.pool[:, p] = self.pool[:, e]
                    self.refs[e] -= 1
                self.table[b, t], self.refs[p] = p, 1

    def compact(self):
        used = int((self.refs > 0).sum())
        holes = [p for p in range(used) if not self.refs[p] > 0]
        high = [p for p in range(used, self.pages) if self.refs[p] > 0]
        to = {s: t for s, t in zip(high, holes)}
        for s, t in to.items():
            self.pool[:, t] = self.pool[:, s]
            self.refs[t], self.refs[s] = self.refs[s], 0
        self.table[:] = np.vectorize(lambda e: to.get(int(e), e))(self.table)
        return used


class Paged:
    def __init__(self, L=2, G=1, H=2, d=128, g=32, P=2, rows=6, tiles=4, extra=1, pages=40, seed=0):
        import decode_attention_rq_gb300 as rq
        self.rq = rq
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.nmax = tiles * 64 - 10
        self.cfg = rq.rq_config(L, P, G, H, d, g, rows, self.nmax, rq.RQ_MODE_SHARED, 0)
        nbytes = rq.rq_cache_paged_bytes(self.cfg, pages)
        self.pool = torch.from_numpy(rng.integers(0, 256, (L * G, pages, nbytes // (L * G * pages)), dtype=np.uint8)).cuda()
        self.table = torch.full((rows, tiles + extra), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.used = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.R = torch.eye(d, device="cuda")
        self.handle = rq.rq_cache_create_paged(self.cfg, pages, self.pool, nbytes, self.table, tiles + extra, self.R)
        self.ws = torch.full((rq.rq_pages_workspace_bytes(self.cfg, pages),), 0xCD, dtype=torch.uint8, device="cuda")
        self.rows, self.tiles, self.pages = rows, tiles, pages

    def fill(self, share=0.4, hole=0.2):
        """Random table: some entries shared, some without a page, counts to match."""
        order = list(self.rng.permutation(self.pages)[: self.pages * 2 // 3])
        t = np.full((self.rows, self.table.shape[1]), -1, dtype=np.int32)
        given = []
        for r in range(self.rows):
            for c in range(self.tiles):
                x = self.rng.random()
                if x < hole or (not order and not given):
                    continue
                if x < hole + share and given or not order:
                    t[r, c] = given[int(self.rng.integers(len(given)))]
                else:
                    t[r, c] = order.pop()
                    given.append(t[r, c])
        self.set(t)
        return self

    def set(self, t):
        self.table.copy_(torch.from_numpy(np.ascontiguousarray(t, dtype=np.int32)))
        refs = np.zeros(self.pages, dtype=np.int32)
        for e in t.flatten():
            if 0 <= e < self.pages:
                refs[e] += 1
        self.refs.copy_(torch.from_numpy(refs))

    def model(self):
        torch.cuda.synchronize()
        return Model(self.pool.cpu().numpy().copy(), self.table.cpu().numpy().copy(), self.refs.cpu().numpy().copy(),
                     self.nmax)

    def same(self, m):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), m.table)
        assert np.array_equal(self.refs.cpu().numpy(), m.refs)
        assert self.status.tolist() == m.status
        assert np.array_equal(self.pool.cpu().numpy(), m.pool)

    def ints(self, x):
        return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")

    def reserve(self, lens, n):
        self.rq.rq_pages_reserve(self.handle, len(lens), self.ints(lens), n, self.refs, self.status, self.ws,
                                 self.ws.numel())

    def compact(self):
        self.rq.rq_pages_compact(self.handle, self.refs, self.used, self.status, self.ws, self.ws.numel())

    def close(self):
        self.rq.rq_cache_destroy(self.handle)


@pytest.mark.parametrize("seed,kw", [(0, {}), (1, dict(L=3, G=2, H=5, d=96, P=4)), (2, dict(H=1, P=1, g=16)),
                                     (3, dict(L=1, H=16, P=4, pages=12))])
def test_copy(seed, kw):
    p = Paged(seed=seed, **kw)
    order = p.rng.permutation(p.pages)
    n = p.pages // 3
    m = p.model()
    src, dst = order[:n], order[n:2 * n]
    p.rq.rq_pages_copy(p.handle, n, p.ints(src), p.ints(dst), p.status)
    m.copy(src, dst)
    p.same(m)
    p.close()


def test_copy_skips_what_collides():
    """Pages outside the pool, a target that is a source, a target named twice, a page onto itself."""
    p = Paged(seed=4)
    src = [0, 1, 2, 3, 4, -1, 6, p.pages, 8, 9]
    dst = [20, 0, 21, 21, p.pages + 3, 22, -5, 23, 8, 24]
    m = p.model()
    p.rq.rq_pages_copy(p.handle, len(src), p.ints(src), p.ints(dst), p.status)
    m.copy(src, dst)
    p.same(m)
    assert p.status.tolist() == [0, 0, 1, 0]
    p.close()


@pytest.mark.parametrize("seed,rows,tiles,extra", [(0, 6, 4, 1), (1, 33, 40, 0), (2, 200, 70, 3), (3, 1, 1, 0)])
def test_fork_is_a_simultaneous_assignment(seed, rows, tiles, extra):
    p = Paged(L=1, H=1, P=1, rows=rows, tiles=tiles, extra=extra, pages=rows * tiles + 7, seed=seed).fill()
    m = p.model()
    src, dst = p.rng.integers(0, rows, rows), p.rng.permutation(rows)
    p.rq.rq_pages_fork(p.handle, rows, p.ints(src), p.ints(dst), p.refs, p.status)
    m.fork(src, dst)
    p.same(m)
    # a target twice (the last pair counts), a row onto itself, rows out of range
    if rows >= 6:
        src, dst = [0, 1, 2, 3, rows, -1], [5, 5, 2, 4, 1, 3]
        p.rq.rq_pages_fork(p.handle, 6, p.ints(src), p.ints(dst), p.refs, p.status)
        m.fork(src, dst)
        p.same(m)
    p.close()


def test_fork_more_pairs_than_full_columns_hold():
    """Above 1440 pairs the columns of a CTA no longer fit 32 wide; 6145 pairs are refused."""
    p = Paged(L=1, H=1, P=1, rows=6145, tiles=3, extra=0, pages=100, seed=7)
    t = p.rng.integers(-1, 100, (6145, 3))
    p.set(t)
    for n in (1500, 3100, 6144):
        m = p.model()
        src, dst = p.rng.integers(0, 6145, n), p.rng.permutation(6145)[:n]
        p.rq.rq_pages_fork(p.handle, n, p.ints(src), p.ints(dst), p.refs, p.status)
        m.fork(src, dst)
        p.same(m)
    with pytest.raises(p.rq.RqError) as e:
        p.rq.rq_pages_fork(p.handle, 6145, p.ints(range(6145)), p.ints(range(6145)), p.refs, p.status)
    assert e.value.status == 6
    p.close()


@pytest.mark.parametrize("seed", [0, 1])
def test_free(seed):
    p = Paged(rows=20, tiles=9, pages=120, L=1, H=1, seed=seed).fill()
    m = p.model()
    rows = [3, 7, 3, 0, 19, -1, 20]
    keep = [130, 0, 64, 1, 9 * 64, 5, 5]
    p.rq.rq_pages_free(p.handle, len(rows), p.ints(rows), p.ints(keep), p.refs, p.status)
    m.free(rows, keep)
    p.same(m)
    assert p.status.tolist() == [0, 1, 0, 0]
    p.rq.rq_pages_free(p.handle, 20, p.ints(range(20)), None, p.refs, p.status)
    m.free(list(range(20)), None)
    p.same(m)
    assert int(p.refs.abs().sum()) == 0 and int((p.table + 1).abs().sum()) == 0
    p.close()


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("n", [1, 40, 64, 129])
def test_reserve(seed, n):
    p = Paged(seed=seed, rows=9, tiles=5, pages=60).fill()
    m = p.model()
    lens = [int(x) for x in p.rng.integers(0, p.nmax - n + 1, 9)]
    lens[0], lens[1], lens[2] = 0, 64, p.nmax - n
    lens[3], lens[4] = -1, p.nmax - n + 1           # skipped
    p.reserve(lens, n)
    m.reserve(lens, n)
    p.same(m)
    p.close()


def test_reserve_last_holder_keeps_the_page_and_the_pool_may_run_out():
    p = Paged(L=2, rows=8, tiles=2, pages=9)
    t = np.full((8, 3), -1)
    t[:4, 0], t[4:, 0] = 5, 2
    p.set(t)
    m = p.model()
    lens = [10] * 8
    p.reserve(lens, 1)                              # rows 0-2 and 4-6 want copies: six of seven free pages
    m.reserve(lens, 1)
    p.same(m)
    assert int(p.table[3, 0]) == 5 and int(p.table[7, 0]) == 2 and p.status.tolist() == [0, 0, 0, 0]
    p.reserve([64] * 8, 1)                          # one page left for eight rows
    m.reserve([64] * 8, 1)
    p.same(m)
    assert p.status.tolist() == [0, 0, 0, 1]
    p.close()


def test_reserve_many_slots():
    """More requests than one pass of the planning block takes, and a pool larger than it."""
    p = Paged(L=1, H=1, P=1, rows=300, tiles=9, extra=0, pages=5000, seed=3)
    t = np.full((300, 9), -1)
    for r in range(300):
        t[r, : r % 9] = p.rng.integers(0, 900, r % 9)
    p.set(t)
    lens = [int(x) for x in p.rng.integers(0, 200, 300)]
    m = p.model()
    p.reserve(lens, 300)
    m.reserve(lens, 300)
    p.same(m)
    p.close()


@pytest.mark.parametrize("seed,kw", [(0, {}), (1, dict(L=3, G=2, H=3, d=96, P=4)), (2, dict(rows=30, tiles=9, pages=2100, L=1, H=1, P=1)),
                                     (3, dict(pages=32)), (4, dict(pages=33))])
def test_compact(seed, kw):
    p = Paged(seed=seed, **kw).fill()
    m = p.model()
    p.compact()
    used = m.compact()
    p.same(m)
    assert int(p.used[0]) == used
    p.compact()                                     # nothing left to move
    assert m.compact() == used
    p.same(m)
    p.rq.rq_pages_free(p.handle, p.rows, p.ints(range(p.rows)), None, p.refs, p.status)
    m.free(list(range(p.rows)), None)
    p.compact()                                     # an empty pool
    assert m.compact() == 0 and p.used.tolist()[0] == 0
    p.same(m)
    p.close()


def test_captured_and_replayed():
    """reserve and compact inside one graph: the planned lists are made anew at every replay."""
    p = Paged(seed=8, rows=6, tiles=4, pages=40).fill()
    t0, r0, pool0 = p.table.clone(), p.refs.clone(), p.pool.clone()
    lens = p.ints([70, 5, 130, 64, 0, 200])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            p.rq.rq_pages_reserve(p.handle, 6, lens, 3, p.refs, p.status, p.ws, p.ws.numel())
            p.rq.rq_pages_compact(p.handle, p.refs, p.used, p.status, p.ws, p.ws.numel())
    for shift in (0, 30):
        p.table.copy_(t0); p.refs.copy_(r0); p.pool.copy_(pool0)
        lens.copy_(p.ints([70 - shift, 5, 130, 64, shift, 200]))
        m = p.model()
        graph.replay()
        m.reserve([70 - shift, 5, 130, 64, shift, 200], 3)
        m.compact()
        p.same(m)
    p.close()


def test_refusals():
    p = Paged(pages=10)
    rq, E = p.rq, p.rq.RqError
    one = p.ints([0] * 8)

    def fails(status, f, *a):
        with pytest.raises(E) as e:
            f(*a)
        assert e.value.status == status, e.value

    fails(3, rq.rq_pages_copy, p.handle, 11, p.ints([0] * 11), p.ints([0] * 11), p.status)
    fails(1, rq.rq_pages_copy, p.handle, -1, one, one, p.status)
    fails(1, rq.rq_pages_copy, p.handle, 9, one, one, p.status)                 # lists too short
    fails(1, rq.rq_pages_copy, p.handle, 1, one.cpu(), one, p.status)
    fails(1, rq.rq_pages_copy, p.handle, 1, one.long(), one, p.status)
    fails(2, rq.rq_pages_copy, p.handle, 1, one[1:], one, p.status)             # alignment
    fails(3, rq.rq_pages_fork, p.handle, 7, one, one, p.refs, p.status)
    fails(1, rq.rq_pages_fork, p.handle, 1, one, None, p.refs, p.status)
    fails(3, rq.rq_pages_free, p.handle, 7, one, one, p.refs, p.status)
    fails(3, rq.rq_pages_reserve, p.handle, 7, one, 1, p.refs, p.status, p.ws, p.ws.numel())
    fails(3, rq.rq_pages_reserve, p.handle, 6, one, p.nmax + 1, p.refs, p.status, p.ws, p.ws.numel())
    fails(1, rq.rq_pages_reserve, p.handle, 0, one, 1, p.refs, p.status, p.ws, p.ws.numel())
    fails(4, rq.rq_pages_reserve, p.handle, 6, one, 1, p.refs, p.status, p.ws, p.ws.numel() - 1)
    fails(4, rq.rq_pages_compact, p.handle, p.refs, p.used, p.status, p.ws, 16)
    m = p.model()
    for call in (lambda: rq.rq_pages_copy(p.handle, 0, one, one, None),
                 lambda: rq.rq_pages_fork(p.handle, 0, one, one, p.refs, None),
                 lambda: rq.rq_pages_free(p.handle, 0, one, None, p.refs, None),
                 lambda: rq.rq_pages_reserve(p.handle, 6, one, 0, p.refs, None, p.ws, p.ws.numel())):
        call()
    p.same(m)
    plain = GpuCache(Case(), rotation32(128)[0])                                # a contiguous cache has no pages
    fails(1, rq.rq_pages_copy, plain.handle, 1, one, one, p.status)
    fails(1, rq.rq_pages_fork, plain.handle, 1, one, one, p.refs, p.status)
    fails(1, rq.rq_pages_free, plain.handle, 1, one, None, p.refs, p.status)
    fails(1, rq.rq_pages_reserve, plain.handle, 1, one, 1, p.refs, p.status, p.ws, p.ws.numel())
    fails(1, rq.rq_pages_compact, plain.handle, p.refs, p.used, p.status, p.ws, p.ws.numel())
    plain.close()
    p.close()
