"""Pages of a cache on the GPU against a model of lists: copying, forking, freeing and compacting, their
refusals, and all of them around the recurrent step."""
import random

import pytest
import torch

import kda_linear_attention_02_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def ints(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def status():
    torch.cuda.synchronize()
    return kda.kda_get_device_status()


def rand_pages(*shape, dtype=torch.int32, seed=0):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return torch.randint(-(1 << 31), 1 << 31, shape, generator=g, device=DEV, dtype=torch.int64).to(torch.int32).view(dtype)


# ------------------------------------------------------------------------------------------------ copy


@pytest.mark.parametrize("words", [4, 12, 8192, 8196, 30000])       # 16 bytes to several blocks a page
@pytest.mark.parametrize("n", [1, 37, 700])
def test_copy_between_pools(words, n):
    r = random.Random(words * 1000 + n)
    src, dst = rand_pages(n + 2, words, seed=1), rand_pages(n + 9, words, seed=2)
    s, d = [r.randrange(n + 2) for _ in range(n)], r.sample(range(n + 9), n)
    if n > 1:
        s[n // 2], d[n // 3] = -1, -5                               # left out
    want = dst.clone()
    for i in range(n):
        if s[i] >= 0 and d[i] >= 0:
            want[d[i]] = src[s[i]]
    kda.kda_pages_copy(dst, src, ints(d), ints(s))
    assert status() == 0
    assert torch.equal(dst, want)


def test_copy_with_one_table():
    src, dst = rand_pages(9, 40, seed=1), rand_pages(20, 40, seed=2)
    want = dst.clone()
    want[:9] = src
    kda.kda_pages_copy(dst, src)
    assert torch.equal(dst, want)
    pick = [3, 3, 0, 8]
    kda.kda_pages_copy(dst, src, src_pages=ints(pick))
    want[:4] = src[pick]
    assert torch.equal(dst, want)
    kda.kda_pages_copy(dst, src, dst_pages=ints([19, 2]))
    want[19], want[2] = src[0], src[1]
    assert status() == 0 and torch.equal(dst, want)


@pytest.mark.parametrize("n", [16, 3000])
def test_copy_within_a_pool_and_its_conflicts(n):
    # forks of page 0 (fine), a page onto itself (nothing), a chain, a swap and a doubled destination (left out)
    pool = rand_pages(2 * n + 20, 8, seed=3)
    base = list(range(n, 2 * n))
    s, d = [0] * n, base[:]
    extra = [(1, 1), (2, 3), (3, 4), (5, 6), (6, 5), (7, 2 * n), (8, 2 * n), (9, 2 * n + 1), (2 * n + 30, 10), (10, 2 * n + 20)]
    s, d = s + [a for a, _ in extra], d + [b for _, b in extra]
    want = pool.clone()
    want[base] = pool[0]
    want[2 * n + 1] = pool[9]
    order = list(range(len(s)))
    random.Random(n).shuffle(order)
    kda.kda_pages_copy(pool, pool, ints([d[i] for i in order]), ints([s[i] for i in order]))
    assert status() == -7
    assert torch.equal(pool, want)


def test_copy_doubled_destinations_with_a_valid_rest():
    src, dst = rand_pages(2000, 4, seed=4), rand_pages(2000, 4, seed=5)
    d = list(range(2000))
    d[1999] = d[3]
    want = src.clone()
    want[3], want[1999] = dst[3], dst[1999]
    kda.kda_pages_copy(dst, src, ints(d))
    assert status() == -7 and torch.equal(dst, want)


@pytest.mark.slow
def test_copy_beyond_32_bit_offsets():
    pool = torch.zeros(5000, 1 << 18, dtype=I32, device=DEV)        # 5.2 GB
    pool[1] = rand_pages(1 << 18, seed=6)
    kda.kda_pages_copy(pool, pool, ints([4999, 4098]), ints([1, 1]))
    assert status() == 0
    assert torch.equal(pool[4999], pool[1]) and torch.equal(pool[4098], pool[1]) and not pool[4097].any()


# ------------------------------------------------------------------------------- the model of a cache


class Model:
    """Rows of pages in lists, and the pages' contents."""

    def __init__(self, pool, n_rows, max_pages):
        self.pool, self.refs, self.rows, self.most = pool.clone(), [0] * pool.shape[1], [[] for _ in range(n_rows)], max_pages

    def fork(self, parents, children, shared, fresh, zero=False):
        free = iter([p for p, r in enumerate(self.refs) if r == 0])
        have = [len(r) for r in self.rows]
        for p, c, k, f in zip(parents, children, shared, fresh):
            if p != c and p >= 0:
                for j in range(have[p]):
                    page = self.rows[p][j]
                    if j >= k:
                        new = next(free)
                        self.pool[:, new] = self.pool[:, page]
                        page = new
                    self.rows[c].append(page)
                    self.refs[page] += 1
            for _ in range(f):
                page = next(free)
                if zero:
                    self.pool[:, page] = 0
                self.rows[c].append(page)
                self.refs[page] += 1

    def free(self, rows):
        for r in rows:
            for p in self.rows[r]:
                self.refs[p] -= 1
            self.rows[r] = []

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r]
        m = len(live)
        to = {p: p for p in live if p < m}
        for hole, p in zip([p for p in range(m) if not self.refs[p]], [p for p in live if p >= m]):
            to[p] = hole
            self.pool[:, hole] = self.pool[:, p]
        refs = [0] * len(self.refs)
        for p in live:
            refs[to[p]] = self.refs[p]
        self.refs, self.rows = refs, [[to[p] for p in r] for r in self.rows]
        return [to.get(p, -1) for p in range(len(refs))], m


class Cache:
    def __init__(self, pool, n_rows, max_pages):
        self.pool = pool
        self.refs = torch.zeros(pool.shape[1], dtype=I32, device=DEV)
        self.table = torch.full((n_rows, max_pages), -99, dtype=I32, device=DEV)
        self.counts = torch.zeros(n_rows, dtype=I32, device=DEV)

    def fork(self, parents, children, shared=None, fresh=None, zero=False):
        kda.kda_pages_fork(self.pool, self.refs, self.table, self.counts, ints(parents), ints(children),
                           None if shared is None else ints(shared), None if fresh is None else ints(fresh), zero_fresh=zero)

    def free(self, rows):
        kda.kda_pages_free(self.refs, self.table, self.counts, ints(rows))

    def compact(self):
        n_live = torch.full((1,), -1, dtype=I32, device=DEV)
        remap = kda.kda_pages_compact(self.pool, self.refs, self.table, self.counts, n_live=n_live)
        return remap.tolist(), int(n_live)

    def assert_like(self, m):
        assert status() == 0
        assert self.refs.tolist() == m.refs
        assert self.counts.tolist() == [len(r) for r in m.rows]
        for got, want in zip(self.table.tolist(), m.rows):
            assert got[:len(want)] == want
        assert torch.equal(self.pool, m.pool)

    def snapshot(self):
        return [x.clone() for x in (self.pool, self.refs, self.table, self.counts)]


@pytest.mark.parametrize("planes,words,n_pages,n_rows,most,seed", [
    (1, 4, 50, 12, 6, 0), (3, 8, 6000, 40, 70, 1), (2, 9000, 90, 20, 7, 2), (1, 4, 9001, 1500, 5, 3)])
def test_random_life_of_a_cache(planes, words, n_pages, n_rows, most, seed):
    r = random.Random(seed)
    pool = rand_pages(planes, n_pages, words, seed=seed)
    c, m = Cache(pool, n_rows, most), Model(pool, n_rows, most)
    for turn in range(14):
        empty = [i for i in range(n_rows) if not m.rows[i]]
        full = [i for i in range(n_rows) if m.rows[i]]
        r.shuffle(empty)
        r.shuffle(full)
        kind = turn % 3 if full else 0
        if kind == 0:    # open fresh rows, extend some, fork others
            ext, parents = full[:len(full) // 3], full[len(full) // 3:]
            entries, room = [], sum(1 for x in m.refs if x == 0)
            for child in empty[:max(1, len(empty) // 2)]:
                p = r.choice(parents + [-1]) if parents else -1
                have = len(m.rows[p]) if p >= 0 else 0
                k = r.randint(0, have)
                entries.append((p, child, k, r.randint(0, most - have)))
            entries += [(x, x, r.randint(-3, 9), r.randint(0, most - len(m.rows[x]))) for x in ext]
            r.shuffle(entries)
            kept = []
            for e in entries:
                need = e[3] + (len(m.rows[e[0]]) - e[2] if e[0] >= 0 and e[0] != e[1] else 0)
                if need <= room:
                    room -= need
                    kept.append(e)
            if not kept:
                continue
            zero = r.random() < 0.5
            args = [list(x) for x in zip(*kept)]
            c.fork(*args, zero=zero)
            m.fork(*args, zero=zero)
        elif kind == 1:
            gone = full[:len(full) // 2] or full
            c.free(gone + gone[:2])      # a row named twice is freed once
            m.free(gone)
        else:
            assert c.compact() == m.compact()
        c.assert_like(m)


def filled(n_pages=12, n_rows=6, most=3):
    pool = rand_pages(1, n_pages, 4, seed=7)
    c = Cache(pool, n_rows, most)
    c.fork([-1, -1], [0, 1], fresh=[2, 3])
    assert status() == 0
    return c


@pytest.mark.parametrize("entries", [
    ([0, 0], [2, 2], [0, 0], [0, 0]),       # a row opened twice
    ([0], [1], [0], [0]),                   # a child that is not empty
    ([0, 2], [2, 3], [0, 0], [0, 0]),       # a row opened and continued at once
    ([0, 0], [0, 2], [0, 0], [1, 0]),       # a row extended and continued at once
    ([0, 0], [0, 0], [0, 0], [1, 0]),       # extended twice
    ([0, -2], [2, 3], [0, 0], [0, 0]), ([6], [2], [0], [0]), ([0], [6], [0], [0]), ([0], [-1], [0], [0]),
    ([0], [2], [3], [0]), ([0], [2], [-1], [0]), ([0], [2], [0], [2]), ([-1], [2], [0], [-1]), ([-1], [2], [0], [4])])
def test_fork_refuses_the_whole_call(entries):
    c = filled()
    before = c.snapshot()
    parents, children, shared, fresh = entries
    c.fork(parents + [-1], children + [5], shared + [0], fresh + [1])
    assert status() == -7
    assert all(torch.equal(a, b) for a, b in zip(before, c.snapshot()))


def test_fork_without_enough_pages_changes_nothing():
    c = filled()
    before = c.snapshot()
    c.fork([1, 1, -1], [2, 3, 4], fresh=[0, 0, 2])       # 8 pages of the 7 that are free
    assert status() == -8
    assert all(torch.equal(a, b) for a, b in zip(before, c.snapshot()))
    c.fork([1, 1, -1], [2, 3, 4], fresh=[0, 0, 1])
    assert status() == 0 and int((c.refs == 0).sum()) == 0


def test_corrupt_tables_are_reported_and_stay_in_bounds():
    c = filled()
    c.table[0, 1] = 12                                    # behind the pool
    before = c.snapshot()
    c.fork([0], [2])
    assert status() == -7 and all(torch.equal(a, b) for a, b in zip(before, c.snapshot()))
    c.compact()
    assert status() == -7 and c.table[0].tolist()[1] == 12
    c.free([0, 6, -1])
    assert status() == -7 and c.counts.tolist()[:2] == [0, 3]
    c.counts[1] = 4                                       # more than a row holds
    c.free([1])
    assert status() == -7


@pytest.mark.parametrize("n_rows", [150_000, 260_000, 400_000, 1 << 20])
def test_fork_with_many_rows(n_rows):
    # a bit for each row in the planning block's shared memory: below and above the default limit, and the most
    pool = rand_pages(1, 4000, 4, seed=11)
    c = Cache(pool, n_rows, 2)
    rows = list(range(0, n_rows, n_rows // 1500))[:1500] + [n_rows - 1]      # more entries than one round takes
    c.fork([-1] * len(rows), rows, fresh=[1] * len(rows))
    assert status() == 0
    assert c.table[rows, 0].tolist() == list(range(len(rows))) and int(c.counts.sum()) == len(rows)
    c.fork([n_rows - 1, -1], [1, n_rows - 1], fresh=[0, 1])                  # opened and continued at once
    assert status() == -7 and int(c.counts.sum()) == len(rows)
    c.fork([n_rows - 1], [1], shared=[1])
    assert status() == 0 and c.table[1, 0] == c.table[n_rows - 1, 0]


def test_compact_of_full_and_empty_caches():
    for fresh in ([3, 3, 3, 3], [0, 0, 0, 0]):
        pool = rand_pages(2, 12, 4, seed=9)
        c, m = Cache(pool, 4, 3), Model(pool, 4, 3)
        args = [-1] * 4, [0, 1, 2, 3], [0] * 4, fresh
        c.fork(*args)
        m.fork(*args)
        assert c.compact() == m.compact()
        c.assert_like(m)


def test_pages_calls_in_a_graph_on_another_stream():
    pool = rand_pages(2, 40, 64, seed=10)
    c, m = Cache(pool, 8, 4), Model(pool, 8, 4)
    c.fork([-1] * 3, [0, 1, 2], fresh=[4, 2, 3])
    m.fork([-1] * 3, [0, 1, 2], [0] * 3, [4, 2, 3])
    args = [ints(x) for x in ([0, 0, 2], [5, 6, 7], [3, 0, 1], [1, 2, 4])]
    n_live, remap = ints([0]), torch.empty(40, dtype=I32, device=DEV)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kda.kda_pages_fork(c.pool, c.refs, c.table, c.counts, args[0][:2].contiguous(), args[1][:2].contiguous(),
                           args[2][:2].contiguous())
        kda.kda_pages_free(c.refs, c.table, c.counts, args[0][:1].contiguous())
        kda.kda_pages_compact(c.pool, c.refs, c.table, c.counts, remap=remap, n_live=n_live)
    g.replay()
    m.fork([0, 0], [5, 6], [3, 0], [0, 0])
    m.free([0])
    want = m.compact()
    c.assert_like(m)
    assert (remap.tolist(), int(n_live)) == want


def test_states_forked_stepped_freed_and_compacted():
    # parallel sampling from one prompt: the prompt's state enters the pool, three children continue it with
    # tokens of their own, one ends, the pool is compacted, the others go on
    H, d = 2, 64
    g = torch.Generator(DEV)
    g.manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    T = 100
    q, k, v, la = 0.1 * r(T, H, d), 0.1 * r(T, H, d), r(T, H, d), -0.1 * r(T, H).abs()
    o, fs = torch.empty(T, H, d, device=DEV), torch.empty(1, H, d, d, device=DEV)
    kda.kda_lin_chunk_fwd(q, k, v, la, None, ints([0, T]), o, fs)
    c = Cache(r(1, 9, H, d, d), 5, 1)
    c.fork([-1, -1], [4, 0], fresh=[1, 1])                                # row 4 takes page 0, the prompt's row 0 page 1
    kda.kda_pages_copy(c.pool[0], fs, c.table[0], None)
    c.fork([0, 0, 0], [1, 2, 3])
    c.free([0, 4])
    want = fs[0].clone().expand(4, H, d, d).clone()
    alive = [1, 2, 3]
    for turn in range(6):
        q1, k1, v1, la1 = 0.1 * r(4, H, d), 0.1 * r(4, H, d), r(4, H, d), -0.1 * r(4, H).abs()
        slots = torch.where(c.counts[:4] > 0, c.table[:4, 0], -1)
        o1 = torch.zeros(4, H, d, device=DEV)
        kda.kda_lin_recurrent_step(c.pool[0], q1, k1, v1, la1, o1, slots=slots)
        want = want * la1.exp()[:, :, None, None] + k1[..., None] * v1[:, :, None, :]
        ow = torch.einsum("nhd,nhde->nhe", q1, want)
        assert torch.allclose(o1[alive], ow[alive], rtol=1e-4, atol=1e-4) and not o1[0].any()
        if turn == 2:
            c.free([2])
            alive = [1, 3]
            remap, n_live = c.compact()
            assert n_live == 2 and sorted(c.table[[1, 3], 0].tolist()) == [0, 1]
        assert status() == 0
    for i in alive:
        assert torch.allclose(c.pool[0, int(c.table[i, 0])], want[i], rtol=1e-4, atol=1e-5)
