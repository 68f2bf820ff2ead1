"""The page pool against a model that does what a call's list says, entry by entry: tables, counts, free pages, bytes."""
import numpy as np
import pytest

from tests import kv_plain as P
from tests.test_gpu_kv import dev, ok_status

pytestmark = pytest.mark.gpu

SHAPES = [("q8_0", 4, 128), ("q8_0", 3, 64), ("f16", 2, 128), ("f16", 5, 64)]


class Model:
    def __init__(self, n_pages, n_seqs, ld, ctype, Hkv, D, rng):
        self.ctype, self.Hkv, self.D, self.ld = ctype, Hkv, D, ld
        self.pages = rng.integers(0, 256, (n_pages, Hkv, P.block_bytes(ctype, D)), dtype=np.uint8)
        self.table = np.full((n_seqs, ld), -1, np.int32)
        self.refs, self.seq_pages = np.zeros(n_pages, np.int32), np.zeros(n_seqs, np.int32)
        self.free = list(rng.permutation(n_pages))

    def take(self):
        page = self.free.pop()
        self.refs[page] = 1
        return page

    def grow(self, lens):
        need = [max(0, -(-n // 64) - k) for n, k in zip(lens, self.seq_pages)]
        if sum(need) > len(self.free):
            return False
        for s, k in enumerate(need):
            for _ in range(k):
                self.table[s, self.seq_pages[s]] = self.take()
                self.seq_pages[s] += 1
        return True

    def rows(self, rest):
        """Bytes of a block that its first `rest` tokens hold."""
        at, voff, sc, soff = P.places(self.ctype, self.D)
        if self.ctype == "f16":
            b = np.concatenate([at[:rest].ravel(), at[:rest].ravel() + 1])
            return np.concatenate([b, b + voff])
        s = np.concatenate([sc[:rest].ravel(), sc[:rest].ravel() + 1])
        return np.concatenate([at[:rest].ravel(), at[:rest].ravel() + voff, s, s + soff])

    def fork(self, src, dst, lens):
        if sum(n % 64 != 0 for n in lens) > len(self.free):
            return False
        for s, d, n in zip(src, dst, lens):
            full, rest = n // 64, n % 64
            self.table[d, :full] = self.table[s, :full]
            np.add.at(self.refs, self.table[s, :full], 1)
            if rest:
                page = self.take()
                self.table[d, full] = page
                b = self.rows(rest)
                self.pages[page][:, b] = self.pages[self.table[s, full]][:, b]
            self.seq_pages[d] = full + (rest != 0)
        return True

    def release(self, seqs, keep):
        where = [(s, i) for s, k in zip(seqs, keep) for i in range(k, self.seq_pages[s])]
        for s, i in where:
            page = self.table[s, i]
            self.refs[page] -= 1
            if self.refs[page] == 0:
                self.free.append(page)
            self.table[s, i] = -1
        for s, k in zip(seqs, keep):
            self.seq_pages[s] = min(self.seq_pages[s], k)

    def compact(self):
        used = int((self.refs > 0).sum())
        hole = [p for p in range(used) if self.refs[p] == 0]
        far = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        for h, f in zip(hole, far):
            self.pages[h] = self.pages[f]
            self.refs[h], self.refs[f] = self.refs[f], 0
            self.table[self.table == f] = h
        self.free = list(range(len(self.refs) - 1, used - 1, -1))


class Pool:
    def __init__(self, mq, m):
        import torch
        self.mq = mq
        self.cache = mq.KVCache(dev(m.pages), dev(m.table), m.ctype, m.Hkv, m.D)
        free = np.zeros(len(m.refs), np.int32)
        free[:len(m.free)] = m.free
        self.pool = mq.KVPool(self.cache, dev(m.seq_pages), dev(m.refs), dev(free),
                              torch.tensor([len(m.free)], dtype=torch.int32, device="cuda"))

    def same(self, m, status=0):
        ok_status(self.mq, status)
        assert np.array_equal(self.cache.table.cpu().numpy(), m.table)
        assert np.array_equal(self.pool.refs.cpu().numpy(), m.refs)
        assert np.array_equal(self.pool.seq_pages.cpu().numpy(), m.seq_pages)
        n = int(self.pool.n_free)
        assert n == len(m.free) and self.pool.free_list.cpu().numpy()[:n].tolist() == [int(x) for x in m.free]
        assert np.array_equal(self.cache.pages.cpu().numpy().reshape(m.pages.shape), m.pages)


i32 = lambda v: dev(np.asarray(v, np.int32))


@pytest.mark.parametrize("ctype,Hkv,D", SHAPES)
def test_a_run_of_calls(cuda_ready, ctype, Hkv, D):
    mq = cuda_ready
    rng = np.random.default_rng(D + Hkv)
    m = Model(90, 12, 20, ctype, Hkv, D, rng)
    p = Pool(mq, m)
    lens = np.array([1, 64, 65, 300, 0, 0, 0, 0, 0, 0, 0, 700])
    m.grow(lens)
    mq.kv_grow(p.cache, p.pool, i32(lens))
    p.same(m)
    steps = 0
    for step in range(25):
        what = rng.choice(["grow", "fork", "free", "keep", "compact"])
        have = [s for s in range(12) if m.seq_pages[s] > 0]
        empty = [s for s in range(12) if m.seq_pages[s] == 0]
        if what == "grow":
            lens = [int(min(20 * 64, k * 64 + rng.integers(0, 100))) for k in m.seq_pages]
            if not m.grow(lens):
                continue
            mq.kv_grow(p.cache, p.pool, i32(lens))
        elif what == "fork" and have and empty:
            dst = rng.permutation(empty)[:rng.integers(1, len(empty) + 1)]
            src = rng.choice(have, len(dst))
            lens = [int(rng.integers(0, 64 * m.seq_pages[s] + 1)) for s in src]
            if not m.fork(src, dst, lens):
                continue
            mq.kv_fork(p.cache, p.pool, i32(src), i32(dst), i32(lens))
        elif what in ("free", "keep") and len(have) > 3:
            gone = rng.permutation(12)[:rng.integers(1, 5)]
            keep = [int(rng.integers(0, 4)) if what == "keep" else 0 for _ in gone]
            m.release(gone, keep)
            mq.kv_free(p.cache, p.pool, i32(gone), i32(keep) if what == "keep" else None)
        elif what == "compact":
            m.compact()
            mq.kv_compact(p.cache, p.pool)
        p.same(m)
        steps += 1
    assert steps > 10


@pytest.mark.parametrize("ctype,Hkv,D", SHAPES)
@pytest.mark.parametrize("rest", [1, 2, 7, 31, 32, 33, 63])
def test_begun_pages_are_copied_to_the_token(cuda_ready, ctype, Hkv, D, rest):
    rng = np.random.default_rng(rest)
    m = Model(12, 4, 6, ctype, Hkv, D, rng)
    m.grow([200, 0, 0, 0])
    p = Pool(cuda_ready, m)
    m.fork([0, 0, 0], [3, 1, 2], [128 + rest, rest, 128])
    cuda_ready.kv_fork(p.cache, p.pool, i32([0, 0, 0]), i32([3, 1, 2]), i32([128 + rest, rest, 128]))
    p.same(m)


def test_large_pools(cuda_ready):
    # more references, sequences and pages than one round of the threads takes; shared pages, all references of some
    rng = np.random.default_rng(5)
    m = Model(40000, 4096, 64, "q8_0", 1, 64, rng)
    lens = np.zeros(4096, np.int64)
    lens[:400] = rng.integers(1, 64 * 64, 400)
    p = Pool(cuda_ready, m)
    assert m.grow(lens)
    cuda_ready.kv_grow(p.cache, p.pool, i32(lens))
    p.same(m)
    dst = rng.permutation(np.arange(400, 4096))[:3000]
    src = rng.integers(0, 400, 3000)
    n = [int(rng.integers(1, lens[s] + 1)) for s in src]
    assert m.fork(src, dst, n)
    cuda_ready.kv_fork(p.cache, p.pool, i32(src), i32(dst), i32(n))
    p.same(m)
    gone = rng.permutation(np.concatenate([np.arange(0, 400, 2), dst[:2500], np.arange(3900, 4000)]))
    gone = np.array(list(dict.fromkeys(gone.tolist())))
    keep = rng.integers(0, 5, len(gone))
    m.release(gone, keep)
    cuda_ready.kv_free(p.cache, p.pool, i32(gone), i32(keep))
    p.same(m)
    m.compact()
    cuda_ready.kv_compact(p.cache, p.pool)
    p.same(m)


def test_too_few_free_pages_change_nothing(cuda_ready):
    mq = cuda_ready
    rng = np.random.default_rng(6)
    m = Model(6, 5, 8, "f16", 2, 64, rng)
    m.grow([100, 150, 0, 0, 0])
    p = Pool(mq, m)
    mq.kv_grow(p.cache, p.pool, i32([100, 300, 0, 0, 0]))
    p.same(m, mq.MQ_DEV_KV_FULL)
    mq.kv_fork(p.cache, p.pool, i32([0, 1]), i32([2, 3]), i32([100, 150]))
    p.same(m, mq.MQ_DEV_KV_FULL)
    mq.kv_fork(p.cache, p.pool, i32([0, 1, 1]), i32([2, 3, 4]), i32([64, 128, 150]))
    m.fork([0, 1, 1], [2, 3, 4], [64, 128, 150])
    p.same(m)
    assert not m.free
    m.compact()
    mq.kv_compact(p.cache, p.pool)
    p.same(m)


def test_bad_entries_are_left_out_and_reported(cuda_ready):
    mq = cuda_ready
    rng = np.random.default_rng(7)
    m = Model(30, 6, 8, "q8_0", 2, 64, rng)
    m.grow([200, 100, 0, 0, 0, 0])
    p = Pool(mq, m)
    R = mq.MQ_DEV_KV_RANGE
    # fork: unknown sequences, more than there is, a sequence that has pages, one named twice, one that is forked from
    mq.kv_fork(p.cache, p.pool, i32([0, -1, 6, 0, 0, 0]), i32([2, 3, 4, 6, 1, 5]), i32([70, 1, 1, 1, 64, 257]))
    m.fork([0], [2], [70])
    p.same(m, R)
    mq.kv_fork(p.cache, p.pool, i32([0, 1, 0, 1, 3]), i32([3, 3, 4, 5, 0]), i32([65, 65, -1, 65, 0]))
    m.fork([1], [5], [65])  # 3 is a source of the last entry too: neither of its own is taken
    p.same(m, R)
    # free: a sequence twice, unknown ones, a negative keep
    mq.kv_free(p.cache, p.pool, i32([1, 1, -1, 6, 2]), i32([1, 0, 0, 0, -1]))
    m.release([1], [1])
    p.same(m, R)
    # grow: more than the table holds, a negative length
    mq.kv_grow(p.cache, p.pool, i32([200, -5, 100, 64 * 9, 64, 70]))
    m.grow([200, 0, 100, 0, 64, 70])
    p.same(m, R)
    # a table entry outside the pool is passed over, a count of free pages outside it finds nothing
    p.cache.table[0, 1] = 30
    mq.kv_free(p.cache, p.pool, i32([0]))
    ok_status(mq, R)
    assert int(p.pool.seq_pages[0]) == 0
    p.pool.n_free.fill_(31)
    before = p.cache.table.clone()
    mq.kv_grow(p.cache, p.pool, i32([64, 64, 64, 64, 64, 64 * 8]))
    ok_status(mq, R | mq.MQ_DEV_KV_FULL)
    mq.kv_free(p.cache, p.pool, i32([1]))
    ok_status(mq, R)
    assert (p.cache.table == before).all()
    p.pool.n_free.fill_(2)
    p.pool.free_list[1] = -4
    mq.kv_fork(p.cache, p.pool, i32([5]), i32([0]), i32([65]))
    ok_status(mq, R)
    assert int(p.pool.seq_pages[0]) == 0


def test_empty_lists_and_lengths(cuda_ready):
    mq = cuda_ready
    m = Model(9, 3, 4, "f16", 1, 64, np.random.default_rng(1))
    p = Pool(mq, m)
    none = i32([])
    mq.kv_grow(p.cache, p.pool, i32([0, 0, 0]))
    mq.kv_fork(p.cache, p.pool, none, none, none)
    mq.kv_free(p.cache, p.pool, none)
    mq.kv_free(p.cache, p.pool, i32([0, 2]))
    mq.kv_fork(p.cache, p.pool, i32([0]), i32([1]), i32([0]))
    p.same(m)
    m.compact()
    mq.kv_compact(p.cache, p.pool)
    p.same(m)


def test_alloc_and_captured_calls(cuda_ready):
    # a captured grow, fork, free and compact follow the device's lists from replay to replay
    import torch
    mq = cuda_ready
    table = torch.zeros((6, 10), dtype=torch.int32, device="cuda")
    cache = mq.KVCache.alloc(40, table, "q8_0", 2, 64)
    cache.pages.random_(0, 255)
    pool = mq.KVPool.alloc(cache)
    m = Model(40, 6, 10, "q8_0", 2, 64, np.random.default_rng(2))
    m.pages, m.free = cache.pages.cpu().numpy().reshape(m.pages.shape).copy(), list(range(39, -1, -1))
    p = Pool.__new__(Pool)
    p.mq, p.cache, p.pool = mq, cache, pool
    p.same(m)
    lens, src, dst, n, gone = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (6, 2, 2, 2, 2))

    def calls():
        mq.kv_grow(cache, pool, lens)
        mq.kv_fork(cache, pool, src, dst, n)
        mq.kv_free(cache, pool, gone)
        mq.kv_compact(cache, pool)

    lens[0] = 100
    dst.copy_(i32([1, 2]))
    gone.copy_(i32([3, 4]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        calls()
    m.grow([100, 0, 0, 0, 0, 0])
    m.compact()
    p.same(m)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls()
    for L, a, b, k, e in (([300, 0, 0, 70, 0, 0], [0, 3], [1, 2], [65, 70], [3, 0]),
                          ([0, 500, 0, 0, 64, 0], [1, 2], [0, 5], [200, 6], [1, 2])):
        for t, v in zip((lens, src, dst, n, gone), (L, a, b, k, e)):
            t.copy_(i32(v))
        torch.cuda.synchronize()
        g.replay()
        m.grow(L)
        m.fork(a, b, k)
        m.release(e, [0, 0])
        m.compact()
        p.same(m)


def test_on_a_given_stream(cuda_ready):
    # by its handle, behind what it is doing
    import torch
    mq = cuda_ready
    m = Model(40, 5, 8, "f16", 2, 64, np.random.default_rng(4))
    p = Pool(mq, m)
    side = torch.cuda.Stream()
    lens, src, dst, n, gone = i32([200, 70, 0, 0, 0]), i32([0, 1]), i32([4, 2]), i32([130, 70]), i32([1])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(2e8))
    h = side.cuda_stream
    mq.kv_grow(p.cache, p.pool, lens, stream=h)
    mq.kv_fork(p.cache, p.pool, src, dst, n, stream=h)
    mq.kv_free(p.cache, p.pool, gone, stream=h)
    mq.kv_compact(p.cache, p.pool, stream=h)
    assert not side.query()
    m.grow([200, 70, 0, 0, 0])
    m.fork([0, 1], [4, 2], [130, 70])
    m.release([1], [0])
    m.compact()
    p.same(m)


def state(p):
    """Everything of a pool, to compare."""
    return [x.clone() for x in (p.cache.table, p.cache.pages, p.pool.refs, p.pool.seq_pages, p.pool.n_free, p.pool.free_list)]


@pytest.mark.parametrize("what", ["in use", "twice", "behind", "negative"])
@pytest.mark.parametrize("at", [0, 3, 1500])
def test_stack_that_names_a_page_that_is_not_free_changes_nothing(cuda_ready, what, at):
    # `at` pages below the top: grow takes it with 2000 others, fork with 40; the pages taken before are free again
    import torch
    mq = cuda_ready
    m = Model(2300, 50, 60, "q8_0", 1, 64, np.random.default_rng(at))
    lens = np.zeros(50, np.int64)
    lens[:4] = [70, 30, 64, 500]
    assert m.grow(lens)
    p = Pool(mq, m)
    more = np.concatenate([lens[:4], np.full(46, 40 * 64 + 1)])
    forks = i32(np.arange(40) % 4), i32(np.arange(4, 44)), i32([20] * 40)
    calls = [lambda: mq.kv_grow(p.cache, p.pool, i32(more))] + \
        [lambda: mq.kv_fork(p.cache, p.pool, *forks)] * (at < 40)
    n = int(p.pool.n_free)
    good = p.pool.free_list.clone()
    p.pool.free_list[n - 1 - at] = {"in use": int(m.table[3, 2]), "twice": int(good[n - 3 - at]), "behind": 2300,
                                    "negative": -1}[what]
    for call in calls:
        before = state(p)
        call()
        ok_status(mq, mq.MQ_DEV_KV_RANGE)
        assert all(torch.equal(a, b) for a, b in zip(state(p), before))
    p.pool.free_list.copy_(good)
    if at < 40:
        calls[1]()
        assert m.fork(np.arange(40) % 4, np.arange(4, 44), [20] * 40)
    else:
        calls[0]()
        assert m.grow(more)
    p.same(m)


@pytest.mark.parametrize("ld", [20, 400])  # one CTA; a cluster
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("counts", [[1], [0], [-3], [1, 0, 2, -1, 1]])
def test_pages_named_more_often_than_counted_are_freed_once(cuda_ready, ld, shared, counts):
    # entries of the table over each other's pages, and pages without a count, among sequences in order
    mq = cuda_ready
    rng = np.random.default_rng(ld + len(counts))
    m = Model(9 * ld, 8, ld, "f16", 1, 64, rng)
    assert m.grow([64 * 19, 64 * (ld - 1), 64 * 7, 64 * 3, 64 * ld, 0, 0, 64])
    if shared:
        assert m.fork([1, 4], [5, 6], [64 * 5, 64 * 9 + 1])
    for j, c in enumerate(counts):
        page = m.table[1, 8 + j]  # of nobody else
        m.refs[page] = c
        if c > 0:  # named c times more than it is counted
            for k in range(c):
                m.refs[m.table[4, ld - 8 + 3 * j + k - 7]] = 0  # (whose page is given up by nobody)
                m.table[4, ld - 8 + 3 * j + k - 7] = page
    p = Pool(mq, m)
    gone, keep = [4, 2, 1, 5], [2, 0, 1, 0]
    where = [(s, i) for s, k in zip(gone, keep) for i in range(k, m.seq_pages[s])]
    names = [int(m.table[s, i]) for s, i in where]
    for at, ((s, i), page) in enumerate(zip(where, names)):
        m.table[s, i] = -1
        n = names.count(page)
        if page in names[at + 1:] or m.refs[page] <= 0:
            continue
        m.refs[page] = max(m.refs[page] - n, 0)
        if m.refs[page] == 0:
            m.free.append(page)
    for s, k in zip(gone, keep):
        m.seq_pages[s] = min(m.seq_pages[s], k)
    mq.kv_free(p.cache, p.pool, i32(gone), i32(keep))
    p.same(m, mq.MQ_DEV_KV_RANGE)


def test_fork_does_not_share_pages_that_are_not_in_use(cuda_ready):
    # outside the pool, or without a count: -1 in the new tables, counts and the other entries as they should be
    mq = cuda_ready
    m = Model(60, 8, 12, "q8_0", 2, 64, np.random.default_rng(8))
    assert m.grow([640, 700, 0, 0, 0, 0, 0, 0])
    free = int(m.free[0])  # the stack's lowest: taken by nobody here
    m.table[0, [1, 4, 6, 9]] = [60, -9, free, 2**31 - 1]
    p = Pool(mq, m)
    mq.kv_fork(p.cache, p.pool, i32([0, 1, 0, 0]), i32([3, 4, 6, 5]), i32([640, 65, 9 * 64 + 5, 64]))
    for s, d, n in ((0, 3, 640), (1, 4, 65), (0, 6, 9 * 64 + 5), (0, 5, 64)):
        for i in range(n // 64):
            page = m.table[s, i]
            fine = 0 <= page < 60 and page != free
            m.table[d, i] = page if fine else -1
            if fine:
                m.refs[page] += 1
        if n % 64:
            m.table[d, n // 64] = m.take()
            if s == 1:  # (sequence 0's begun page is outside the pool)
                m.pages[m.table[d, 1]][:, m.rows(1)] = m.pages[m.table[1, 1]][:, m.rows(1)]
        m.seq_pages[d] = -(-n // 64)
    p.same(m, mq.MQ_DEV_KV_RANGE)


@pytest.mark.parametrize("n_pages", [60, 3000])  # one CTA; a cluster
@pytest.mark.parametrize("moves", [True, False])
def test_compact_takes_pages_without_a_count_out_of_the_table(cuda_ready, n_pages, moves):
    # before and behind the pages in use, where another page moves to and where none does; what earlier calls left in
    # the scratch is nothing to go by
    mq = cuda_ready
    rng = np.random.default_rng(n_pages)
    m = Model(n_pages, 6, 12, "q8_0", 1, 64, rng)
    if not moves:
        m.free = sorted(m.free, reverse=True)
    assert m.grow([64 * 10, 64 * 7, 300, 64, 64 * 12, 64])
    p = Pool(mq, m)
    p.pool.scratch.copy_(dev(rng.integers(-5, n_pages, p.pool.scratch.numel()).astype(np.int32)))
    used, held = int((m.refs > 0).sum()), m.table.copy()
    low = [x for x in range(used) if m.refs[x] == 0][:2] if moves else []
    lost = low + [int(x) for x in m.free[:2]] + [n_pages, -1, 2**31 - 1]
    for j, x in enumerate(lost):  # the pages that were named there stay in use, nobody names them
        m.table[4, 2 + j] = x
    for x in m.free[2:4]:
        m.refs[x] = -7
    p.cache.table.copy_(dev(m.table))
    p.pool.refs.copy_(dev(m.refs))
    assert (m.table[4, 2:2 + len(lost)] != held[4, 2:2 + len(lost)]).all()
    m.table[4, 2:2 + len(lost)] = -1
    m.refs[m.refs < 0] = 0
    m.compact()
    mq.kv_compact(p.cache, p.pool)
    p.same(m, mq.MQ_DEV_KV_RANGE)
    p.pool.seq_pages[2] = 13
    mq.kv_compact(p.cache, p.pool)
    ok_status(mq, mq.MQ_DEV_KV_RANGE)
