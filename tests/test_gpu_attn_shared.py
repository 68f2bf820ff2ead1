"""Attention over shared prefixes against a plain 64-bit form of the whole context.

The bound is the tree attention's (tests/test_gpu_attn.py) plus 2^-20 A for the join of a prefix and what is behind it:
a few fp32 roundings of the two parts' factors, sums and outputs.
"""
import numpy as np
import pytest

from tests import kv_plain as P
from tests.test_gpu_attn import HEADS, as_i64, bound, tree_masks, values_of
from tests.test_gpu_kv import dev, ok_status

pytestmark = pytest.mark.gpu


class Batch:
    """groups: (pages shared, [(own tokens of context, new tokens) of each sequence]); pages 0: nothing in common.
    Sequences before `lead` and the last `tail` ones lie in no group (their groups are listed with 0 pages)."""

    def __init__(self, rng, groups, Hq, Hkv, D, ctype, lead=0, tail=0, spread=1.0, q_pad=0, masks="tree"):
        self.Hq, self.Hkv, self.D, self.ctype = Hq, Hkv, D, ctype
        draw = lambda n: [(rng.standard_normal((n, Hkv, D)) * s).astype(np.float32) for s in (spread, 1.0)]
        shared = [draw(64 * g[0]) for g in groups]
        own = [draw(c + t) for g in groups for c, t in g[1]]
        parts = shared + own
        pages, table = P.build([k for k, _ in parts], [v for _, v in parts], ctype, rng)
        self.group = [i for i, g in enumerate(groups) for _ in g[1]]
        self.new = [t for g in groups for _, t in g[1]]
        self.ctx = [64 * g[0] + c for g in groups for c, _ in g[1]]
        most = max(g[0] for g in groups)
        self.table = np.full((len(self.new), most + table.shape[1]), -7, np.int32)
        for s, g in enumerate(self.group):
            n = groups[g][0]
            self.table[s, :n] = table[g, :n]
            self.table[s, n:n + table.shape[1]] = table[len(groups) + s]
        self.pages = pages
        self.K = [np.concatenate([shared[g][0], own[s][0]]) for s, g in enumerate(self.group)]
        self.V = [np.concatenate([shared[g][1], own[s][1]]) for s, g in enumerate(self.group)]
        n = sum(self.new)
        self.q = rng.standard_normal((n, Hq * D + q_pad)).astype(np.float16)
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.bits = [tree_masks(rng, t) if masks == "tree" else [(2 << i) - 1 for i in range(t)] if masks == "chain"
                     else [0] * t for t in self.new]
        self.masks = masks
        counts = [len(g[1]) for g in groups]
        ends = np.cumsum(counts)
        named = range(lead, len(groups) - tail)
        self.grp_start = np.array([int(ends[i] - counts[i]) for i in named] +
                                  [int(ends[named[-1]]) if len(named) else 0], np.int32)
        self.grp_pages = np.array([groups[i][0] for i in named], np.int32)

    def cache(self, mq):
        return mq.KVCache(dev(self.pages), dev(self.table), self.ctype, self.Hkv, self.D)

    def call(self, mq, cache=None, scale=None, out_type="f16", tree=False, **kw):
        m = None if self.masks == "chain" else dev(as_i64([b for s in self.bits for b in s]))
        args = dict(mask=m, scale=scale, out_type=out_type, max_len=max(c + t for c, t in zip(self.ctx, self.new)),
                    max_tokens=max(1, max(self.new)))
        args.update(kw)
        c, q = self.cache(mq) if cache is None else cache, dev(self.q)[:, :self.Hq * self.D]
        if tree:
            return mq.attn_tree(c, q, dev(self.start), dev(np.array(self.ctx, np.int32)), **args)
        return mq.attn_shared(c, q, dev(self.start), dev(np.array(self.ctx, np.int32)), dev(self.grp_start),
                              dev(self.grp_pages), **args)

    def check(self, out, scale=None, out_type="f16", only=None):
        Hq, D, n = self.Hq, self.D, sum(self.new)
        got = (out.cpu().numpy().astype(np.float64) if out_type == "f16" else values_of(out, n, Hq * D)).reshape(n, Hq, D)
        for s in range(len(self.new)) if only is None else only:
            a, b = self.start[s], self.start[s + 1]
            ref, A, big = P.attention(self.q[a:b, :Hq * D].reshape(-1, Hq, D), P.stored(self.K[s], self.ctype),
                                      P.stored(self.V[s], self.ctype), self.ctx[s], self.bits[s],
                                      D**-0.5 if scale is None else scale)
            tol = bound(ref, A, big) + 2.0**-20 * A
            if out_type == "q8_0":
                top = (np.abs(ref) + tol).reshape(b - a, Hq, D // 32, 32).max(-1).repeat(32, -1)
                tol = tol + top / 127 * (0.5 + 2 * 127 * 2**-11)
            err = np.abs(got[a:b] - ref)
            assert (err <= tol).all(), (s, self.ctx[s], self.new[s], float((err / tol).max()), np.argwhere(err > tol)[:3])


def run(mq, rng, groups, *shape, scale=None, out_type="f16", call={}, **kw):
    b = Batch(rng, groups, *shape, **kw)
    out = b.call(mq, scale=scale, out_type=out_type, **call)
    ok_status(mq)
    b.check(out, scale, out_type)
    return b, out


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_decode(cuda_ready, ctype, Hq, Hkv, D):
    # one token per sequence: own contexts empty, inside, at and past page borders; groups of one, without pages, none
    rng = np.random.default_rng(Hq)
    own = [0, 1, 15, 62, 63, 64, 65, 127, 128, 200]
    run(cuda_ready, rng, [(0, [(5, 1), (70, 1)]), (3, [(c, 1) for c in own]), (0, [(9, 1)]), (1, [(0, 1)]),
                          (7, [(c, 1) for c in own[::-2]]), (2, [(30, 1), (31, 1)])], Hq, Hkv, D, ctype, lead=1, tail=1,
        masks="chain")


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("masks", ["tree", "chain", "none"])
def test_trees(cuda_ready, ctype, Hq, Hkv, D, masks):
    # ragged trees, sequences without tokens, whole groups without; rows that see the prefix alone
    rng = np.random.default_rng(Hq + D)
    run(cuda_ready, rng, [(2, [(0, 7), (60, 64), (5, 0), (130, 3)]), (4, [(10, 0), (3, 0)]), (1, [(64, 33), (63, 1), (0, 19)]),
                          (5, [(1, 2)])], Hq, Hkv, D, ctype, masks=masks)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 9, 64])
@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
def test_long_prefix_over_many_blocks_of_rows(cuda_ready, ctype, T):
    # a prefix that many CTAs share, several blocks of 256 rows and one of a few
    rng = np.random.default_rng(T)
    seqs = 90 // T + 1
    run(cuda_ready, rng, [(60, [(int(c), T) for c in rng.integers(0, 200, seqs)])], 28, 4, 128, ctype)


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_groups(cuda_ready, ctype, D):
    # more groups than SMs, most of them one CTA's; some longer
    rng = np.random.default_rng(D)
    groups = [(int(p), [(int(c), int(t)) for c, t in zip(rng.integers(0, 100, k), rng.integers(0, 4, k))])
              for p, k in zip(rng.integers(0, 5, 60), rng.integers(1, 5, 60))]
    groups[30] = (33, groups[30][1])
    run(cuda_ready, rng, groups, 16, 4, D, ctype)


def test_wide_groups_of_heads(cuda_ready):
    # one key/value head for 64 query heads, and as many heads as there are
    rng = np.random.default_rng(8)
    run(cuda_ready, rng, [(9, [(3, 2), (70, 1), (0, 5)]), (3, [(20, 5)] * 11)], 64, 1, 64, "q8_0")
    run(cuda_ready, rng, [(4, [(3, 1), (70, 1), (0, 1)])], 24, 24, 64, "f16")


@pytest.mark.parametrize("T", [1, 6, 40])
def test_q8_0_output(cuda_ready, T):
    rng = np.random.default_rng(T + 50)
    for Hq, Hkv, D in [(28, 4, 128), (16, 8, 64)]:
        run(cuda_ready, rng, [(0, [(9, T)]), (11, [(30, T), (0, 1), (64, T)])], Hq, Hkv, D, "q8_0", out_type="q8_0")


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
def test_large_scores_and_scales(cuda_ready, ctype):
    # the largest scores in the prefix or behind it, scales of both signs
    rng = np.random.default_rng(77)
    for scale in (0.0, -0.3, 4.0, 1e-6):
        for T in (1, 24):
            run(cuda_ready, rng, [(3, [(40, T), (5, 1), (90, T)])], 28, 4, 128, ctype, scale=scale)
    run(cuda_ready, rng, [(50, [(300, 2)] * 5)], 14, 2, 64, ctype, spread=6.0)


def test_strided_queries_and_output(cuda_ready):
    import torch
    rng = np.random.default_rng(5)
    for T in (2, 30):
        full = torch.full((2 * T + 3, 28 * 128 + 8), -9.0, dtype=torch.float16, device="cuda")
        run(cuda_ready, rng, [(4, [(9, T), (20, 3), (1, T)])], 28, 4, 128, "q8_0", q_pad=16, call=dict(out=full[:, :28 * 128]))
        assert (full[:, 28 * 128:] == -9).all()


def test_without_groups_it_is_the_tree_attention(cuda_ready):
    import torch
    mq = cuda_ready
    b = Batch(np.random.default_rng(1), [(0, [(100, 3), (5, 1)])], 28, 4, 128, "q8_0", lead=1)
    assert torch.equal(b.call(mq), b.call(mq, tree=True))
    b = Batch(np.random.default_rng(1), [(0, [(100, 3), (5, 1)])], 28, 4, 128, "q8_0")
    assert torch.equal(b.call(mq, max_pages=0), b.call(mq, tree=True))
    assert torch.equal(b.call(mq, max_pages=3), b.call(mq, tree=True))
    ok_status(mq)


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("T", [1, 3, 20])
def test_what_is_not_finite(cuda_ready, ctype, T):
    # an infinite value in the prefix reaches every row; NaN or infinity behind it the rows that see it, and no other
    mq = cuda_ready
    Hq, Hkv, D = 28, 4, 128
    for where, value in (("prefix", np.inf), ("own", np.inf), ("own", np.nan), ("key", np.nan)):
        rng = np.random.default_rng(T)
        b = Batch(rng, [(2, [(40, T), (3, T), (70, T)])], Hq, Hkv, D, ctype)
        big = value if ctype == "f16" or np.isnan(value) else 7.6e6  # scale 59843, code 127
        pages, table = b.pages.copy(), b.table
        j = T // 2
        slot = 20 if where == "prefix" else b.ctx[1] + j
        page, row = table[1, slot // 64], slot % 64
        k, v = P.unpack(pages[page, 1], ctype, D)
        k, v = k.astype(np.float32), v.astype(np.float32)
        (k if where == "key" else v)[row, 5] = big
        with np.errstate(all="ignore"):
            pages[page, 1] = P.pack(k, v, ctype)
        # the other values are those of the changed block: packed again, a q8_0 row keeps its codes but the changed one's
        k2, v2 = P.unpack(pages[page, 1], ctype, D)
        b.pages = pages
        stored = {}
        for s in range(3):
            K, V = P.stored(b.K[s], ctype).copy(), P.stored(b.V[s], ctype).copy()
            if where == "prefix" or s == 1:
                lo = slot - row
                n = min(64, len(K) - lo)
                K[lo:lo + n, 1], V[lo:lo + n, 1] = k2[:n], v2[:n]
            stored[s] = K, V
        out = b.call(mq).cpu().numpy().astype(np.float64).reshape(-1, Hq, D)
        ok_status(mq)
        for s in range(3):
            a, e = b.start[s], b.start[s + 1]
            with np.errstate(all="ignore"):
                ref, A, big_ = P.attention(b.q[a:e].reshape(-1, Hq, D), *stored[s], b.ctx[s], b.bits[s], D**-0.5)
            inf, fine = np.isinf(ref), np.isfinite(ref)
            if where == "prefix":
                assert inf[:, 7:14, 5].all()
            assert np.array_equal(out[a:e][inf], ref[inf]), (where, value, s)
            assert np.isnan(out[a:e][np.isnan(ref)]).all(), (where, value, s)
            tol = bound(ref, A, big_) + 2.0**-20 * A
            assert (np.abs(out[a:e] - ref)[fine] <= tol[fine]).all(), (where, value, s)


def test_agrees_call_by_call_in_one_workspace(cuda_ready):
    # batches that grow and shrink, other heads, other row counts, in one workspace
    import torch
    mq = cuda_ready
    calls = [([(40, [(30, 1)] * 9)], 28, 4, 128, "q8_0"), ([(3, [(30, 5)] * 4), (1, [(0, 5)])], 16, 8, 64, "f16"),
             ([(20, [(100, 40)] * 3)], 28, 4, 128, "q8_0"), ([(2, [(5, 1)] * 64), (7, [(6, 1)] * 3)], 28, 4, 128, "f16"),
             ([(0, [(300, 2)])], 8, 1, 128, "q8_0"), ([(40, [(30, 1)] * 9)], 28, 4, 128, "q8_0")]
    batches = [Batch(np.random.default_rng(i), *c) for i, c in enumerate(calls)]
    size = max(mq.attn_shared_workspace(b.cache(mq), b.Hq, sum(b.new), len(b.grp_pages), max(b.new)).numel() for b in batches)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for b in batches:
        x, y = b.call(mq, workspace=ws), b.call(mq, workspace=ws)
        ok_status(mq)
        b.check(x)
        assert torch.equal(x, y)
    with pytest.raises(mq.MQError):
        batches[0].call(mq, workspace=ws[:1024])


def test_one_workspace_for_this_and_the_tree_attention(cuda_ready):
    import torch
    mq = cuda_ready
    b = [Batch(np.random.default_rng(i), [(20, [(50, t)] * 9)], 28, 4, 128, "q8_0") for i, t in enumerate((1, 2, 9))]
    caches = [x.cache(mq) for x in b]
    size = max(mq.attn_shared_workspace(c, 28, sum(x.new), 1, max(x.new)).numel() for x, c in zip(b, caches))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 1, 0, 2):
        for tree in (True, False, True):
            b[i].check(b[i].call(mq, caches[i], workspace=ws, tree=tree))
    ok_status(mq)


def test_sequences_without_tokens_need_no_pages(cuda_ready):
    # answers that are given up stay in their group: their rows of the table are empty, the first's too
    mq = cuda_ready
    b = Batch(np.random.default_rng(3), [(4, [(9, 0), (3, 0), (40, 2), (5, 0), (70, 1)]), (2, [(5, 0), (6, 0)]), (3, [(1, 1)])],
              28, 4, 128, "q8_0")
    for s in (0, 1, 3, 5, 6):
        b.table[s] = -1
        b.ctx[s] = 0
    out = b.call(mq)
    ok_status(mq)
    b.check(out, only=[2, 4, 7])


def test_graph_replay_follows_device_lengths(cuda_ready):
    # a captured call: lengths, groups and prefixes change between replays; two graphs share a workspace
    import torch
    mq = cuda_ready
    b = Batch(np.random.default_rng(31), [(8, [(100, 3), (400, 3), (0, 3), (64, 3)])], 28, 4, 128, "q8_0")
    cache, q, start = b.cache(mq), dev(b.q), dev(b.start)
    mask = dev(as_i64([x for s in b.bits for x in s]))
    ctx, gs, gp = dev(np.array(b.ctx, np.int32)), dev(np.array([0, 4, 4], np.int32)), dev(np.array([8, 0], np.int32))
    ws = mq.attn_shared_workspace(cache, 28, 12, 2, 3)
    outs = [torch.empty((12, 28 * 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    call = lambda o, w: mq.attn_shared(cache, q, start, ctx, gs, gp, mask=mask, max_len=1000, max_tokens=3, max_pages=8,
                                       out=o, workspace=w)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(outs[0], ws)
    side.synchronize()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(o, ws)
        graphs.append(g)
    for lens, starts, pages in ((b.ctx, [0, 4, 4], [8, 0]), ([520, 600, 512, 512], [0, 2, 4], [8, 5]),
                                (b.ctx, [1, 1, 4], [8, 7]), ([9, 10, 500, 512], [2, 3, 4], [3, 8])):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        gs.copy_(torch.tensor(starts, dtype=torch.int32))
        gp.copy_(torch.tensor(pages, dtype=torch.int32))
        want = mq.attn_tree(cache, q, start, ctx, mask=mask, max_len=1000, max_tokens=3).float()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for g in graphs:
                g.replay()
        side.synchronize()
        ok_status(mq)
        fresh = torch.empty_like(outs[0])
        call(fresh, mq.attn_shared_workspace(cache, 28, 12, 2, 3))
        ok_status(mq)
        assert torch.equal(outs[0], fresh) and torch.equal(outs[1], fresh)
        # both within 2^-10 + 2^-11 of the exact result: of values around 1
        assert float((fresh.float() - want).abs().max()) < 2**-8


@pytest.mark.parametrize("T", [1, 3, 40])
def test_bad_device_data_is_skipped_and_reported(cuda_ready, T):
    import torch
    mq = cuda_ready
    b = Batch(np.random.default_rng(41), [(0, [(20, T)]), (3, [(100, T), (7, T), (0, T)]), (2, [(50, T), (9, T)])], 8, 2, 64, "f16")
    R, n = mq.MQ_DEV_KV_RANGE, 6 * T

    def call(ctx=b.ctx, gs=b.grp_start, gp=b.grp_pages, start=b.start, table=b.table, max_pages=3, max_len=400):
        cache = mq.KVCache(dev(b.pages), dev(np.asarray(table, np.int32)), "f16", 2, 64)
        out = torch.full((n, 8 * 64), 3.0, dtype=torch.float16, device="cuda")
        mq.attn_shared(cache, dev(b.q), dev(np.asarray(start, np.int32)), dev(np.asarray(ctx, np.int32)),
                       dev(np.asarray(gs, np.int32)), dev(np.asarray(gp, np.int32)),
                       mask=dev(as_i64([x for s in b.bits for x in s])), max_len=max_len, max_tokens=T, max_pages=max_pages,
                       out=out)
        torch.cuda.synchronize()
        return out, mq.mq_read_device_status(0)

    def same(out, st, gone, want=R):
        assert st == want
        # what is skipped changes how the rest is split, and with it roundings
        b.check(out, only=[s for s in range(6) if s not in gone])
        for s in gone:
            assert (out[s * T:(s + 1) * T] == 3).all(), s

    good, st = call()
    b.check(good)
    assert st == 0
    # one sequence wrong: the others of its group are right
    for c in (-1, 3 * 64 - 1, 401 - T, 2**31 - 1):
        same(*call(ctx=[*b.ctx[:2], c, *b.ctx[3:]]), {2})
    # a group wrong: its sequences stay unwritten
    same(*call(gp=[0, 4, 2]), {1, 2, 3})
    same(*call(gp=[0, -1, 2]), {1, 2, 3})
    same(*call(gp=[0, 4, 2], max_pages=4), {2, 3})  # within the bound, longer than two contexts
    same(*call(gs=[0, 1, 4, 7]), {4, 5})
    # a page outside the cache: of the prefix, of one sequence's own
    wrong = b.table.copy()
    wrong[1, 1] = len(b.pages)
    same(*call(table=wrong), {1, 2, 3})
    wrong = b.table.copy()
    wrong[2, 3] = -1
    same(*call(table=wrong), {2})
    # the table row of the first sequence is the group's
    wrong = b.table.copy()
    wrong[2:4, :3] = -5
    same(*call(table=wrong), set(), 0)
    # tokens that a sequence does not have
    out, st = call(start=[*b.start[:6], n + 1])
    same(out, st, {4, 5})
    assert call()[1] == 0


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("T", [1, 2, 40])
def test_wait_that_runs_out_is_reported_and_writes_nothing(cuda_ready, ctype, T):
    import torch
    mq = cuda_ready
    b = Batch(np.random.default_rng(T), [(60, [(3000, T), (20, T), (100, T)])], 28, 4, 128, ctype)
    cache = b.cache(mq)
    ws = mq.attn_shared_workspace(cache, 28, 3 * T, 1, T)
    want = b.call(mq, cache, workspace=ws)
    ok_status(mq)
    out = torch.full_like(want, 3.0)
    assert mq.mq_debug_set_fault(mq.MQ_FAULT_WITHHOLD_TILE) == mq.MQ_OK
    try:
        b.call(mq, cache, workspace=ws, out=out)
        torch.cuda.synchronize()
        st = mq.mq_read_device_status(0)
    finally:
        assert mq.mq_debug_set_fault(mq.MQ_FAULT_NONE) == mq.MQ_OK
    assert st == mq.MQ_DEV_TIMEOUT and (out == 3).all()
    ws.zero_()
    assert torch.equal(b.call(mq, cache, workspace=ws), want)
    ok_status(mq)


def test_on_a_given_stream_beside_another_call(cuda_ready):
    # two calls at once, each on its stream with its workspace
    import torch
    mq = cuda_ready
    b = [Batch(np.random.default_rng(i), [(30, [(50, 1 + 3 * i)] * 20)], 28, 4, 128, "q8_0") for i in range(2)]
    caches = [x.cache(mq) for x in b]
    want = [x.call(mq, c) for x, c in zip(b, caches)]
    side = [torch.cuda.Stream() for _ in b]
    ws = [mq.attn_shared_workspace(c, 28, sum(x.new), 1, max(x.new)) for x, c in zip(b, caches)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [x.call(mq, c, workspace=w, stream=s) for x, c, w, s in zip(b, caches, ws, side)]
    torch.cuda.synchronize()
    ok_status(mq)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("T", [1, 2, 40])
@pytest.mark.parametrize("where", ["no pages", "no tokens"])
def test_call_in_which_no_group_has_work_ends_when_its_outputs_are_written(cuda_ready, ctype, T, where):
    # groups without pages, or without tokens beside sequences in no group: the join has no rows, and the own keys'
    # kernel writes all there is.  In a graph the copy behind the call, and the next call in the same workspace, start
    # when the call ends.  (7, 14 and 280 query rows of a key/value head: each of the kernels)
    import torch
    mq = cuda_ready
    own = [(5000, T), (70, T), (2000, T)]
    groups = [(0, own), (0, [(9, T)])] if where == "no pages" else [(0, own), (3, [(9, 0), (70, 0)])]
    b = Batch(np.random.default_rng(T), groups, 28, 4, 128, ctype, lead=where != "no pages")
    cache, n = b.cache(mq), sum(b.new)
    args = (cache, dev(b.q), dev(b.start), dev(np.array(b.ctx, np.int32)), dev(b.grp_start), dev(b.grp_pages))
    kw = dict(mask=dev(as_i64([x for s in b.bits for x in s])), max_len=6000, max_tokens=T, max_pages=4,
              workspace=mq.attn_shared_workspace(cache, 28, n, len(b.grp_pages), T))
    out = torch.empty((n, 28 * 128), dtype=torch.float16, device="cuda")
    got = [torch.empty_like(out) for _ in range(4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        mq.attn_shared(*args, out=out, **kw)
    side.synchronize()
    ok_status(mq)
    b.check(out)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for x in got:
            out.fill_(3.0)
            mq.attn_shared(*args, out=out, **kw)
            x.copy_(out)
    for _ in range(3):
        for x in got:
            x.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in got)
    ok_status(mq)


@pytest.mark.parametrize("T", [1, 2, 40])
@pytest.mark.parametrize("groups", [3, 50])
def test_groups_out_of_order_are_reported_and_write_nothing(cuda_ready, T, groups):
    # two groups over the same sequences, the one between them empty backwards: whose prefix it is cannot be told
    import torch
    mq = cuda_ready
    b = Batch(np.random.default_rng(T), [(2, [(30, T), (5, T)]), (1, [(70, T)])], 8, 2, 64, "f16")
    good = b.grp_start, b.grp_pages
    cache = b.cache(mq)
    ws = mq.attn_shared_workspace(cache, 8, 3 * T, groups, T)
    b.grp_start = np.array([0] * (groups - 2) + [3, 0, 3], np.int32)
    b.grp_pages = np.array([0] * (groups - 3) + [2, 0, 1], np.int32)
    out = torch.full((3 * T, 8 * 64), 3.0, dtype=torch.float16, device="cuda")
    b.call(mq, cache, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert mq.mq_read_device_status(0) == mq.MQ_DEV_KV_RANGE and (out == 3).all()
    b.grp_start, b.grp_pages = good
    b.call(mq, cache, out=out, workspace=ws)
    ok_status(mq)
    b.check(out)
