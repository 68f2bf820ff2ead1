"""Tree attention over the paged cache against a plain 64-bit form.

Bound per output: the result's f16 rounding, 2^-11 |ref|; the probabilities' f16 rounding in the products and in the
sum, 2 * 2^-11 A with A = sum p|v| / sum p; the scores' fp32 error, 2^-19 of the largest sum |q||k| scale, as a
relative error of each probability; and 2^-24 for results below f16's normal range.  A q8_0 result is within half a
step and the roundings of scale and value (127 * 2^-11 steps each) of that.
"""
import numpy as np
import pytest

from tests import kv_plain as P
from tests.test_gpu_kv import dev, ok_status

pytestmark = pytest.mark.gpu


def tree_masks(rng, T):
    m = []
    for i in range(T):
        m.append((m[rng.integers(0, i)] if i else 0) | (1 << i))
    return m


def as_i64(masks):
    return np.array([m - (1 << 64) if m >> 63 else m for m in masks], np.int64)


def bound(ref, A, big):
    return 2**-11 * np.abs(ref) + A * (2**-10 + 2**-19 * big) + 2**-24


def values_of(out, n, width):
    b = out.cpu().numpy().reshape(n, width // 32, 34)
    d = b[..., :2].copy().view(np.float16).astype(np.float64)
    return (b[..., 2:].view(np.int8) * d).reshape(n, width)


def run_case(mq, rng, ctx, new, Hq, Hkv, D, ctype, out_type="f16", masks="tree", scale=None, spread=1.0, offset=0.0,
             q_pad=0, **kw):
    """Random cache and tree, the call, and the comparison; returns the output."""
    S, n = len(ctx), sum(new)
    K = [(rng.standard_normal((c + t, Hkv, D)) * spread + offset).astype(np.float32) for c, t in zip(ctx, new)]
    V = [rng.standard_normal((c + t, Hkv, D)).astype(np.float32) for c, t in zip(ctx, new)]
    pages, table = P.build(K, V, ctype, rng)
    cache = mq.KVCache(dev(pages), dev(table), ctype, Hkv, D)
    q = rng.standard_normal((n, Hq * D + q_pad)).astype(np.float16)
    bits = {"tree": lambda: [tree_masks(rng, t) for t in new],
            "chain": lambda: [[(2 << i) - 1 for i in range(t)] for t in new],
            "random": lambda: [[int(rng.integers(0, 2**63)) & int(rng.integers(0, 2**63)) for _ in range(t)] for t in new],
            "none": lambda: [[0] * t for t in new]}[masks]()
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    m = None if masks == "chain" else dev(as_i64([b for s in bits for b in s]))
    out = mq.attn_tree(cache, dev(q)[:, :Hq * D], dev(start), dev(np.array(ctx, np.int32)), mask=m, scale=scale,
                       max_len=max(c + t for c, t in zip(ctx, new)), max_tokens=max(1, max(new)), out_type=out_type, **kw)
    ok_status(mq)
    got = (out.cpu().numpy().astype(np.float64) if out_type == "f16" else values_of(out, n, Hq * D)).reshape(n, Hq, D)
    for s in range(S):
        a, b = start[s], start[s + 1]
        ref, A, big = P.attention(q[a:b, :Hq * D].reshape(-1, Hq, D), P.stored(K[s], ctype), P.stored(V[s], ctype),
                                  ctx[s], bits[s], D**-0.5 if scale is None else scale)
        tol = bound(ref, A, big)
        if out_type == "q8_0":
            top = (np.abs(ref) + tol).reshape(b - a, Hq, D // 32, 32).max(-1).repeat(32, -1)
            tol = tol + top / 127 * (0.5 + 2 * 127 * 2**-11)
        err = np.abs(got[a:b] - ref)
        assert (err <= tol).all(), (s, ctx[s], new[s], float((err / tol).max()), np.argwhere(err > tol)[:3])
    return out, cache, q, start


HEADS = [(28, 4, 128), (16, 8, 64), (8, 1, 128), (3, 3, 64), (10, 2, 64), (32, 2, 128)]


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_decode_lengths(cuda_ready, ctype, Hq, Hkv, D):
    # one token per sequence; the context empty, inside, at and past page borders
    rng = np.random.default_rng(Hq)
    ctx = [0, 1, 15, 16, 17, 62, 63, 64, 65, 127, 128, 200, 511, 1000]
    run_case(cuda_ready, rng, ctx, [1] * len(ctx), Hq, Hkv, D, ctype, masks="chain")


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("masks", ["tree", "random", "chain"])
def test_trees(cuda_ready, ctype, Hq, Hkv, D, masks):
    # ragged trees, some sequences without tokens; trees that straddle pages
    rng = np.random.default_rng(Hq + D)
    ctx, new = [0, 60, 130, 5, 64, 300, 63], [64, 7, 0, 33, 2, 19, 1]
    run_case(cuda_ready, rng, ctx, new, Hq, Hkv, D, ctype, masks=masks)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 18, 19, 32, 36, 37, 48, 64])
@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
def test_tree_sizes(cuda_ready, ctype, T):
    rng = np.random.default_rng(T)
    run_case(cuda_ready, rng, [333, 50], [T, max(1, T // 2)], 28, 4, 128, ctype)


@pytest.mark.parametrize("T", [1, 5, 20, 64])
@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
def test_rows_that_see_nothing(cuda_ready, ctype, T):
    out, *_ = run_case(cuda_ready, np.random.default_rng(T), [0, 0], [T, 1], 28, 4, 128, ctype, masks="none")
    assert (out == 0).all()


@pytest.mark.parametrize("T", [1, 6, 40])
def test_q8_0_output(cuda_ready, T):
    rng = np.random.default_rng(T + 50)
    for Hq, Hkv, D in [(28, 4, 128), (16, 8, 64)]:
        run_case(cuda_ready, rng, [100, 700, 0], [T, 1, T], Hq, Hkv, D, "q8_0", out_type="q8_0")
    out, *_ = run_case(cuda_ready, rng, [0], [T], 28, 4, 128, "f16", out_type="q8_0", masks="none")
    assert (out == 0).all()


@pytest.mark.parametrize("T", [1, 7, 64])
@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
def test_long_contexts(cuda_ready, ctype, T):
    # enough pages that a head's work is split many ways; scores far apart, so the running maximum moves
    rng = np.random.default_rng(T + 7)
    run_case(cuda_ready, rng, [9000, 2], [T, 1], 14, 2, 64, ctype, spread=6.0, offset=0.7)


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,T", [(14, 2, 128, 1), (16, 2, 64, 1), (14, 2, 128, 2), (14, 2, 64, 2)])
def test_many_pages_per_sm(cuda_ready, ctype, Hq, Hkv, D, T):
    # every SM's ring of pages goes round several times
    run_case(cuda_ready, np.random.default_rng(T), [150000, 3], [T, T], Hq, Hkv, D, ctype)


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
def test_large_scores_and_scales(cuda_ready, ctype):
    rng = np.random.default_rng(77)
    for scale in (0.0, -0.3, 4.0, 1e-6):
        for T in (1, 24):
            run_case(cuda_ready, rng, [150], [T], 28, 4, 128, ctype, scale=scale)


def test_strided_queries_and_output(cuda_ready):
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(5)
    for T in (2, 30):
        full = torch.full((T + 3, 28 * 128 + 8), -9.0, dtype=torch.float16, device="cuda")
        run_case(mq, rng, [90, 20], [T, 3], 28, 4, 128, "q8_0", q_pad=16, out=full[:, :28 * 128])
        assert (full[:, 28 * 128:] == -9).all()


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("T", [1, 4, 20, 64])
def test_what_a_node_does_not_see_never_reaches_it(cuda_ready, ctype, T):
    # NaN and infinities in the keys and values of one branch, and in every slot past the end (build's default)
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(T)
    Hq, Hkv, D, ctx = 28, 4, 128, 100
    for kind in ("k_nan", "k_inf", "v_nan", "v_inf"):
        K = rng.standard_normal((ctx + T, Hkv, D)).astype(np.float32)
        V = rng.standard_normal((ctx + T, Hkv, D)).astype(np.float32)
        Kc, Vc = K.copy(), V.copy()
        j = T // 2
        x = Kc if kind[0] == "k" else Vc
        x[ctx + j, 1, 5] = np.nan if "nan" in kind else np.inf
        with np.errstate(invalid="ignore"):
            pages, table = P.build([Kc], [Vc], ctype, rng)
        cache = mq.KVCache(dev(pages), dev(table), ctype, Hkv, D)
        q = rng.standard_normal((T, Hq * D)).astype(np.float16)
        masks = [(1 << i) | (1 << j if i % 3 == 2 or i == j else 0) for i in range(T)]
        out = mq.attn_tree(cache, dev(q), dev(np.array([0, T], np.int32)), dev(np.array([ctx], np.int32)),
                           mask=dev(as_i64(masks)), max_tokens=T, max_len=ctx + T)
        ok_status(mq)
        got = out.cpu().numpy().reshape(T, Hq, D).astype(np.float64)
        ref, A, big = P.attention(q.reshape(T, Hq, D), P.stored(K, ctype), P.stored(V, ctype), ctx, masks, D**-0.5)
        clean = np.ones((T, Hq, D), bool)
        for i in range(T):
            if (masks[i] >> j) & 1:
                clean[i, 7:14] = False  # the query heads of key/value head 1
        assert (np.abs(got - ref) <= bound(ref, A, big))[clean].all(), kind
        if kind == "v_nan":
            assert all(np.isnan(got[i, 7:14, 5]).all() for i in range(T) if (masks[i] >> j) & 1)
        if kind == "v_inf":
            assert not any(np.isfinite(got[i, 7:14, 5]).any() for i in range(T) if (masks[i] >> j) & 1)


def test_repeated_calls_share_a_workspace_and_agree(cuda_ready):
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(21)
    ws = None
    for T in (1, 64, 5, 30, 1):
        args = ([4000, 100, 2500], [T, 1, T], 28, 4, 128, "q8_0")
        if ws is None:
            cache = mq.KVCache.alloc(1, torch.zeros((3, 100), dtype=torch.int32, device="cuda"), "q8_0", 4, 128)
            ws = mq.attn_workspace(cache, 28, 64)
        a, *_ = run_case(mq, np.random.default_rng(T), *args, workspace=ws)
        b, *_ = run_case(mq, np.random.default_rng(T), *args, workspace=ws)
        assert torch.equal(a, b)


def test_graph_replay_follows_device_lengths(cuda_ready):
    # a captured call: lengths, masks and pages change between replays
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(31)
    Hq, Hkv, D, T = 28, 4, 128, 4
    K = [rng.standard_normal((900, Hkv, D)).astype(np.float32) for _ in range(2)]
    V = [rng.standard_normal((900, Hkv, D)).astype(np.float32) for _ in range(2)]
    pages, table = P.build(K, V, "q8_0", rng)
    cache = mq.KVCache(dev(pages), dev(table), "q8_0", Hkv, D)
    q = dev(rng.standard_normal((2 * T, Hq * D)).astype(np.float16))
    start, ctx = dev(np.array([0, T, 2 * T], np.int32)), dev(np.array([5, 700], np.int32))
    mask = dev(as_i64(tree_masks(rng, T) + tree_masks(rng, T)))
    ws = mq.attn_workspace(cache, Hq, T)
    out = torch.empty((2 * T, Hq * D), dtype=torch.float16, device="cuda")
    call = lambda o, w: mq.attn_tree(cache, q, start, ctx, mask=mask, max_len=904, max_tokens=T, out=o, workspace=w)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(out, ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(out, ws)
    for lens in ([5, 700], [0, 896], [896, 0], [64, 63]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        mask.copy_(dev(as_i64(tree_masks(rng, T) + tree_masks(rng, T))))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        want = torch.empty_like(out)
        call(want, mq.attn_workspace(cache, Hq, T))
        ok_status(mq)
        assert torch.equal(out, want)


def test_bad_device_data_is_skipped_and_reported(cuda_ready):
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(41)
    Hq, Hkv, D = 8, 2, 64
    for T in (1, 40):
        K = [rng.standard_normal((200, Hkv, D)).astype(np.float32) for _ in range(2)]
        pages, table = P.build(K, K, "f16", rng)
        n = 2 * T
        q = dev(rng.standard_normal((n, Hq * D)).astype(np.float16))

        def call(start, ctx, tab, max_len=200, max_tokens=T):
            cache = mq.KVCache(dev(pages), dev(tab), "f16", Hkv, D)
            out = torch.full((n, Hq * D), 3.0, dtype=torch.float16, device="cuda")
            mq.attn_tree(cache, q, dev(np.array(start, np.int32)), dev(np.array(ctx, np.int32)), max_len=max_len,
                         max_tokens=max_tokens, out=out)
            torch.cuda.synchronize()
            return out, mq.mq_read_device_status(0)

        good, st = call([0, T, n], [100, 50], table)
        assert st == 0 and not (good == 3).any()
        # the second sequence is wrong: it stays unwritten and the first is right
        wrong = table.copy()
        wrong[1, 0] = pages.shape[0]
        for start, ctx, tab in (([0, T, n], [100, -1], table), ([0, T, n], [100, 201 - T], table),
                                ([0, T, n], [100, 50], wrong), ([0, T, n + 1], [100, 50], table),
                                ([0, T, T - 1], [100, 50], table), ([0, T, n], [100, 2**31 - 1], table)):
            out, st = call(start, ctx, tab)
            assert st == mq.MQ_DEV_KV_RANGE, (start, ctx)
            assert torch.equal(out[:T], good[:T]) and (out[T:] == 3).all()
        # a length within max_len but past the table
        out, st = call([0, T, n], [100, 64 * table.shape[1] - T + 1], table, max_len=100000)
        assert st == mq.MQ_DEV_KV_RANGE and torch.equal(out[:T], good[:T]) and (out[T:] == 3).all()
        # tokens outside every sequence are not written
        out, st = call([0, T, T], [100, 50], table)
        assert st == 0 and torch.equal(out[:T], good[:T]) and (out[T:] == 3).all()


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,T", [(14, 2, 128, 3), (14, 2, 64, 18), (8, 2, 128, 64), (14, 2, 128, 33), (16, 2, 64, 48)])
def test_many_pages_of_trees(cuda_ready, ctype, Hq, Hkv, D, T):
    # more pages than SMs, of one long sequence (many parts of a group) and short ones; blocks of up to 128 rows and more
    run_case(cuda_ready, np.random.default_rng(T), [20000, 3, 0, 700], [T, T, 1, T // 2], Hq, Hkv, D, ctype)


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("T", [2, 33])
def test_many_sequences(cuda_ready, ctype, T):
    # more groups than SMs: most are one CTA's own, in one kernel's call and in the other's
    rng = np.random.default_rng(T + 5)
    ctx = [int(c) for c in rng.integers(0, 200, 50)]
    run_case(cuda_ready, rng, ctx, [int(t) for t in rng.integers(0, T + 1, 50)], 16, 4, 64, ctype, out_type="q8_0")


@pytest.mark.parametrize("T", [3, 40])
def test_not_finite_values_in_a_q8_0_output(cuda_ready, T):
    # a value that is not finite: the blocks of the rows that see it say so by their scale, the others are untouched
    import torch
    mq, D, Hkv, Hq = cuda_ready, 64, 1, 4
    rng = np.random.default_rng(T)
    ctx = 4000
    K = rng.standard_normal((ctx + T, Hkv, D)).astype(np.float32)
    V = rng.standard_normal((ctx + T, Hkv, D)).astype(np.float32)
    masks = tree_masks(rng, T)
    masks[T - 1] = 1 << (T - 1)
    bad = V.copy()
    bad[ctx + 1, 0, 40] = np.inf  # node 1
    start, lens = dev(np.array([0, T], np.int32)), dev(np.array([ctx], np.int32))
    q = dev(rng.standard_normal((T, Hq * D)).astype(np.float16))
    got = []
    for v in (V, bad):
        pages, table = P.build([K], [v], "f16", np.random.default_rng(1))
        out = mq.attn_tree(mq.KVCache(dev(pages), dev(table), "f16", Hkv, D), q, start, lens, mask=dev(as_i64(masks)),
                           max_len=ctx + T, max_tokens=T, out_type="q8_0")
        got.append(out.cpu().numpy().reshape(T, Hq, D // 32, 34))
    ok_status(mq)
    for i in range(T):
        scale = got[1][i, :, 1, :2].copy().view(np.float16)
        assert np.array_equal(got[0][i, :, 0], got[1][i, :, 0])
        if masks[i] >> 1 & 1:
            assert not np.isfinite(scale).any()
        else:
            assert np.array_equal(got[0][i], got[1][i])


def test_one_workspace_for_batches_that_grow_and_shrink(cuda_ready):
    # a few long sequences, many short ones, other heads, other row counts: each call finds the workspace ready
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(61)
    many = [int(c) for c in rng.integers(100, 700, 64)]
    calls = [([4000, 100, 2500], 28, 4, 128, 1), (many, 28, 4, 128, 1), ([4000, 100, 2500], 28, 4, 128, 1),
             (many[:20], 16, 8, 64, 4), ([3000, 2000], 28, 4, 128, 30), (many, 28, 4, 128, 1), ([5000], 8, 1, 128, 1)]
    size = 0
    for ctx, Hq, Hkv, D, T in calls:
        table = torch.zeros((len(ctx), 1), dtype=torch.int32, device="cuda")
        cache = mq.KVCache.alloc(1, table, "q8_0", Hkv, D)
        size = max(size, mq.attn_workspace(cache, Hq, T).numel())
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for ctx, Hq, Hkv, D, T in calls:
        run_case(mq, rng, ctx, [T] * len(ctx), Hq, Hkv, D, "q8_0", workspace=ws)


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("T", [1, 2, 4, 20, 64])
@pytest.mark.parametrize("ctx", [100, 4000])
def test_an_infinite_value_makes_an_infinite_output(cuda_ready, ctype, T, ctx):
    # on both kernels, in groups of one CTA and of several: a value of a node that is infinite (a q8_0 product that
    # overflows f16), whatever the node weighs, and one of the context that weighs like the others
    mq = cuda_ready
    rng = np.random.default_rng(T + ctx)
    Hq, Hkv, D = 28, 4, 128
    q = (np.abs(rng.standard_normal((T, Hq * D))) + 0.5).astype(np.float16)
    masks = tree_masks(rng, T)
    for kind, slot in (("node", ctx + T // 2), ("faint node", ctx + T // 2), ("context", 5)):
        K = (rng.standard_normal((ctx + T, Hkv, D)) * 0.3).astype(np.float32)
        V = rng.standard_normal((ctx + T, Hkv, D)).astype(np.float32)
        big = np.inf if ctype == "f16" else 7.6e6  # scale 59843, code 127
        V[slot, 1, 5], V[slot, 1, 70] = big, -big
        if kind == "faint node":
            K[slot] = -8.0  # 2^-150 of the others and less: q is positive
        with np.errstate(over="ignore"):
            pages, table = P.build([K], [V], ctype, rng)
            k, v = P.stored(K, ctype), P.stored(V, ctype)
        cache = mq.KVCache(dev(pages), dev(table), ctype, Hkv, D)
        out = mq.attn_tree(cache, dev(q), dev(np.array([0, T], np.int32)), dev(np.array([ctx], np.int32)),
                           mask=dev(as_i64(masks)), max_tokens=T, max_len=ctx + T)
        ok_status(mq)
        got = out.cpu().numpy().reshape(T, Hq, D).astype(np.float64)
        ref, A, largest = P.attention(q.reshape(T, Hq, D), k, v, ctx, masks, D**-0.5)
        assert np.isinf(ref[T // 2, 7:14, 5]).all()
        inf = np.isinf(ref)
        assert np.array_equal(got[inf], ref[inf]), kind
        assert (np.abs(got[~inf] - ref[~inf]) <= bound(ref, A, largest)[~inf]).all(), kind


@pytest.mark.parametrize("handle", [False, True])
def test_calls_on_a_given_stream(cuda_ready, handle):
    # stream= as a torch stream or its handle: work and new outputs are that stream's, behind what it is doing
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(71)
    Hq, Hkv, D, n = 8, 2, 64, 200
    table = dev(np.arange(8, dtype=np.int32).reshape(1, 8))
    cache = mq.KVCache.alloc(8, table, "q8_0", Hkv, D)
    qkv = dev(rng.standard_normal((n, (Hq + 2 * Hkv) * D)).astype(np.float32))
    at = dev(np.arange(n, dtype=np.int32))
    seq, start, ctx = torch.zeros_like(at), dev(np.array([0, 1], np.int32)), dev(np.array([n - 1], np.int32))
    path, one = dev(np.array([[2, 5]], np.int32)), dev(np.array([2], np.int32))
    from_ = dev(np.array([100], np.int32))

    def step(**kw):
        q = mq.kv_append(cache, qkv, None, seq, at, Hq, **kw)
        out = mq.attn_tree(cache, q[-1:], start, ctx, max_len=n, max_tokens=1, **kw)
        mq.kv_accept(cache, from_, path, one, **kw)
        return (q, out) + mq.kv_read(cache, seq, at, **kw)

    want = [t.clone() for t in step()]
    cache.pages.zero_()
    side = torch.cuda.Stream()
    on = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    step(stream=on)  # what has to be loaded is loaded
    torch.cuda.synchronize()
    assert not (cache.pages == 0).all()
    cache.pages.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(1e9))  # some 0.5 s
    got = step(stream=on)
    assert (cache.pages == 0).all()  # on the current stream, which did not wait
    assert not side.query()
    side.synchronize()
    ok_status(mq)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
