"""Verification of drafted trees against a walk in exact rational arithmetic (probabilities are fp32, so rationals),
bit for bit, and against the target's distribution."""
from fractions import Fraction as F

import numpy as np
import pytest

from tests.test_gpu_kv import dev, ok_status

pytestmark = pytest.mark.gpu


def walk(target, draft, token, parent, u, path_ld, greedy=False):
    """One tree: rows of its nodes; returns (path, next)."""
    T, V = target.shape
    path, i = [0], 0
    while True:
        kids = [c for c in range(1, T) if parent[c] == i and 0 <= token[c] < V and 0 <= parent[c] < c]
        if len(path) >= path_ld:
            kids = []
        if greedy:
            row = np.where(np.isnan(target[i]), -np.inf, target[i])
            best = int(row.argmax()) if row.max() > -np.inf else -1
            go = next((c for c in kids if token[c] == best), None)
            if go is None:
                return path, best
        else:
            p = [F(float(v)) for v in target[i]]
            q = [F(float(v)) for v in draft[i]] if draft is not None else None
            S, W, go, a = list(p), F(1), None, F(0)
            for c in kids:
                x = token[c]
                if S[x] > 0 and F(float(u[c])) * (q[x] if q else 1) * W < S[x]:
                    go = c
                    break
                if q:
                    a += W
                    S = [max(pv - a * qv, F(0)) for pv, qv in zip(p, q)]
                    W = sum(S)
                else:
                    W -= S[x]
                    S[x] = F(0)
            if go is None:
                if sum(S) == 0:
                    S = p
                mark, run = F(float(u[0])) * sum(S), F(0)
                if sum(S) == 0:
                    return path, -1
                for j, v in enumerate(S):
                    run += v
                    if run > mark:
                        return path, j
        path.append(go)
        i = go


def tree(rng, T, wide=4):
    return [0][:T] + [int(rng.integers(max(0, i - wide), i)) for i in range(1, T)]


def probabilities(rng, n, V, spread=2.5):
    z = rng.standard_normal((n, V)) * spread
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def batch(rng, sizes, V, near, lookup=False, wide=4):
    n = sum(sizes)
    target = probabilities(rng, n, V)
    draft = None
    if not lookup:
        d = np.log(target.astype(np.float64)) + near * rng.standard_normal((n, V))
        e = np.exp(d - d.max(-1, keepdims=True))
        draft = (e / e.sum(-1, keepdims=True)).astype(np.float32)
    start = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    parent = np.concatenate([tree(rng, t, wide) for t in sizes] + [[]]).astype(np.int32)
    token = np.zeros(n, np.int32)
    for s, t in enumerate(sizes):
        for i in range(t):
            row = (target if draft is None else draft)[start[s] + parent[start[s] + i]].astype(np.float64)
            token[start[s] + i] = rng.choice(V, p=row / row.sum())
    u = rng.random(n, dtype=np.float32)
    return target, draft, start, token, parent, u


def compare(mq, target, draft, start, token, parent, u, path_ld, greedy=False):
    path, n_path, last = mq.verify_tree(dev(target), dev(start), dev(token), dev(parent), u=None if u is None else dev(u),
                                        draft=None if draft is None else dev(draft), greedy=greedy, path_ld=path_ld)
    ok_status(mq)
    path, n_path, last = path.cpu().numpy(), n_path.cpu().numpy(), last.cpu().numpy()
    lens = []
    for s in range(len(start) - 1):
        a, b = start[s], start[s + 1]
        if a == b:
            assert n_path[s] == 0 and last[s] == -1 and (path[s] == 0).all()
            continue
        want, tok = walk(target[a:b], None if draft is None else draft[a:b], token[a:b], parent[a:b],
                         None if u is None else u[a:b], path_ld, greedy)
        assert n_path[s] == len(want) and path[s, :len(want)].tolist() == want, (s, path[s], want)
        assert last[s] == tok and (path[s, len(want):] == 0).all(), (s, last[s], tok)
        lens.append(len(want))
    return lens


@pytest.mark.parametrize("V", [1, 2, 31, 512, 513, 1000, 2049, 4100, 16384, 20001])
@pytest.mark.parametrize("mode", ["draft", "lookup"])
def test_trees(cuda_ready, V, mode):
    rng = np.random.default_rng(V)
    sizes = [1, 7, 0, 16, 2, 5] if V < 4000 else [9, 3]
    args = batch(rng, sizes, V, 0.5, mode == "lookup")
    compare(cuda_ready, *args, path_ld=64)


@pytest.mark.parametrize("mode", ["draft", "lookup"])
def test_bushes_are_refused_many_times(cuda_ready, mode):
    # every node a child of the root, 63 of them; few tokens, so that drafts repeat and the residual runs out
    rng = np.random.default_rng(9)
    for V, near in ((6, 3.0), (50, 4.0), (1500, 6.0)):
        target, draft, start, token, parent, u = batch(rng, [64, 64, 33], V, near, mode == "lookup")
        parent[:] = 0
        token = np.concatenate([rng.integers(0, V, 64), rng.choice(V, 97)]).astype(np.int32)
        u[:] = rng.uniform(0.9, 0.99999, u.shape).astype(np.float32)
        compare(cuda_ready, target, draft, start, token, parent, u, path_ld=3)


def test_chains_and_path_limits(cuda_ready):
    rng = np.random.default_rng(11)
    target, draft, start, token, parent, u = batch(rng, [64, 20, 5], 300, 0.05)
    for a, b in zip(start[:-1], start[1:]):
        parent[a:b] = np.maximum(np.arange(b - a) - 1, 0)
    u[:] *= 0.8
    u[start[:-1]] = rng.random(3, dtype=np.float32)
    for limit in (1, 2, 7, 64):
        lens = compare(cuda_ready, target, draft, start, token, parent, u, path_ld=limit)
        assert max(lens) <= limit
    assert max(lens) > 3


def test_borders_are_exact(cuda_ready):
    # probabilities and numbers that meet exactly: a test is strict, and the running sum passes the mark
    V = 1024
    p = np.full((2, V), 2.0**-10, np.float32)
    q = np.full((2, V), 2.0**-10, np.float32)
    q[0, :512], q[0, 512:] = 2.0**-9, 0.0
    start, parent = np.array([0, 2], np.int32), np.array([0, 0], np.int32)
    for tok in (3, 700):
        for uc in (0.5, np.nextafter(np.float32(0.5), np.float32(0)), 0.0, 0.99):
            for ur in (0.0, 0.25, 0.5, np.nextafter(np.float32(0.5), np.float32(0)), np.float32(1 - 2**-24), 2.0**-30):
                u = np.array([ur, uc], np.float32)
                for d in (q, None):
                    compare(cuda_ready, p, d, start, np.array([0, tok], np.int32), parent, u, path_ld=4)


def test_rows_without_mass_and_odd_numbers(cuda_ready):
    mq = cuda_ready
    V = 700
    start, parent, token = np.array([0, 2, 4, 6, 8], np.int32), np.zeros(8, np.int32), np.full(8, 5, np.int32)
    p = np.zeros((8, V), np.float32)
    p[2] = p[3] = 1.0 / V                   # equal to the draft: refused at u = 1, the residual is empty
    p[4, 7], p[4, 9] = 1.0, np.nan          # a value that is no number counts as nothing
    p[6, 600] = -1.0
    p[6, 601] = 2.0**-140                   # below 2^-60: nothing
    q = np.full((8, V), 1.0 / V, np.float32)
    u = np.array([0.5, 0.5, 0.5, 1.0, 0.9, 0.9, 0.3, 0.2], np.float32)
    path, n_path, last = mq.verify_tree(dev(p), dev(start), dev(token), dev(parent), u=dev(u), draft=dev(q), path_ld=2)
    ok_status(mq)
    assert n_path.tolist() == [1, 1, 1, 1]
    assert last.tolist()[0] == -1 and last.tolist()[1] in (349, 350) and last.tolist()[2:] == [7, -1]
    # numbers outside [0, 1): in range all the same
    for v in (1.0, 2.0, np.nan, -1.0, np.inf):
        _, n_path, last = mq.verify_tree(dev(p[2:4]), dev(start[:2]), dev(token[:2]), dev(parent[:2]),
                                         u=dev(np.full(2, v, np.float32)), draft=dev(q[2:4]), path_ld=2)
        ok_status(mq)
        assert 0 <= int(last) < V and 1 <= int(n_path) <= 2


@pytest.mark.parametrize("V", [1, 33, 5000, 40001])
def test_greedy(cuda_ready, V):
    rng = np.random.default_rng(V + 1)
    sizes = [16, 1, 0, 7, 3]
    target, _, start, token, parent, _ = batch(rng, sizes, V, 0.0, lookup=True)
    logits = np.round(np.log(target) * 4) / 4  # ties
    logits[3, rng.random(V) < 0.5] = np.nan
    logits[start[3]] = -np.inf
    for s in range(len(sizes)):  # half of the drafts are the best ones
        for i in range(start[s] + 1, start[s + 1]):
            if i % 2:
                r = np.where(np.isnan(logits[start[s] + parent[i]]), -np.inf, logits[start[s] + parent[i]])
                token[i] = r.argmax()
    lens = compare(cuda_ready, logits.astype(np.float32), None, start, token, parent, None, path_ld=16, greedy=True)
    assert max(lens) > 1
    zeros = np.array([[-0.0, 0.0, -1.0, -0.0]], np.float32)[:, :max(1, min(4, V))]
    _, _, last = cuda_ready.verify_tree(dev(zeros), dev(np.array([0, 1], np.int32)), dev(np.zeros(1, np.int32)),
                                        dev(np.zeros(1, np.int32)), greedy=True)
    assert int(last) == 0  # the lowest of equals


def test_strides_and_alignment(cuda_ready):
    rng = np.random.default_rng(17)
    V = 9000
    target, draft, start, token, parent, u = batch(rng, [6, 4], V, 0.5)
    want = None
    for off, pad in ((0, 0), (0, 4), (1, 0), (2, 3), (3, 8)):
        import torch
        wide = [torch.full((10, V + off + pad), float("nan"), device="cuda") for _ in range(2)]
        for w, x in zip(wide, (target, draft)):
            w[:, off:off + V] = dev(x)
        got = cuda_ready.verify_tree(wide[0][:, off:off + V], dev(start), dev(token), dev(parent), u=dev(u),
                                     draft=wide[1][:, off:off + V], path_ld=8)
        ok_status(cuda_ready)
        want = got if want is None else want
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bad_device_data_is_skipped_and_reported(cuda_ready):
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(19)
    target, draft, start, token, parent, u = batch(rng, [5, 5, 5], 200, 0.2)

    def call(st=start, tok=token, par=parent):
        path = torch.full((3, 5), 9, dtype=torch.int32, device="cuda")
        n, last = (torch.full((3,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
        mq.verify_tree(dev(target), dev(np.asarray(st, np.int32)), dev(tok), dev(par), u=dev(u), draft=dev(draft), path=path,
                       n_path=n, next_token=last)
        torch.cuda.synchronize()
        return path.cpu().numpy(), n.cpu().numpy(), last.cpu().numpy(), mq.mq_read_device_status(0)

    good = call()
    assert good[3] == 0
    for st in ([0, 5, 16, 15], [0, 5, 4, 15], [0, 5, 10, 2**31 - 1], [-1, 5, 10, 15]):
        got = call(st)
        assert got[3] == mq.MQ_DEV_KV_RANGE
        for s in range(3):
            if 0 <= st[s] <= st[s + 1] <= 15:
                if (st[s], st[s + 1]) == (start[s], start[s + 1]):
                    assert got[1][s] == good[1][s] and got[2][s] == good[2][s]
            else:
                assert got[1][s] == 9 and got[2][s] == 9 and (got[0][s] == 9).all()
    for what, bad in (("token", 200), ("token", -1), ("parent", 4), ("parent", -1), ("parent", 2**31 - 1)):
        tok, par = token.copy(), parent.copy()
        for i in range(1, 5):
            (tok if what == "token" else par)[5 + i] = bad
        got = call(start, tok, par)
        assert got[3] == mq.MQ_DEV_KV_RANGE and got[1][1] == 1
        assert got[1][0] == good[1][0] and got[1][2] == good[1][2]


def test_what_comes_out_is_distributed_as_the_target(cuda_ready):
    # the token behind the root, accepted or drawn, over many trees: 6 standard deviations
    mq = cuda_ready
    rng = np.random.default_rng(23)
    V, S, T = 8, 4096, 4
    p, q = probabilities(rng, 1, V, 1.0)[0], probabilities(rng, 1, V, 1.0)[0]
    target, start = np.tile(p, (S * T, 1)), (np.arange(S + 1) * T).astype(np.int32)
    parent = np.tile(np.array([0, 0, 0, 0], np.int32), S)
    for draft in (np.tile(q, (S * T, 1)), None):
        token = rng.choice(V, S * T, p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)
        path, n, last = mq.verify_tree(dev(target), dev(start), dev(token), dev(parent),
                                       u=dev(rng.random(S * T, dtype=np.float32)),
                                       draft=None if draft is None else dev(draft), path_ld=2)
        ok_status(mq)
        path, n, last = path.cpu().numpy(), n.cpu().numpy(), last.cpu().numpy()
        out = np.where(n == 2, token[np.arange(S) * T + path[:, 1]], last)
        assert (n == 2).sum() > S // 4 and (n == 1).sum() > 10
        seen = np.bincount(out, minlength=V) / S
        assert (np.abs(seen - p) <= 6 * np.sqrt(p * (1 - p) / S)).all(), (draft is None, seen, p)


def test_large_vocabulary_in_many_tiles(cuda_ready):
    # one value above the rest at a time, at the borders of tiles and parts: greedy and a draw find it
    import torch
    mq = cuda_ready
    V = 5_000_011
    x = torch.full((1, V), 1e-12, device="cuda")
    start, zero = dev(np.array([0, 1], np.int32)), dev(np.zeros(1, np.int32))
    for i in (0, 511, 512, 16383, 625001, 625152, 2_500_000, V - 2, V - 1):
        x[0, i] = 0.9
        for kw in (dict(greedy=True), dict(u=dev(np.array([0.5], np.float32)))):
            _, _, last = mq.verify_tree(x, start, zero, zero, **kw)
            assert int(last) == i, (i, kw)
        x[0, i] = 1e-12
    ok_status(mq)


@pytest.mark.parametrize("handle", [False, True])
def test_on_a_given_stream_and_captured(cuda_ready, handle):
    # behind what the stream is doing; a captured call follows the numbers
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(29)
    target, draft, start, token, parent, u = batch(rng, [9, 4, 16], 3000, 0.5)
    d = dict(target=dev(target), draft=dev(draft), start=dev(start), token=dev(token), parent=dev(parent), u=dev(u))
    call = lambda **k: mq.verify_tree(d["target"], d["start"], d["token"], d["parent"], u=d["u"], draft=d["draft"], path_ld=8, **k)
    want = call()
    side = torch.cuda.Stream()
    on = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(2e8))
    got = call(stream=on)
    assert not side.query()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(stream=on, path=got[0], n_path=got[1], next_token=got[2])
    for _ in range(3):
        d["u"].uniform_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, call()))
    ok_status(mq)


@pytest.mark.parametrize("mode", ["draft", "lookup"])
def test_odd_numbers_at_drafted_tokens(cuda_ready, mode):
    # NaN, infinities, negative and large values where a child is tested: the same numbers there as in the sums
    mq = cuda_ready
    rng = np.random.default_rng(31)
    odd = np.array([np.nan, np.inf, -np.inf, -0.5, -2.0**-20, 3.0, 1.5, -0.0], np.float32)
    clean = lambda x: None if x is None else np.clip(np.where(np.isnan(x), 0, x), 0, 1).astype(np.float32)
    ends = set()
    for V in (5, 40, 700):
        sizes = [16] * 24
        target, draft, start, token, parent, u = batch(rng, sizes, V, 2.0, mode == "lookup")
        for s, t in enumerate(sizes):
            for i in range(1, t):
                row = start[s] + parent[start[s] + i]
                if rng.random() < 0.4:
                    target[row, token[start[s] + i]] = rng.choice(odd)
                if draft is not None and rng.random() < 0.4:
                    draft[row, token[start[s] + i]] = rng.choice(odd)
        path, n_path, last = (x.cpu().numpy() for x in mq.verify_tree(
            dev(target), dev(start), dev(token), dev(parent), u=dev(u), draft=None if draft is None else dev(draft), path_ld=16))
        ok_status(mq)
        P, Q = clean(target), clean(draft)
        for s in range(len(sizes)):
            a, b = start[s], start[s + 1]
            want, tok = walk(P[a:b], None if Q is None else Q[a:b], token[a:b], parent[a:b], u[a:b], 16)
            assert path[s, :n_path[s]].tolist() == want and last[s] == tok, (V, s, path[s], want, last[s], tok)
            ends.add(len(want))
    assert len(ends) > 2


@pytest.mark.parametrize("V", [2**17 + 4099, 2**18 - 1, 2**18, 2**18 + 4099])
def test_rows_that_sum_to_too_much(cuda_ready, V):
    # 2^17 - 1 is drawn from, exactly; from 2^17 on a row holds no probabilities: the walk ends there, and says so
    import torch
    mq = cuda_ready
    start, zero2 = dev(np.array([0, 2], np.int32)), dev(np.zeros(2, np.int32))
    target = torch.zeros((2, V), device="cuda")
    token = dev(np.array([0, V - 1], np.int32))
    draft = torch.zeros((2, V), device="cuda")
    for ones in (2**17 - 1, 2**17, min(2**18, V - 1), V - 1):
        for value in (1.0, 7.0):  # above 1 is 1
            target[:] = 0
            target[0, 1:1 + ones] = value
            target[0, V - 1] = 0  # the child's: refused
            held = min(ones, V - 2)
            for u0 in (0.0, 0.5, 1 - 2.0**-24):
                for d in (None, draft):
                    path, n_path, last = mq.verify_tree(target, start, token, zero2, u=dev(np.array([u0, 0.5], np.float32)),
                                                        draft=d, path_ld=4)
                    torch.cuda.synchronize()
                    st = mq.mq_read_device_status(0)
                    assert path.tolist() == [[0, 0, 0, 0]] and n_path.tolist() == [1]
                    if held < 2**17:
                        assert st == 0 and int(last) == 1 + int(u0 * held), (ones, u0)
                    else:
                        assert st == mq.MQ_DEV_KV_RANGE and int(last) == -1, (ones, u0)
    # the largest vocabulary, all ones
    if V == 2**18 and torch.cuda.mem_get_info()[0] > 3 * 2**30:
        target = torch.ones((1, 2**28), device="cuda")
        _, _, last = mq.verify_tree(target, start[:1].repeat(2) + dev(np.array([0, 1], np.int32)), zero2[:1], zero2[:1],
                                    u=dev(np.array([0.5], np.float32)))
        torch.cuda.synchronize()
        assert mq.mq_read_device_status(0) == mq.MQ_DEV_KV_RANGE and int(last) == -1


def walk_64(target, draft, token, parent, u, path_ld):
    """walk() of rows on the GPU in fp64: the sums are off by some 2^-50, which changes a draw about never."""
    import torch
    path, i = [0], 0
    while True:
        kids = [c for c in range(1, len(token)) if parent[c] == i] if len(path) < path_ld else []
        p, q = target[i].double(), None if draft is None else draft[i].double()
        S, W, a, go = p.clone(), 1.0, 0.0, None
        for c in kids:
            x = token[c]
            if float(S[x]) > 0 and float(u[c]) * (1.0 if q is None else float(q[x])) * W < float(S[x]):
                go = c
                break
            if q is None:
                W -= float(S[x])
                S[x] = 0
            else:
                a += W
                S = (p - a * q).clamp(min=0)
                W = float(S.sum())
        if go is None:
            S = S if float(S.sum()) > 0 else p
            run = S.cumsum(0)
            return path, int(torch.searchsorted(run, float(u[0]) * run[-1], right=True))
        path.append(go)
        i = go


@pytest.mark.parametrize("seqs,V", [(9, 40000), (9, 131072), (9, 151936), (10, 131072), (20, 131071), (3, 262147),
                                    (1, 9_000_011), (10, 4_500_003)])
@pytest.mark.parametrize("mode", ["draft", "lookup"])
def test_large_vocabularies(cuda_ready, seqs, V, mode):
    # clusters of sixteen (up to 9 sequences) and of eight; tiles of several units (the last two)
    import torch
    mq = cuda_ready
    torch.manual_seed(V)
    rng = np.random.default_rng(V)
    sizes = [6] * seqs if V < 10**6 else [3] * seqs
    n = sum(sizes)
    x = torch.randn((n, V), device="cuda") * 2.5
    target = torch.softmax(x, -1)
    draft = torch.softmax(x.add_(0.7 * torch.randn((n, V), device="cuda")), -1) if mode == "draft" else None
    del x
    start = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    parent = np.concatenate([tree(rng, t, 3) for t in sizes]).astype(np.int32)
    up = [int(start[s]) + int(parent[start[s] + i]) for s, t in enumerate(sizes) for i in range(t)]
    source = target if draft is None else draft
    token = np.array([int(torch.searchsorted(source[r].double().cumsum(0), rng.random())) for r in up], np.int32).clip(0, V - 1)
    refused = 0
    for case in range(4):
        u = rng.random(n, dtype=np.float32)
        if case >= 2:
            u[:] = 0.999
            u[start[:-1]] = rng.random(seqs, dtype=np.float32)
        if case == 3:  # tokens that the draft likes better than the target: every child is refused at first
            for i, r in enumerate(up):
                token[i] = int((target[r] if draft is None else target[r] - draft[r]).argmin())
        path, n_path, last = (v.cpu().numpy() for v in mq.verify_tree(
            target, dev(start), dev(token), dev(parent), u=dev(u), draft=draft, path_ld=6))
        ok_status(mq)
        for s in range(seqs):
            a, b = start[s], start[s + 1]
            want, tok = walk_64(target[a:b], None if draft is None else draft[a:b], token[a:b].tolist(), parent[a:b].tolist(),
                                u[a:b], 6)
            assert path[s, :n_path[s]].tolist() == want and last[s] == tok, (s, path[s], want, last[s], tok)
            refused += len(want) == 1
    assert refused
