"""The key/value cache on the GPU: append (norms, rotation, write), read and accept against plain 64-bit forms.

Bounds: q and f16 keys are one f16 rounding (2^-11 relative) of an fp32 computation whose error is at most 2^-19 of
the row's largest value (norm: a few fp32 roundings; rotation: cosine and sine within 2^-22, two products).  A q8_0
element is within half a step of its value, plus the scale's and the value's f16 roundings (127 * 2^-11 steps each).
What is not computed (values, unrotated keys, reads, moves) is compared bit for bit.
"""
import numpy as np
import pytest

from tests import kv_plain as P

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def cache_of(mq, pages, table, ctype, Hkv, D):
    return mq.KVCache(dev(pages), dev(table), ctype, Hkv, D)


def make(rng, lens, Hkv, D, ctype):
    K = [rng.standard_normal((n, Hkv, D)).astype(np.float32) for n in lens]
    V = [rng.standard_normal((n, Hkv, D)).astype(np.float32) for n in lens]
    return K, V, *P.build(K, V, ctype, rng)


def ok_status(mq, want=0):
    import torch
    torch.cuda.synchronize()
    assert mq.mq_read_device_status(0) == want


HEADS = [(28, 4, 128), (16, 8, 64), (3, 3, 128), (5, 1, 64)]


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("rot,inter,norm,n", [(1.0, False, True, 1), (1.0, True, False, 67), (0.5, False, True, 130),
                                              (0.5, True, True, 3), (0.0, False, False, 70), (6, False, True, 5)])
def test_append(cuda_ready, ctype, Hq, Hkv, D, rot, inter, norm, n):
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(Hq * 1000 + D + n)
    R = rot if isinstance(rot, int) else int(rot * D)
    lens = [200, 65, 1]
    K, V, pages, table = make(rng, lens, Hkv, D, ctype)
    H = Hq + 2 * Hkv
    pad = 6  # a row stride that is not the row's length
    qkv = rng.standard_normal((n, H * D + pad)).astype(np.float32) * 1.5
    qkv[:, ::37] *= 9.0
    qkv[0, :32] = 0.0
    pos = rng.integers(0, 200000, n).astype(np.int32)
    # distinct slots of the first two sequences, some tokens padding
    where = [(0, j) for j in range(190)] + [(1, j) for j in range(64)]
    pick = rng.permutation(len(where))[:n]
    seq = np.array([where[i][0] for i in pick], np.int32)
    slot = np.array([where[i][1] for i in pick], np.int32)
    if n > 2:
        slot[1] = -1
    w_q = rng.uniform(0.5, 1.5, D).astype(np.float32) if norm else None
    w_k = rng.uniform(0.5, 1.5, D).astype(np.float32) if norm else None
    freq = (1e6 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32) if R else None
    cache = cache_of(mq, pages, table, ctype, Hkv, D)
    before = cache.pages.clone()
    x = dev(qkv)[:, :H * D]
    o = {k: (None if v is None else dev(v)) for k, v in dict(q_norm=w_q, k_norm=w_k, inv_freq=freq).items()}
    q = mq.kv_append(cache, x, dev(pos), dev(seq), dev(slot), Hq, interleaved=inter, eps=1e-5, **o)
    ok_status(mq)
    xs = qkv[:, :H * D].reshape(n, H, D)
    ref = P.norm_rope(xs[:, :Hq], w_q, 1e-5, pos, freq, inter)
    row = np.abs(ref).max(-1, keepdims=True)
    got = q.cpu().numpy().reshape(n, Hq, D).astype(np.float64)
    assert (np.abs(got - ref) <= 2**-11 * np.abs(ref) + 2**-19 * row + 2**-24).all()
    # the cache: every written slot, and nothing else
    after = cache.pages.cpu().numpy().reshape(pages.shape)
    kref = P.norm_rope(xs[:, Hq:Hq + Hkv], w_k, 1e-5, pos, freq, inter)
    expect = before.cpu().numpy().reshape(pages.shape).copy()
    at, voff, sc, soff = P.places(ctype, D)
    for i in range(n):
        if slot[i] < 0:
            continue
        p, r = table[seq[i], slot[i] // 64], slot[i] % 64
        for h in range(Hkv):
            k, v = (m[r] for m in P.unpack(after[p, h], ctype, D))
            assert np.array_equal(v.view(np.uint16), P.stored(xs[i, Hq + Hkv + h], ctype).view(np.uint16))
            if not norm and not R:
                assert np.array_equal(k.view(np.uint16), P.stored(xs[i, Hq + h], ctype).view(np.uint16))
            big = np.abs(kref[i, h]).max()
            if ctype == "f16":
                tol = 2**-11 * np.abs(kref[i, h]) + 2**-19 * big + 2**-24
            else:
                step = np.abs(kref[i, h]).reshape(-1, 32).max(-1).repeat(32) / 127
                tol = step * (0.5 + 2 * 127 * 2**-11) + 2**-18 * big
            assert (np.abs(k.astype(np.float64) - kref[i, h]) <= tol).all()
            for vv in (0, 1):
                bytes_ = (at[r] + vv * voff)
                if ctype == "f16":
                    bytes_ = np.concatenate([bytes_, bytes_ + 1])
                else:
                    s = sc[r] + vv * soff
                    bytes_ = np.concatenate([bytes_, s, s + 1])
                expect[p, h, bytes_] = after[p, h, bytes_]
    assert np.array_equal(expect, after)


def test_append_long_positions_and_zero_tokens(cuda_ready):
    # at position 10^6 and beyond a product rounded to fp32 would be off by up to 2^-5 rad
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(3)
    K, V, pages, table = make(rng, [64], 1, 64, "f16")
    cache = cache_of(mq, pages, table, "f16", 1, 64)
    pos = np.array([0, 1, 131071, 1048575, 16777217, 2147483647, -5], np.int32)
    n = len(pos)
    freq = (1e4 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)
    freq[3], freq[5], freq[7] = 3.7, 0.0, 1e-30
    qkv = rng.standard_normal((n, 3 * 64)).astype(np.float32)
    q = mq.kv_append(cache, dev(qkv), dev(pos), dev(np.zeros(n, np.int32)), dev(np.arange(n, dtype=np.int32)), 1,
                     inv_freq=dev(freq))
    ok_status(mq)
    # the definition's angle in extended precision, so that the reference itself loses nothing
    t = (pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)) % (2 * np.longdouble(np.pi))
    if np.finfo(np.longdouble).nmant < 60:
        from fractions import Fraction
        tau = Fraction(6283185307179586476925286766559005768394, 10**39)
        t = np.array([[float(Fraction(int(p)) * Fraction(float(f)) % tau) for f in freq] for p in pos])
    else:
        tau = 2 * np.longdouble("3.14159265358979323846264338327950288")
        t = (pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)) % tau
    t = t.astype(np.float64)
    x = qkv[:, :64].astype(np.float64)
    ref = np.concatenate([x[:, :32] * np.cos(t) - x[:, 32:] * np.sin(t), x[:, 32:] * np.cos(t) + x[:, :32] * np.sin(t)], 1)
    got = q.cpu().numpy().astype(np.float64)
    row = np.abs(x).max(-1, keepdims=True)
    assert (np.abs(got - ref) <= 2**-11 * np.abs(ref) + 2**-19 * row + 2**-24).all()
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert mq.kv_append(cache, dev(qkv)[:0], e, e, e, 1, inv_freq=dev(freq)).shape == (0, 64)
    assert mq.kv_read(cache, e, e)[0].shape == (0, 1, 64)
    ok_status(mq)


def test_append_of_values_that_are_not_finite(cuda_ready):
    # a NaN or an infinity stays within its own block of 32 (q8_0) or element (f16) of its own head and token
    mq = cuda_ready
    rng = np.random.default_rng(4)
    for ctype in ("f16", "q8_0"):
        K, V, pages, table = make(rng, [64], 2, 64, ctype)
        cache = cache_of(mq, pages, table, ctype, 2, 64)
        qkv = rng.standard_normal((3, 5 * 64)).astype(np.float32)
        clean = qkv.copy()
        qkv[1, 3 * 64 + 5] = np.nan   # V of head 0
        qkv[1, 4 * 64 + 40] = np.inf  # V of head 1
        ids = dev(np.arange(3, dtype=np.int32))
        mq.kv_append(cache, dev(qkv), ids, dev(np.zeros(3, np.int32)), ids, 1)
        _, v = mq.kv_read(cache, dev(np.zeros(3, np.int32)), ids)
        ok_status(mq)
        v = v.cpu().numpy()
        want = P.stored(clean[:, 3 * 64:].reshape(3, 2, 64), ctype)
        same = np.ones((3, 2, 64), bool)
        if ctype == "f16":
            same[1, 0, 5] = same[1, 1, 40] = False
        else:
            same[1, 0, :32] = same[1, 1, 32:] = False
        assert np.array_equal(v[same].view(np.uint16), want[same].view(np.uint16))
        assert np.isnan(v[1, 0, 5]) and not np.isfinite(v[1, 1, 40])


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hkv,D", [(4, 128), (8, 64), (1, 64), (3, 128)])
def test_read(cuda_ready, ctype, Hkv, D):
    mq = cuda_ready
    rng = np.random.default_rng(Hkv + D)
    lens = [1, 64, 65, 300]
    K, V, pages, table = make(rng, lens, Hkv, D, ctype)
    cache = cache_of(mq, pages, table, ctype, Hkv, D)
    seq = np.concatenate([np.full(n, s) for s, n in enumerate(lens)]).astype(np.int32)
    slot = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    mix = rng.permutation(len(seq))
    k, v = mq.kv_read(cache, dev(seq[mix]), dev(slot[mix]))
    ok_status(mq)
    for got, src in ((k, K), (v, V)):
        want = P.stored(np.concatenate(src)[mix], ctype)
        assert np.array_equal(got.cpu().numpy().view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hkv,D", [(4, 128), (2, 64)])
def test_accept(cuda_ready, ctype, Hkv, D):
    mq = cuda_ready
    rng = np.random.default_rng(9)
    ctx = [0, 60, 127, 5, 64]
    paths = [[0, 2, 5], list(range(64)), [], [63, 0, 1], [7, 3, 7, 0]]  # overlap, page borders, empty, any order, repeats
    lens = [c + 64 for c in ctx]
    K, V, pages, table = make(rng, lens, Hkv, D, ctype)
    cache = cache_of(mq, pages, table, ctype, Hkv, D)
    path = np.full((5, 64), 99, np.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = p
    mq.kv_accept(cache, dev(np.array(ctx, np.int32)), dev(path), dev(np.array([len(p) for p in paths], np.int32)))
    ok_status(mq)
    after = cache.pages.cpu().numpy().reshape(pages.shape)
    at, voff, sc, soff = P.places(ctype, D)

    def rows(pg, s, j):
        """Every byte of a slot, in the order of the elements."""
        p, r = table[s, j // 64], j % 64
        got = []
        for v in (0, 1):
            b = at[r] + v * voff
            if ctype == "f16":
                got += [pg[p][:, b], pg[p][:, b + 1]]
            else:
                got += [pg[p][:, b], pg[p][:, sc[r] + v * soff], pg[p][:, sc[r] + v * soff + 1]]
        return np.concatenate(got, 1)

    for s, p in enumerate(paths):
        for j in range(lens[s]):
            src = ctx[s] + p[j - ctx[s]] if ctx[s] <= j < ctx[s] + len(p) else j
            assert np.array_equal(rows(after, s, j), rows(pages, s, src)), (s, j)


def test_outside_the_cache_is_skipped_and_reported(cuda_ready):
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(11)
    K, V, pages, table = make(rng, [70, 70], 2, 64, "f16")
    n_pages = pages.shape[0]
    table[1, 1] = n_pages  # a page that does not exist
    cache = cache_of(mq, pages, table, "f16", 2, 64)
    i32 = lambda *v: dev(np.array(v, np.int32))
    qkv = dev(rng.standard_normal((1, 5 * 64)).astype(np.float32))
    before = cache.pages.clone()
    for seq, slot in ((2, 0), (-1, 0), (0, 64 * table.shape[1]), (1, 64), (0, 2**31 - 1)):
        mq.kv_append(cache, qkv, i32(0), i32(seq), i32(slot), 1)
        ok_status(mq, mq.MQ_DEV_KV_RANGE)
        k = torch.full((1, 2, 64), 7.0, dtype=torch.float16, device="cuda")
        v = k.clone()
        mq.kv_read(cache, i32(seq), i32(slot), k_out=k, v_out=v)
        ok_status(mq, mq.MQ_DEV_KV_RANGE)
        assert (k == 7).all() and (v == 7).all()
    for ctx, path, n in ((10, 64, 1), (10, -1, 1), (63, 1, 1), (-1, 0, 1), (10, 0, 2), (2**31 - 1, 0, 1), (10, 0, -1)):
        mq.kv_accept(cache, i32(0, ctx), i32(0, path).view(2, 1), i32(0, n))
        ok_status(mq, mq.MQ_DEV_KV_RANGE)
    assert torch.equal(before, cache.pages)


def test_pages_beyond_4_gib(cuda_ready):
    # page offsets pass 32 bits: the last page of a 5 GB pool
    import torch
    mq = cuda_ready
    Hkv, D = 4, 128
    n_pages = 5 * 2**30 // mq.mq_kv_page_bytes(mq.MQ_TYPE_F16, Hkv, D)
    table = torch.tensor([[n_pages - 1, 0]], dtype=torch.int32, device="cuda")
    cache = mq.KVCache.alloc(n_pages, table, "f16", Hkv, D)
    rng = np.random.default_rng(12)
    qkv = rng.standard_normal((2, 12 * D)).astype(np.float32)
    seq, slot = dev(np.zeros(2, np.int32)), dev(np.array([63, 64], np.int32))
    mq.kv_append(cache, dev(qkv), seq, seq, slot, 4)
    k, v = mq.kv_read(cache, seq, slot)
    ok_status(mq)
    x = qkv.reshape(2, 12, D).astype(np.float16)
    assert np.array_equal(k.cpu().numpy(), x[:, 4:8]) and np.array_equal(v.cpu().numpy(), x[:, 8:])
    at, voff, _, _ = P.places("f16", D)
    tail = cache.pages[-Hkv * P.block_bytes("f16", D):].cpu().numpy().view(np.float16).reshape(Hkv, -1)
    assert np.array_equal(tail[:, at[63] // 2], x[0, 4:8])


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_append_of_many_tokens_is_the_same_as_of_few(cuda_ready, ctype, Hq, Hkv, D):
    # long runs of heads per warp, rows on and off a 16-byte boundary: the same bits as token by token
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(Hq + D)
    n, H = 900, Hq + 2 * Hkv
    x = dev(rng.standard_normal((n, H * D + 2)).astype(np.float32))
    even = x[:, :H * D].contiguous()
    freq = dev((1e5 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
    w = dev(rng.uniform(0.5, 1.5, D).astype(np.float32))
    table = dev(rng.permutation(15).reshape(1, 15).astype(np.int32))
    at = dev(np.arange(n, dtype=np.int32))
    seq = torch.zeros_like(at)
    got = []
    for rows, step in ((x[:, :H * D], n), (even, n), (even, 7)):
        cache = mq.KVCache(torch.zeros(15 * mq.mq_kv_page_bytes(mq.KV_TYPES[ctype], Hkv, D), dtype=torch.uint8,
                                       device="cuda"), table, ctype, Hkv, D)
        q = [mq.kv_append(cache, rows[a:a + step], at[a:a + step], seq[a:a + step], at[a:a + step], Hq, inv_freq=freq,
                          q_norm=w, k_norm=w) for a in range(0, n, step)]
        got.append((torch.cat(q), cache.pages))
    ok_status(mq)
    for q, pages in got[1:]:
        assert torch.equal(q, got[0][0]) and torch.equal(pages, got[0][1])
    ref = P.norm_rope(even.cpu().numpy().reshape(n, H, D)[:, :Hq], w.cpu().numpy(), 1e-6, np.arange(n),
                      freq.cpu().numpy(), False)
    q = got[0][0].cpu().numpy().reshape(n, Hq, D).astype(np.float64)
    assert (np.abs(q - ref) <= 2**-11 * np.abs(ref) + 2**-19 * np.abs(ref).max(-1, keepdims=True) + 2**-24).all()


@pytest.mark.parametrize("ctype,Hkv,D", [("q8_0", 3, 128), ("f16", 5, 64), ("q8_0", 40, 64), ("f16", 20, 128)])
def test_read_of_many_tokens_is_the_same_as_of_few(cuda_ready, ctype, Hkv, D):
    # a read of several chunks per thread; a row of more chunks than a CTA has threads; an odd number of heads
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(Hkv)
    n_pages = 24
    size = mq.mq_kv_page_bytes(mq.KV_TYPES[ctype], Hkv, D)
    pages = dev(rng.integers(0, 120, n_pages * size, dtype=np.uint8))  # high bytes below 0x78: finite f16 values
    cache = mq.KVCache(pages, dev(rng.permutation(n_pages).reshape(2, -1).astype(np.int32)), ctype, Hkv, D)
    n = 70001
    seq, slot = dev(rng.integers(0, 2, n).astype(np.int32)), dev(rng.integers(0, 12 * 64, n).astype(np.int32))
    k, v = mq.kv_read(cache, seq, slot)
    for a in range(0, n, 997):
        ks, vs = mq.kv_read(cache, seq[a:a + 997], slot[a:a + 997])
        assert torch.equal(ks, k[a:a + 997]) and torch.equal(vs, v[a:a + 997])
    ok_status(mq)
    table = cache.table.cpu().numpy()
    blocks = cache.pages.cpu().numpy().reshape(n_pages, Hkv, -1)
    for i in [0, 1, n // 2, n - 1]:
        p, r = table[int(seq[i]), int(slot[i]) // 64], int(slot[i]) % 64
        for h in range(Hkv):
            for got, want in zip((k, v), P.unpack(blocks[p, h], ctype, D)):
                assert np.array_equal(got[i, h].cpu().numpy().view(np.uint16), want[r].view(np.uint16))


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_append_leaves_elements_that_are_not_rotated_alone(cuda_ready, ctype, D, inter):
    # half of the head rotated; in the other half infinities, a NaN and -0 of queries and keys stay where they are
    mq = cuda_ready
    rng = np.random.default_rng(D + inter)
    Hq, Hkv, n, R = 3, 2, 5, D // 2
    K, V, pages, table = make(rng, [64], Hkv, D, ctype)
    cache = cache_of(mq, pages, table, ctype, Hkv, D)
    freq = (1e4 ** (-np.arange(0, R, 2) / R)).astype(np.float32)
    pos = np.arange(7, 7 + n, dtype=np.int32)
    qkv = rng.standard_normal((n, (Hq + 2 * Hkv) * D)).astype(np.float32)
    x = qkv.reshape(n, Hq + 2 * Hkv, D)
    for h in (1, Hq):  # a query and a key head
        x[2, h, R + 2], x[2, h, R + 5], x[2, h, D - 1], x[2, h, D - 4] = np.inf, np.nan, -np.inf, -0.0
    ids = dev(np.arange(n, dtype=np.int32))
    q = mq.kv_append(cache, dev(qkv), dev(pos), dev(np.zeros(n, np.int32)), ids, Hq, inv_freq=dev(freq), interleaved=inter)
    k, _ = mq.kv_read(cache, dev(np.zeros(n, np.int32)), ids)
    ok_status(mq)
    q, k = q.cpu().numpy().reshape(n, Hq, D), k.cpu().numpy()
    assert np.array_equal(q[..., R:], x[:, :Hq, R:].astype(np.float16), equal_nan=True)
    assert np.signbit(q[2, 1, D - 4]) and q[2, 1, D - 4] == 0
    assert np.isfinite(q[..., :R]).all() and np.isfinite(k[..., :R]).all()
    if ctype == "f16":
        assert np.array_equal(k[..., R:], x[:, Hq:Hq + Hkv, R:].astype(np.float16), equal_nan=True)
    else:
        same = np.ones((n, Hkv, D), bool)
        same[2, 0, R:] = False  # the blocks with values that are not finite
        want = P.stored(x[:, Hq:Hq + Hkv], ctype)
        same[..., :R] = False
        assert np.array_equal(k[same], want[same])


@pytest.mark.parametrize("inter,R", [(False, 64), (True, 64), (False, 32)])
def test_append_with_frequencies_that_have_no_angle(cuda_ready, inter, R):
    # NaN, an infinity or 2^64 and more in inv_freq: NaN in the pairs that it turns, and nowhere else
    mq = cuda_ready
    rng = np.random.default_rng(R + inter)
    n, D = 3, 64
    K, V, pages, table = make(rng, [64], 1, D, "f16")
    cache = cache_of(mq, pages, table, "f16", 1, D)
    freq = (1e4 ** (-np.arange(0, R, 2) / R)).astype(np.float32)
    bad = {3: np.nan, 7: np.inf, 9: -np.inf, 11: np.float32(2.0**64)}
    for i, f in bad.items():
        freq[i] = f
    freq[5] = 2.0**63  # the largest binade that is taken
    pos = np.array([0, 1, 131071], np.int32)
    qkv = rng.standard_normal((n, 3 * D)).astype(np.float32)
    ids = dev(np.arange(n, dtype=np.int32))
    q = mq.kv_append(cache, dev(qkv), dev(pos), dev(np.zeros(n, np.int32)), ids, 1, inv_freq=dev(freq), interleaved=inter)
    k, _ = mq.kv_read(cache, dev(np.zeros(n, np.int32)), ids)
    ok_status(mq)
    i = np.array(list(bad))
    pair = np.concatenate([2 * i, 2 * i + 1] if inter else [i, i + R // 2])
    nan = np.zeros(D, bool)
    nan[pair] = True
    for x in (q.cpu().numpy(), k.cpu().numpy()[:, 0]):
        assert (np.isnan(x) == nan).all()
