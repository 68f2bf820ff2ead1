"""Shared-prefix attention, softmax, verification and page pool on the host: sizes, and refusals before anything
reaches CUDA."""
import ctypes

import pytest

from tests.test_kv_host import attn, cache


def groups(m, **kw):
    f = dict(grp_start=0x6000, grp_pages=0x7000, n_groups=2, max_pages=2)
    f.update(kw)
    return m.AttnGroups(*[f[n] for n, _ in m.AttnGroups._fields_])


def verify(m, **kw):
    f = dict(target=0x1000, draft=0x2000, tok_start=0x3000, token=0x4000, parent=0x5000, u=0x6000, path=0x7000,
             n_path=0x8000, next=0x9000, target_ld=1000, draft_ld=1000, n_tokens=8, n_seqs=2, vocab=1000, path_ld=4,
             flags=0, reserved=0)
    f.update(kw)
    return m.VerifyArgs(*[f[n] for n, _ in m.VerifyArgs._fields_])


def pool(m, **kw):
    f = dict(refs=0x1000, free_list=0x2000, n_free=0x3000, seq_pages=0x4000, scratch=0x5000)
    f.update(kw)
    return m.KvPoolStruct(*[f[n] for n, _ in m.KvPoolStruct._fields_])


def test_struct_sizes(mq_lib):
    assert ctypes.sizeof(mq_lib.AttnGroups) == 2 * 8 + 2 * 4
    assert ctypes.sizeof(mq_lib.VerifyArgs) == 11 * 8 + 6 * 4
    assert ctypes.sizeof(mq_lib.KvPoolStruct) == 5 * 8


def test_attn_shared_checks(mq_lib):
    m = mq_lib
    c = cache(m)
    call = lambda a, g, ws=0x9000, n=2**50: m._lib.mq_attn_shared(c, a, g, ws, n, 0)
    # what mq_attn_tree refuses
    for kw, st in ((dict(n_heads=27), m.MQ_ERR_SHAPE), (dict(max_tokens=65), m.MQ_ERR_SHAPE),
                   (dict(q_ld=28 * 128 + 4), m.MQ_ERR_SHAPE), (dict(out_type=m.MQ_TYPE_Q4_0), m.MQ_ERR_INVALID_ARG),
                   (dict(scale=float("nan")), m.MQ_ERR_INVALID_ARG), (dict(q=0), m.MQ_ERR_INVALID_ARG),
                   (dict(q=0x1008), m.MQ_ERR_ALIGN), (dict(n_tokens=0, q=0), m.MQ_OK)):
        assert call(attn(m, **kw), groups(m)) == st, kw
    for kw, st in ((dict(n_groups=-1), m.MQ_ERR_SHAPE), (dict(max_pages=-1), m.MQ_ERR_SHAPE),
                   (dict(n_groups=5000), m.MQ_ERR_UNSUPPORTED), (dict(grp_start=0), m.MQ_ERR_INVALID_ARG),
                   (dict(grp_pages=0), m.MQ_ERR_INVALID_ARG), (dict(grp_start=0x6002), m.MQ_ERR_ALIGN),
                   (dict(grp_pages=0x7001), m.MQ_ERR_ALIGN),
                   (dict(n_groups=4096, max_pages=2**17), m.MQ_ERR_UNSUPPORTED)):
        assert call(attn(m), groups(m, **kw)) == st, kw
    assert call(attn(m), groups(m), ws=0x9010) == m.MQ_ERR_ALIGN
    assert call(attn(m), None) == m.MQ_ERR_INVALID_ARG
    assert call(None, groups(m)) == m.MQ_ERR_INVALID_ARG
    # query rows are divided by the heads of a group with 32-bit factors: 64 tokens * 1024^2 heads, and 4096
    one = cache(m, n_kv_heads=1)
    wide = dict(n_heads=1024, q_ld=2**17, out_ld=2**17)
    assert m._lib.mq_attn_shared(one, attn(m, n_tokens=4096, **wide), groups(m), 0x9000, 2**50, 0) == m.MQ_ERR_UNSUPPORTED
    assert m._lib.mq_attn_shared(one, attn(m, n_tokens=4095, **wide), groups(m, grp_start=0), 0x9000, 2**50, 0) \
        == m.MQ_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    size = lambda *a: m._lib.mq_attn_shared_workspace_bytes(c, *a, ctypes.byref(n))
    assert size(28, -1, 1, 1) == m.MQ_ERR_SHAPE and size(28, 1, 0, 1) == m.MQ_ERR_SHAPE
    assert size(28, 1, 1, -1) == m.MQ_ERR_SHAPE and size(28, 1, 1, 5000) == m.MQ_ERR_UNSUPPORTED
    assert m._lib.mq_attn_shared_workspace_bytes(c, 28, 1, 1, 1, None) == m.MQ_ERR_INVALID_ARG


def test_softmax_checks(mq_lib):
    m = mq_lib
    for a, st in (((0x1000, 0x2000, -1, 8, 8, 8, 1.0), m.MQ_ERR_SHAPE), ((0x1000, 0x2000, 1, -1, 8, 8, 1.0), m.MQ_ERR_SHAPE),
                  ((0x1000, 0x2000, 1, 8, 7, 8, 1.0), m.MQ_ERR_SHAPE), ((0x1000, 0x2000, 1, 8, 8, 7, 1.0), m.MQ_ERR_SHAPE),
                  ((0x1000, 0x2000, 1, 8, 8, 8, 0.0), m.MQ_ERR_INVALID_ARG),
                  ((0x1000, 0x2000, 1, 8, 8, 8, -1.0), m.MQ_ERR_INVALID_ARG),
                  ((0x1000, 0x2000, 1, 8, 8, 8, float("nan")), m.MQ_ERR_INVALID_ARG),
                  ((0x1000, 0x2000, 1, 8, 8, 8, float("inf")), m.MQ_ERR_INVALID_ARG),
                  ((0x1000, 0x2000, 1, 8, 8, 8, 3e38), m.MQ_ERR_INVALID_ARG),
                  ((0, 0x2000, 1, 8, 8, 8, 1.0), m.MQ_ERR_INVALID_ARG), ((0x1000, 0, 1, 8, 8, 8, 1.0), m.MQ_ERR_INVALID_ARG),
                  ((0x1000, 0x1000, 2, 8, 8, 9, 1.0), m.MQ_ERR_INVALID_ARG),
                  ((0x1002, 0x2000, 1, 8, 8, 8, 1.0), m.MQ_ERR_ALIGN), ((0x1000, 0x2001, 1, 8, 8, 8, 1.0), m.MQ_ERR_ALIGN),
                  ((0x1000, 0x2000, 1, 2**28 + 1, 2**29, 2**29, 1.0), m.MQ_ERR_UNSUPPORTED),
                  ((0x1000, 0x2000, 2**24 + 1, 8, 8, 8, 1.0), m.MQ_ERR_UNSUPPORTED),
                  ((0, 0, 0, 8, 8, 8, 1.0), m.MQ_OK), ((0, 0, 8, 0, 8, 8, 1.0), m.MQ_OK)):
        assert m.mq_softmax(*a) == st, a


def test_verify_checks(mq_lib):
    m = mq_lib
    for kw, st in ((dict(n_tokens=-1), m.MQ_ERR_SHAPE), (dict(n_seqs=-1), m.MQ_ERR_SHAPE), (dict(vocab=0), m.MQ_ERR_SHAPE),
                   (dict(path_ld=0), m.MQ_ERR_SHAPE), (dict(target_ld=999), m.MQ_ERR_SHAPE),
                   (dict(draft_ld=999), m.MQ_ERR_SHAPE), (dict(n_seqs=5000), m.MQ_ERR_UNSUPPORTED),
                   (dict(vocab=2**28 + 1, target_ld=2**30, draft_ld=2**30), m.MQ_ERR_UNSUPPORTED),
                   (dict(flags=2), m.MQ_ERR_INVALID_ARG), (dict(reserved=1), m.MQ_ERR_INVALID_ARG),
                   (dict(target=0), m.MQ_ERR_INVALID_ARG), (dict(tok_start=0), m.MQ_ERR_INVALID_ARG),
                   (dict(token=0), m.MQ_ERR_INVALID_ARG), (dict(parent=0), m.MQ_ERR_INVALID_ARG),
                   (dict(u=0), m.MQ_ERR_INVALID_ARG), (dict(path=0), m.MQ_ERR_INVALID_ARG),
                   (dict(n_path=0), m.MQ_ERR_INVALID_ARG), (dict(next=0), m.MQ_ERR_INVALID_ARG),
                   (dict(target=0x1002), m.MQ_ERR_ALIGN), (dict(draft=0x2001), m.MQ_ERR_ALIGN),
                   (dict(u=0x6002), m.MQ_ERR_ALIGN), (dict(path=0x7003), m.MQ_ERR_ALIGN), (dict(n_seqs=0, path=0), m.MQ_OK)):
        assert m.mq_verify_tree(verify(m, **kw)) == st, kw
    assert m._lib.mq_verify_tree(None, 0) == m.MQ_ERR_INVALID_ARG


def test_pool_checks(mq_lib):
    m = mq_lib
    c = cache(m)
    assert m.mq_kv_pool_scratch(c) == 2 * 8 + 4 + 2
    assert m.mq_kv_pool_scratch(cache(m, head_dim=96)) == 0
    calls = {"grow": lambda c, p, n=1: m.mq_kv_grow(c, p, 0x6000), "compact": lambda c, p, n=1: m.mq_kv_compact(c, p),
             "fork": lambda c, p, n=1: m.mq_kv_fork(c, p, 0x6000, 0x7000, 0x8000, n),
             "free": lambda c, p, n=1: m.mq_kv_free(c, p, 0x6000, 0x7000, n)}
    for name, call in calls.items():
        for f in ("refs", "free_list", "n_free", "seq_pages", "scratch"):
            assert call(c, pool(m, **{f: 0})) == m.MQ_ERR_INVALID_ARG, (name, f)
            assert call(c, pool(m, **{f: 0x1002})) == m.MQ_ERR_ALIGN, (name, f)
        assert call(cache(m, head_dim=96), pool(m)) == m.MQ_ERR_SHAPE
        assert call(cache(m, n_seqs=4096, table_ld=2**20), pool(m)) == m.MQ_ERR_UNSUPPORTED
        assert call(cache(m, n_pages=2**30), pool(m)) == m.MQ_ERR_UNSUPPORTED
        assert call(cache(m, n_seqs=0), pool(m)) == m.MQ_OK
        if name in ("fork", "free"):
            assert call(c, pool(m), -1) == m.MQ_ERR_SHAPE and call(c, pool(m), 5000) == m.MQ_ERR_UNSUPPORTED
            assert call(c, pool(m), 0) == m.MQ_OK
    assert m.mq_kv_fork(c, pool(m), 0x6000, 0x7000, 0x8000, 3) == m.MQ_ERR_SHAPE  # more than there are sequences
    assert m.mq_kv_fork(c, pool(m), 0, 0x7000, 0x8000, 1) == m.MQ_ERR_INVALID_ARG
    assert m.mq_kv_fork(c, pool(m), 0x6000, 0x7002, 0x8000, 1) == m.MQ_ERR_ALIGN
    assert m.mq_kv_free(c, pool(m), 0, 0, 1) == m.MQ_ERR_INVALID_ARG
    assert m.mq_kv_free(c, pool(m), 0x6000, 0x7002, 1) == m.MQ_ERR_ALIGN
    assert m.mq_kv_grow(c, pool(m), 0) == m.MQ_ERR_INVALID_ARG and m.mq_kv_grow(c, pool(m), 0x6002) == m.MQ_ERR_ALIGN


def host_cache(m):
    import torch
    page = m.mq_kv_page_bytes(m.MQ_TYPE_F16, 2, 64)
    p = torch.zeros(4 * page + 128, dtype=torch.uint8)
    return m.KVCache(p[(-p.data_ptr()) % 128:][:4 * page], torch.zeros((2, 3), dtype=torch.int32), "f16", 2, 64)


def test_tensor_helpers_refuse_what_they_would_misread(mq_lib):
    import torch
    m, c = mq_lib, host_cache(mq_lib)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    q, ws = torch.zeros((3, 4 * 64), dtype=torch.float16), torch.zeros(128, dtype=torch.uint8)
    for a in ((q.float(), i32(3), i32(2), i32(2), i32(1)), (q, i32(2), i32(2), i32(2), i32(1)),
              (q, i32(3), i32(2), i32(3), i32(1)), (q, i32(3), i32(2), i32(2).long(), i32(1))):
        with pytest.raises(ValueError):
            m.attn_shared(c, *a, out=q, workspace=ws)
    x = torch.zeros((3, 10))
    for bad in (x.half(), x[0], x.t()):
        with pytest.raises(ValueError):
            m.softmax(bad)
    with pytest.raises(ValueError):
        m.softmax(x, out=x[:2])
    with pytest.raises(ValueError):
        m.verify_tree(x, i32(2), i32(3), i32(3))  # no random numbers
    with pytest.raises(ValueError):
        m.KVPool(c, i32(2), i32(4), i32(5), i32(1))
    with pytest.raises(ValueError):
        m.KVPool(c, i32(2), i32(4).long(), i32(4), i32(1))
    pl = m.KVPool(c, i32(2), i32(4), i32(4), i32(1))
    with pytest.raises(ValueError):
        m.kv_grow(c, pl, i32(3))
    with pytest.raises(ValueError):
        m.kv_fork(c, pl, i32(2), i32(1), i32(2))
    with pytest.raises(ValueError):
        m.kv_free(c, pl, i32(2), i32(1))


def test_calls_refuse_what_is_not_on_the_current_device(mq_lib):
    import torch
    m, c = mq_lib, host_cache(mq_lib)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    q, ws, x = torch.zeros((3, 4 * 64), dtype=torch.float16), torch.zeros(128, dtype=torch.uint8), torch.zeros((3, 10))
    pl = m.KVPool(c, i32(2), i32(4), i32(4), i32(1))
    out = torch.zeros((1, 2), dtype=torch.int32)
    for f in (lambda **k: m.attn_shared(c, q, i32(3), i32(2), i32(2), i32(1), out=q, workspace=ws, **k),
              lambda **k: m.attn_shared_workspace(c, 4, 3, 1, **k), lambda **k: m.softmax(x, out=x, **k),
              lambda **k: m.verify_tree(x, i32(2), i32(3), i32(3), u=torch.zeros(3), path=out, n_path=i32(1),
                                        next_token=i32(1), **k),
              lambda **k: m.kv_grow(c, pl, i32(2), **k), lambda **k: m.kv_fork(c, pl, i32(1), i32(1), i32(1), **k),
              lambda **k: m.kv_free(c, pl, i32(1), **k), lambda **k: m.kv_compact(c, pl, **k)):
        for stream in (None, 0x1000):
            with pytest.raises((ValueError, RuntimeError, AssertionError)):
                f(stream=stream)
