"""The key/value cache and attention calls on the host: sizes, and refusals before anything reaches CUDA."""
import ctypes

import numpy as np
import pytest

from tests import kv_plain as P


def cache(m, **kw):
    f = dict(pages=0x10000, table=0x20000, n_pages=8, n_seqs=2, table_ld=4, type=m.MQ_TYPE_Q8_0, n_kv_heads=4,
             head_dim=128, reserved=0)
    f.update(kw)
    return m.KvCacheStruct(*[f[n] for n, _ in m.KvCacheStruct._fields_])


def append(m, **kw):
    f = dict(qkv=0x1000, q_norm=0x2000, k_norm=0x3000, inv_freq=0x4000, pos=0x5000, seq=0x6000, slot=0x7000, q_out=0x8000,
             qkv_ld=36 * 128, q_ld=28 * 128, n_tokens=1, n_heads=28, rot_dims=128, flags=0, eps=1e-6, reserved=0)
    f.update(kw)
    return m.KvAppendArgs(*[f[n] for n, _ in m.KvAppendArgs._fields_])


def attn(m, **kw):
    f = dict(q=0x1000, out=0x2000, tok_start=0x3000, ctx_len=0x4000, mask=0x5000, q_ld=28 * 128, out_ld=28 * 128,
             n_tokens=1, n_heads=28, max_len=100, max_tokens=1, out_type=m.MQ_TYPE_F16, scale=0.1)
    f.update(kw)
    return m.AttnArgs(*[f[n] for n, _ in m.AttnArgs._fields_])


def test_struct_sizes(mq_lib):
    assert ctypes.sizeof(mq_lib.KvCacheStruct) == 3 * 8 + 6 * 4
    assert ctypes.sizeof(mq_lib.KvAppendArgs) == 10 * 8 + 6 * 4
    assert ctypes.sizeof(mq_lib.AttnArgs) == 7 * 8 + 6 * 4


def test_page_bytes(mq_lib):
    m = mq_lib
    for D in (64, 128):
        for H in (1, 4):
            assert m.mq_kv_page_bytes(m.MQ_TYPE_F16, H, D) == H * P.block_bytes("f16", D)
            assert m.mq_kv_page_bytes(m.MQ_TYPE_Q8_0, H, D) == H * P.block_bytes("q8_0", D)
    for bad in ((m.MQ_TYPE_Q4_K, 4, 128), (m.MQ_TYPE_F16, 0, 128), (m.MQ_TYPE_F16, 4, 96), (m.MQ_TYPE_F16, 4, 256)):
        assert m.mq_kv_page_bytes(*bad) == 0


def test_layout_is_a_permutation():
    rng = np.random.default_rng(0)
    for ctype in ("f16", "q8_0"):
        for D in (64, 128):
            K, V = (rng.standard_normal((64, D)).astype(np.float32) for _ in range(2))
            k, v = P.unpack(P.pack(K, V, ctype), ctype, D)
            assert np.array_equal(k, P.stored(K, ctype)) and np.array_equal(v, P.stored(V, ctype))
            at, voff, sc, soff = P.places(ctype, D)
            step = 2 if ctype == "f16" else 1
            spots = np.concatenate([at.ravel(), at.ravel() + voff]) // step
            assert len(np.unique(spots)) == 2 * 64 * D and spots.max() * step < P.block_bytes(ctype, D)


def test_cache_checks(mq_lib):
    m = mq_lib
    chk = m.mq_check_kv_cache
    assert chk(cache(m)) == m.MQ_OK
    for kw, st in ((dict(type=m.MQ_TYPE_Q4_0), m.MQ_ERR_INVALID_ARG), (dict(pages=0), m.MQ_ERR_INVALID_ARG),
                   (dict(table=0), m.MQ_ERR_INVALID_ARG), (dict(pages=0x10040), m.MQ_ERR_ALIGN),
                   (dict(table=0x20002), m.MQ_ERR_ALIGN), (dict(head_dim=96), m.MQ_ERR_SHAPE),
                   (dict(n_kv_heads=0), m.MQ_ERR_SHAPE), (dict(n_pages=-1), m.MQ_ERR_SHAPE),
                   (dict(table_ld=-1), m.MQ_ERR_SHAPE), (dict(n_seqs=5000), m.MQ_ERR_UNSUPPORTED),
                   (dict(table_ld=2**27), m.MQ_ERR_UNSUPPORTED), (dict(reserved=1), m.MQ_ERR_INVALID_ARG)):
        assert chk(cache(m, **kw)) == st, kw


def test_append_checks(mq_lib):
    m = mq_lib
    c = cache(m)
    for kw, st in ((dict(qkv_ld=36 * 128 - 2), m.MQ_ERR_SHAPE), (dict(qkv_ld=36 * 128 + 1), m.MQ_ERR_SHAPE),
                   (dict(q_ld=28 * 128 - 2), m.MQ_ERR_SHAPE), (dict(rot_dims=130), m.MQ_ERR_SHAPE),
                   (dict(rot_dims=7), m.MQ_ERR_SHAPE), (dict(n_tokens=-1), m.MQ_ERR_SHAPE),
                   (dict(flags=2), m.MQ_ERR_INVALID_ARG), (dict(eps=-1.0), m.MQ_ERR_INVALID_ARG),
                   (dict(eps=float("nan")), m.MQ_ERR_INVALID_ARG), (dict(qkv=0), m.MQ_ERR_INVALID_ARG),
                   (dict(seq=0), m.MQ_ERR_INVALID_ARG), (dict(slot=0), m.MQ_ERR_INVALID_ARG),
                   (dict(q_out=0), m.MQ_ERR_INVALID_ARG), (dict(pos=0), m.MQ_ERR_INVALID_ARG),
                   (dict(inv_freq=0), m.MQ_ERR_INVALID_ARG), (dict(qkv=0x1004), m.MQ_ERR_ALIGN),
                   (dict(q_out=0x8002), m.MQ_ERR_ALIGN), (dict(q_norm=0x2004), m.MQ_ERR_ALIGN),
                   (dict(n_heads=2000, qkv_ld=2**20, q_ld=2**20), m.MQ_ERR_UNSUPPORTED),
                   (dict(n_tokens=0, qkv=0), m.MQ_OK)):
        assert m.mq_kv_append(c, append(m, **kw)) == st, kw
    assert m.mq_kv_append(cache(m, head_dim=32), append(m)) == m.MQ_ERR_SHAPE
    assert m.mq_kv_read(c, 0x1000, 0x2000, -1, 0x3000, 0x4000) == m.MQ_ERR_SHAPE
    assert m.mq_kv_read(c, 0, 0, 0, 0, 0) == m.MQ_OK
    assert m.mq_kv_read(c, 0x1000, 0x2000, 1, 0, 0x4000) == m.MQ_ERR_INVALID_ARG
    assert m.mq_kv_read(c, 0x1000, 0x2000, 1, 0x3008, 0x4000) == m.MQ_ERR_ALIGN
    assert m.mq_kv_accept(c, 0x1000, 0x2000, 0x3000, 65) == m.MQ_ERR_SHAPE
    assert m.mq_kv_accept(c, 0, 0, 0, 0) == m.MQ_OK
    assert m.mq_kv_accept(c, 0x1000, 0, 0x3000, 4) == m.MQ_ERR_INVALID_ARG
    assert m.mq_kv_accept(c, 0x1002, 0x2000, 0x3000, 4) == m.MQ_ERR_ALIGN


def test_attn_checks(mq_lib):
    m = mq_lib
    c = cache(m)
    for kw, st in ((dict(n_heads=27), m.MQ_ERR_SHAPE), (dict(n_heads=0), m.MQ_ERR_SHAPE),
                   (dict(max_tokens=0), m.MQ_ERR_SHAPE), (dict(max_tokens=65), m.MQ_ERR_SHAPE),
                   (dict(q_ld=28 * 128 - 8), m.MQ_ERR_SHAPE), (dict(q_ld=28 * 128 + 4), m.MQ_ERR_SHAPE),
                   (dict(out_ld=28 * 128 - 8), m.MQ_ERR_SHAPE), (dict(n_tokens=-1), m.MQ_ERR_SHAPE),
                   (dict(max_len=-1), m.MQ_ERR_SHAPE), (dict(out_type=m.MQ_TYPE_Q4_0), m.MQ_ERR_INVALID_ARG),
                   (dict(scale=float("nan")), m.MQ_ERR_INVALID_ARG), (dict(scale=float("inf")), m.MQ_ERR_INVALID_ARG),
                   (dict(q=0), m.MQ_ERR_INVALID_ARG), (dict(tok_start=0), m.MQ_ERR_INVALID_ARG),
                   (dict(q=0x1008), m.MQ_ERR_ALIGN), (dict(out=0x2008), m.MQ_ERR_ALIGN),
                   (dict(mask=0x5004), m.MQ_ERR_ALIGN), (dict(n_heads=1028, q_ld=2**20, out_ld=2**20), m.MQ_ERR_UNSUPPORTED),
                   (dict(max_len=2**31 - 1, max_tokens=64), m.MQ_ERR_UNSUPPORTED), (dict(n_tokens=0, q=0), m.MQ_OK)):
        assert m.mq_attn_tree(c, attn(m, **kw), 0x9000, 2**40) == st, kw
    assert m.mq_attn_tree(c, attn(m), 0, 2**40) == m.MQ_ERR_INVALID_ARG
    assert m.mq_attn_tree(c, attn(m), 0x9010, 2**40) == m.MQ_ERR_ALIGN


def test_tensor_helpers_refuse_what_they_would_misread(mq_lib):
    import torch
    m = mq_lib
    table = torch.zeros((2, 3), dtype=torch.int32)
    page = m.mq_kv_page_bytes(m.MQ_TYPE_F16, 2, 64)
    pool = torch.zeros(4 * page + 128, dtype=torch.uint8)
    pool = pool[(-pool.data_ptr()) % 128:][:4 * page]
    c = m.KVCache(pool, table, "f16", 2, 64)
    with pytest.raises(ValueError):
        m.KVCache(pool[:-128], table, "f16", 2, 64)   # not whole pages
    with pytest.raises(ValueError):
        m.KVCache(pool, table.long(), "f16", 2, 64)
    with pytest.raises(ValueError):
        m.KVCache(pool, table, "q5", 2, 64)
    with pytest.raises(m.MQError):
        m.KVCache(pool, table, "f16", 2, 80)
    i = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros((3, 8 * 64))
    q = torch.zeros((3, 4 * 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        m.kv_append(c, x.half(), i, i, i, 4, q_out=q)
    with pytest.raises(ValueError):
        m.kv_append(c, x, i, i[:2], i, 4, q_out=q)
    with pytest.raises(ValueError):
        m.kv_append(c, x, i, i, i, 4, q_norm=torch.ones(32), q_out=q)
    with pytest.raises(ValueError):
        m.kv_append(c, x, i, i, i, 4, q_out=q[:2])
    with pytest.raises(ValueError):
        m.kv_read(c, i, i, k_out=q.view(3, 4, 64), v_out=q.view(3, 4, 64))
    with pytest.raises(ValueError):
        m.kv_accept(c, i[:2], torch.zeros((3, 4), dtype=torch.int32), i[:2])
    ws = torch.zeros(128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.attn_tree(c, q.float(), i, i[:2], out=q, workspace=ws)
    with pytest.raises(ValueError):
        m.attn_tree(c, q, i, i[:2], mask=i, out=q, workspace=ws)
    with pytest.raises(ValueError):
        m.attn_tree(c, q, i, i[:2], out=q[:2], workspace=ws)
    with pytest.raises(ValueError):
        m.attn_tree(c, q, i, i[:2], out_type="f32", workspace=ws)


def test_attention_work_is_counted_with_its_groups(mq_lib):
    # pages and the cost of a group together pass 31 bits where the pages alone do not
    m = mq_lib
    c = m.KvCacheStruct(0x10000, 0x20000, 10, 4096, 2**20, m.MQ_TYPE_Q8_0, 256, 64, 0)
    a = m.AttnArgs(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 1024 * 64, 1024 * 64, 64, 1024, 0, 64, m.MQ_TYPE_F16, 1.0)
    for max_len, want in ((64 * 51, m.MQ_OK), (64 * 52, m.MQ_ERR_UNSUPPORTED)):
        a.max_len, a.n_tokens = max_len, 0
        assert m._lib.mq_attn_tree(c, a, 0, 0, 0) == want


def test_calls_refuse_a_cache_that_is_not_on_the_current_device(mq_lib, monkeypatch):
    # the library launches on the current device: a cache elsewhere, or in host memory, must not reach it
    import torch
    m = mq_lib
    page = m.mq_kv_page_bytes(m.MQ_TYPE_F16, 2, 64)
    pool = torch.zeros(4 * page + 128, dtype=torch.uint8)
    c = m.KVCache(pool[(-pool.data_ptr()) % 128:][:4 * page], torch.zeros((2, 3), dtype=torch.int32), "f16", 2, 64)
    i = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros((3, 4 * 64), dtype=torch.float16)
    kv = torch.zeros((3, 2, 64), dtype=torch.float16)
    ws = torch.zeros(128, dtype=torch.uint8)

    class Stream:
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device("cuda", index), 0x1000

    class Library:  # what a call would launch
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or m.MQ_OK

    calls = []
    monkeypatch.setattr(m, "_lib", Library())
    run = [lambda **k: m.kv_append(c, torch.zeros((3, 8 * 64)), i, i, i, 4, q_out=q, **k),
           lambda **k: m.kv_read(c, i, i, k_out=kv, v_out=kv.clone(), **k),
           lambda **k: m.kv_accept(c, i[:2], torch.zeros((2, 4), dtype=torch.int32), i[:2], **k),
           lambda **k: m.attn_tree(c, q, i, i[:2], max_len=64, out=q.clone(), workspace=ws, **k),
           lambda **k: m.attn_workspace(c, 4, **k)]
    for f in run:  # host memory, whatever the stream
        for stream in (0x1000, Stream(0)):
            with pytest.raises(ValueError):
                f(stream=stream)
    # device memory, as far as the calls can tell
    c.device = torch.device("cuda", 1)
    monkeypatch.setattr(m, "_want", lambda t, *a, **k: t.data_ptr())
    monkeypatch.setattr(m, "_rows", lambda t, *a, **k: (t.data_ptr(), t.shape[1]))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for f in run:
        for stream in (0x1000, Stream(0), Stream(1), None):
            with pytest.raises(ValueError):
                f(stream=stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for f in run:  # the right device, a stream of another
        with pytest.raises(ValueError):
            f(stream=Stream(0))
    assert not calls
    for f in run[:4]:
        f(stream=Stream(1))
        f(stream=0x1000)
    assert calls == [n for n in ("mq_kv_append", "mq_kv_read", "mq_kv_accept", "mq_attn_tree") for _ in range(2)]
