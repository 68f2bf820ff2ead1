"""The speculative-decoding example: its attention against the plain 64-bit form, and its cache after acceptances
against a cache that got the accepted tokens one chain after the other."""
import importlib.util
import os

import numpy as np
import pytest

from tests import kv_plain as P
from tests.test_gpu_attn import bound, values_of
from tests.test_gpu_kv import dev, ok_status

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")
    spec = importlib.util.spec_from_file_location("tree_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("nodes", [4, 30])
def test_example(cuda_ready, ctype, nodes):
    from quantized_decode_matvec_gb300 import synth
    mq = cuda_ready
    seen = []

    def read(cache, s, n):
        k, v = mq.kv_read(cache, dev(np.full(n, s, np.int32)), dev(np.arange(n, dtype=np.int32)))
        return k.cpu().numpy(), v.cpu().numpy()

    def on_step(cache, layer, tree, q, att):
        ctx, start, masks = tree
        got = values_of(att, q.shape[0], layer.heads * layer.D).reshape(-1, layer.heads, layer.D)
        qs = q.cpu().numpy().reshape(-1, layer.heads, layer.D)
        for s, c in enumerate(ctx):
            k, v = read(cache, s, c + nodes)
            a, b = start[s], start[s + 1]
            ref, A, big = P.attention(qs[a:b], k, v, c, masks[s], layer.D**-0.5)
            tol = bound(ref, A, big)
            top = (np.abs(ref) + tol).reshape(b - a, layer.heads, -1, 32).max(-1).repeat(32, -1)
            assert (np.abs(got[a:b] - ref) <= tol + top / 127 * (0.5 + 2 * 127 * 2**-11)).all()
        seen.append(1)

    ex = example()
    cache, layer, length, tokens = ex.run(mq, synth, ctype, steps=3, nodes=nodes, on_step=on_step)
    ok_status(mq)
    assert len(seen) == 3 and all(n > p for n, p in zip(length, (150, 37)))
    # the same tokens as chains from the start: the same projections up to the order of their fp32 sums, so a stored
    # value differs by an f16 rounding or a q8_0 step
    again, *_ = ex.run(mq, synth, ctype, steps=0, nodes=nodes, prompts=tuple(length))
    work = mq.attn_workspace(again, layer.heads)
    i32 = lambda a: dev(np.asarray(a, np.int32))
    for s, n in enumerate(length):
        for c in range(0, n, 64):
            m = min(64, n - c)
            start = np.zeros(len(length) + 1, np.int32)
            start[s + 1:] = m
            layer.forward(again, dev(tokens[s][c:c + m]), i32(np.arange(c, c + m)), i32([s] * m),
                          i32(np.arange(c, c + m)), i32(start), i32([c if i == s else 0 for i in range(len(length))]),
                          None, max(length), work)
        for x, y in zip(read(cache, s, n), read(again, s, n)):
            x, y = x.astype(np.float64), y.astype(np.float64)
            top = np.abs(y).reshape(*y.shape[:-1], -1, 32).max(-1).repeat(32, -1)
            step = top / 127 if ctype == "q8_0" else 2**-10 * np.abs(y) + 2**-18 * top
            assert (np.abs(x - y) <= step * 1.01 + 2**-10 * np.abs(y)).all()
    ok_status(mq)
