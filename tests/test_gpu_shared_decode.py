"""The example of several answers to one prompt: its attention against the plain 64-bit form, its verification against
the walk in rational arithmetic, its pool against what the sequences hold, its cache against one that was never forked."""
import importlib.util
import os

import numpy as np
import pytest

from tests import kv_plain as P
from tests.test_gpu_attn import bound, values_of
from tests.test_gpu_kv import dev, ok_status
from tests.test_gpu_verify import walk

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_decode.py")
    spec = importlib.util.spec_from_file_location("shared_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ctype", ["q8_0", "f16"])
@pytest.mark.parametrize("nodes,prompt", [(1, 130), (6, 150), (10, 128)])
def test_example(cuda_ready, ctype, nodes, prompt):
    from quantized_decode_matvec_gb300 import synth
    mq = cuda_ready
    seen = []

    def read(d, s, n):
        k, v = mq.kv_read(d.cache, dev(np.full(n, s, np.int32)), dev(np.arange(n, dtype=np.int32)))
        return k.cpu().numpy(), v.cpu().numpy()

    def on_step(d, step):
        layer, start = d.layer, step["start"]
        got = values_of(step["att"], step["q"].shape[0], layer.heads * layer.D).reshape(-1, layer.heads, layer.D)
        qs = step["q"].cpu().numpy().reshape(-1, layer.heads, layer.D)
        target, ids = step["target"].cpu().numpy(), step["ids"].cpu().numpy()
        draft, path, n_path, last = (x.cpu().numpy() for x in (d.draft[step["ids"]], step["path"], step["n_path"], step["last"]))
        u = np.concatenate([step["u"][s] for s in range(len(start) - 1) if start[s + 1] > start[s]])
        for s in range(len(start) - 1):
            a, b = start[s], start[s + 1]
            if a == b:
                assert n_path[s] == 0 and last[s] == -1
                continue
            c = step["ctx"][s]
            k, v = read(d, s, c + b - a)
            ref, A, big = P.attention(qs[a:b], k, v, c, step["masks"][s], layer.D**-0.5)
            tol = bound(ref, A, big) + 2.0**-20 * A
            top = (np.abs(ref) + tol).reshape(b - a, layer.heads, -1, 32).max(-1).repeat(32, -1)
            assert (np.abs(got[a:b] - ref) <= tol + top / 127 * (0.5 + 2 * 127 * 2**-11)).all()
            want, tok = walk(target[a:b], draft[a:b], ids[a:b], np.array(step["parent"][a:b]), u[a:b], d.nodes)
            assert path[s, :n_path[s]].tolist() == want and last[s] == tok
        seen.append(int(n_path.max()))

    d, live, accepted = example().run(mq, synth, ctype, answers=5, steps=3, nodes=nodes, prompt=prompt, on_step=on_step)
    ok_status(mq)
    assert len(seen) == 4 and accepted >= 4 * len(live)
    # the pool: as many references as table entries, pages as the lengths want, those in use in front
    table, seq_pages = d.cache.table.cpu().numpy(), d.pool.seq_pages.cpu().numpy()
    held = [table[s, :seq_pages[s]] for s in range(len(table))]
    refs = np.bincount(np.concatenate(held), minlength=d.cache.struct.n_pages)
    assert np.array_equal(refs, d.pool.refs.cpu().numpy())
    assert seq_pages.tolist() == [-(-n // 64) for n in d.length] and int(d.pool.n_free) == (refs == 0).sum()
    for s in live:
        assert table[s, :prompt // 64].tolist() == table[0, :prompt // 64].tolist()
    # the prompt's slots of an answer are the prompt's, bit for bit, forked and moved or not
    k0, v0 = read(d, 0, prompt)
    for s in live:
        k, v = read(d, s, prompt)
        assert np.array_equal(k, k0) and np.array_equal(v, v0)
    # the accepted tokens, written as a chain into a cache that was never forked: the same projections up to the order
    # of their fp32 sums, so a stored value differs by an f16 rounding or a q8_0 step
    s = live[-1]
    again = example().Decoder(mq, synth, ctype, 5, d.length[s], 1, nodes)
    again.prompt(d.tokens[s])
    ok_status(mq)
    for x, y in zip(read(d, s, d.length[s]), read(again, 0, d.length[s])):
        x, y = x.astype(np.float64), y.astype(np.float64)
        top = np.abs(y).reshape(*y.shape[:-1], -1, 32).max(-1).repeat(32, -1)
        step = top / 127 if ctype == "q8_0" else 2**-10 * np.abs(y) + 2**-18 * top
        assert (np.abs(x - y) <= step * 1.01 + 2**-10 * np.abs(y)).all()
