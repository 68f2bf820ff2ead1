"""softmax of rows against 64 bits.

Bound, relative to the reference: an exponent is (x - m) k with x - m and the product rounded once (2^-24 each of
|x - max| scale, as a relative error of the exponential) and k to 2^-25, in two steps that add up to x - max where a CTA's
own maximum stands between: 2.5 * 2^-24; two exponentials and three products 2^-21; the sum of up to 64 values per thread, then of 5 + 16 + 8 levels, 2^-17.  2^-126 absolute, where
the factors are below the normal range.
"""
import numpy as np
import pytest

from tests.test_gpu_kv import dev, ok_status

pytestmark = pytest.mark.gpu


def check(got, x, scale):
    z = x.astype(np.float64) * np.float64(np.float32(scale))
    d = z - z.max(-1, keepdims=True)
    e = np.exp(d)
    ref = e / e.sum(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        tol = np.where(e > 0, ref * (2**-17 + 2**-21 + 2**-22 * np.abs(d)), 0) + 2.0**-126
    err = np.abs(got - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:3])


@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 31), (5, 32), (1, 2047), (1, 2048), (4, 2049), (200, 1000),
                                        (7, 50001), (2, 131072), (1, 131071), (3, 200003), (1, 262144), (2, 300001),
                                        (1, 1000003)])
def test_sizes(cuda_ready, rows, vocab):
    rng = np.random.default_rng(vocab)
    x = (rng.standard_normal((rows, vocab)) * 4).astype(np.float32)
    x[rng.random(x.shape) < 0.001] += 30
    for scale in (1.0, 0.3, 2.5):
        got = cuda_ready.softmax(dev(x), scale=scale)
        ok_status(cuda_ready)
        check(got.cpu().numpy().astype(np.float64), x, scale)


@pytest.mark.parametrize("vocab", [1001, 70003, 300001])
def test_strides_offsets_and_in_place(cuda_ready, vocab):
    import torch
    mq = cuda_ready
    rng = np.random.default_rng(3)
    full = (rng.standard_normal((4, vocab + 9)) * 3).astype(np.float32)
    for x0 in range(4):
        for y0 in (0, 1):
            src, out = dev(full), torch.full((4, vocab + 7), -1.0, device="cuda")
            mq.softmax(src[:, x0:x0 + vocab], out=out[:, y0:y0 + vocab])
            ok_status(mq)
            check(out[:, y0:y0 + vocab].cpu().numpy().astype(np.float64), full[:, x0:x0 + vocab], 1.0)
            assert (out[:, :y0] == -1).all() and (out[:, y0 + vocab:] == -1).all()
            same = src[:, x0:x0 + vocab]
            mq.softmax(same, out=same)
            ok_status(mq)
            check(same.cpu().numpy().astype(np.float64), full[:, x0:x0 + vocab], 1.0)
            assert np.array_equal(src.cpu().numpy()[:, x0 + vocab:], full[:, x0 + vocab:])


@pytest.mark.parametrize("vocab", [5, 9000, 131072, 300001])
def test_infinities_and_nan(cuda_ready, vocab):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, vocab)).astype(np.float32)
    x[0, :-1] = -np.inf                       # one value left
    x[1, rng.random(vocab) < 0.9] = -np.inf   # a mask
    x[1, 0] = 0.5
    x[2] = -np.inf
    x[3, 2] = np.inf
    x[4, 3] = np.nan
    x[5, :vocab // 2 + 1] = -np.inf           # whole parts of the row
    x[6] = -3e38                              # the type's lowest values
    x[6, 1] = -1e38
    x[7, 4] = np.nan
    x[7, 5:] = -np.inf
    got = cuda_ready.softmax(dev(x), scale=1.0).cpu().numpy().astype(np.float64)
    ok_status(cuda_ready)
    fine = [0, 1, 5, 6] if vocab > 5 else [0, 1, 6]
    check(got[fine], x[fine], 1.0)
    assert got[0, -1] == 1.0 and got[6, 1] == 1.0
    assert np.isnan(got[[2, 3, 4, 7]]).all()


def test_captured_and_replayed(cuda_ready):
    import torch
    mq = cuda_ready
    x, y = torch.randn((3, 40000), device="cuda"), torch.empty((3, 40000), device="cuda")
    side = torch.cuda.Stream()
    mq.softmax(x, out=y, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        mq.softmax(x, out=y, stream=side)
    for _ in range(3):
        x.normal_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mq.softmax(x))
    ok_status(mq)


@pytest.mark.parametrize("vocab", [3, 700, 3000, 9000, 50001, 131072, 300001])
@pytest.mark.parametrize("scale", [1e-45, 1e-39, 1e-38, 3e-38, 1e-30, 0.99, 1.0, 2.0, 1e30])
def test_finite_rows_whose_values_are_further_apart_than_the_largest_number(cuda_ready, vocab, scale):
    # a difference beyond 3.4e38 still weighs something at a small scale: (3e38 + 3e38) 1e-38 = 6
    rng = np.random.default_rng(vocab)
    x = np.stack([rng.uniform(-1, 1, vocab) * 3.4e38, np.full(vocab, -3.4e38), np.full(vocab, 3.4e38),
                  rng.standard_normal(vocab) * 1e38])
    with np.errstate(over="ignore"):
        x = x.astype(np.float32)  # the normal numbers reach an infinity in some rows: NaN
    x[1, rng.integers(0, vocab)] = 3.4e38
    x[2, rng.integers(0, vocab)] = -3.4e38
    got = cuda_ready.softmax(dev(x), scale=scale).cpu().numpy().astype(np.float64)
    ok_status(cuda_ready)
    fine = ~np.isinf(x).any(-1)
    assert fine[:3].all() and np.isnan(got[(x == np.inf).any(-1)]).all()
    check(got[fine], x[fine], scale)


@pytest.mark.parametrize("vocab", [1000003, 2**22 + 1, 2**25])
def test_sums_of_long_rows(cuda_ready, vocab):
    # Values that round alike when a thread adds them one after the other (8192 of them at 2^25: 2^-13), rising and falling
    # ones.  Of an output: its own exponential 2^-22 + 2^-23 (|d| + 6), the base being up to 2^8 (5.6) below the maximum;
    # the sum's exponentials alike, weighted by themselves, with a mean |d| of at most ln(vocab) < 18: 2^-18.1; its
    # additions 2^-19 (a unit's, and 29 levels over threads and CTAs), its scalings, of which some six still count, 2^-19;
    # the factors behind it 2^-22: 2^-17 + 2^-21 + 2^-22 |d| as above.
    import torch
    mq = cuda_ready
    steps = torch.arange(vocab, device="cuda", dtype=torch.float32)
    for name, x in (("0.7", torch.full((vocab,), float(np.log(0.7)), device="cuda")),
                    ("0.1", torch.full((vocab,), float(np.log(0.1)), device="cuda")),
                    ("rising", steps * (30.0 / vocab)), ("falling", steps * (-30.0 / vocab)),
                    ("rising fast", steps * 0.01), ("steps", (steps % 997) * 0.01)):
        x[vocab // 2] = max(0.0, float(x.max()))
        for scale in (1.0, 0.4):
            got = mq.softmax(x[None], scale=scale)[0].double()
            ok_status(mq)
            z = x.double() * float(np.float32(scale))
            d = z - z.max()
            ref = torch.exp(d)
            ref /= ref.sum()
            tol = ref * (2**-17 + 2**-21 + 2**-22 * d.abs()) + 2.0**-126
            assert bool(((got - ref).abs() <= tol).all()), (name, scale, float(((got - ref).abs() / tol).max()))


@pytest.mark.parametrize("vocab", [5, 9000, 131072, 300001])
@pytest.mark.parametrize("scale", [1e-37, 9.99e-37, 1.01e-36, 1e-35])
def test_smallest_scales(cuda_ready, vocab, scale):
    # on both sides of where differences are taken of halves: masks, NaN and infinities as at any scale
    rng = np.random.default_rng(vocab)
    x = (rng.uniform(-3.4, 3.4, (6, vocab)) * 1e38).astype(np.float32)
    x[0, :-1] = -np.inf
    x[1, rng.random(vocab) < 0.5] = -np.inf
    x[1, 0] = 1.0
    x[2] = -np.inf
    x[3, 1] = np.inf
    x[4, 2] = np.nan
    got = cuda_ready.softmax(dev(x), scale=scale).cpu().numpy().astype(np.float64)
    ok_status(cuda_ready)
    check(got[[0, 1, 5]], x[[0, 1, 5]], scale)
    assert np.isnan(got[[2, 3, 4]]).all() and got[0, -1] == 1.0


# (rows, values): a row in 2, 4 and 8 units of a thread by one CTA, in clusters of two, four and eight, and in 9 units;
# more rows than are on the chip at once, so that parts of later ones are called for ahead
@pytest.mark.parametrize("rows,vocab", [(400, 3000), (400, 6001), (400, 14002), (200, 20003), (100, 50001), (60, 100000),
                                        (60, 131072), (50, 131071), (50, 147000), (40, 200003)])
@pytest.mark.parametrize("at,pad", [(0, 0), (0, 3), (1, 0), (3, 5)])
def test_many_rows_wherever_they_start(cuda_ready, rows, vocab, at, pad):
    import torch
    mq = cuda_ready
    torch.manual_seed(rows + vocab)
    full = torch.randn((rows, vocab + at + pad), device="cuda") * 3
    full[:, :at] = full[:, at + vocab:] = float("nan")
    x, out = full[:, at:at + vocab], torch.full((rows, vocab + 5), -1.0, device="cuda")
    want = torch.softmax(x.double(), -1)
    d = x.double() - x.double().amax(-1, keepdim=True)
    tol = want * (2**-17 + 2**-21 + 2**-22 * d.abs()) + 2.0**-126
    for y0 in (0, 1):
        out.fill_(-1)
        mq.softmax(x, out=out[:, y0:y0 + vocab])
        ok_status(mq)
        err = (out[:, y0:y0 + vocab].double() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert (out[:, :y0] == -1).all() and (out[:, y0 + vocab:] == -1).all()
    mq.softmax(x, out=x)
    ok_status(mq)
    assert torch.equal(x, out[:, 1:1 + vocab]) and bool(torch.isnan(full[:, :at]).all() and torch.isnan(full[:, at + vocab:]).all())
