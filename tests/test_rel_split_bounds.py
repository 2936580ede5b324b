"""The error bounds that the fp32 kernels of the relative position bias state for their split operands,
on the splits' arithmetic restated in NumPy (no GPU)."""
import numpy as np
import pytest


def fp16_terms(x, top):
    """x as two fp16 terms under the scale that brings top, the row's largest, to 2^13 .. 2^14."""
    mul = 2.0 ** (13 - np.floor(np.log2(top)))
    y = x * mul
    hi = y.astype(np.float16).astype(np.float64)
    lo = (y - hi).astype(np.float16).astype(np.float64)
    return hi / mul, lo / mul


def tf32_terms(x):
    """x as the nearest tf32 (ties away from 0) and the rest, cut to a tf32's 11 bits."""
    bits = x.astype(np.float32).view(np.uint32)
    hi = ((bits + np.uint32(0x1000)) & np.uint32(0xffffe000)).view(np.float32)
    lo = (x.astype(np.float32) - hi).astype(np.float32)
    cut = (lo.view(np.uint32) & np.uint32(0xffffe000)).view(np.float32)
    return hi.astype(np.float64), lo.astype(np.float64), cut.astype(np.float64)


def values(seed):
    g = np.random.Generator(np.random.PCG64(seed))
    x = np.ldexp(1 + g.integers(0, 2 ** 23, 400000) * 2.0 ** -23, g.integers(-30, 1, 400000))
    return x.astype(np.float32).astype(np.float64)  # below 2


@pytest.mark.parametrize("seed", [1, 2])
def test_two_fp16_terms(seed):
    x = np.concatenate([values(seed), [2.0 ** -16 + 2.0 ** -38, 1 + 2.0 ** -11 - 2.0 ** -23]])
    hi, lo = fp16_terms(x, 1.0)
    left = np.abs(x - hi - lo)
    assert np.all(left <= np.maximum(2.0 ** -23 * x, 2.0 ** -38))
    assert np.all(np.abs(lo) <= np.maximum(2.0 ** -11 * x, 2.0 ** -37))
    # neither bound can be halved
    assert left[-2] == 2.0 ** -38 and left[-2] > 2.0 ** -23 * x[-2]
    large = x > 2.0 ** -10
    assert (left[large] / x[large]).max() > 2.0 ** -24


@pytest.mark.parametrize("seed", [3, 4])
def test_two_tf32_terms(seed):
    x = np.concatenate([values(seed), [1 + 2.0 ** -11 - 2.0 ** -23]])
    hi, lo, cut = tf32_terms(x)
    assert np.all(np.abs(lo) <= 2.0 ** -11 * x) and np.all(hi + lo == x)
    assert np.all(np.abs(x - hi - cut) <= 2.0 ** -23 * x)
    assert np.abs(lo[-1]) > 0.99 * 2.0 ** -11 * x[-1]
    drop = lo * np.roll(lo, 1)
    assert np.all(np.abs(drop) <= 2.0 ** -22 * x * np.roll(x, 1))
    assert lo[-1] ** 2 > 0.99 * 2.0 ** -22 * x[-1] ** 2


@pytest.mark.parametrize("hidden", [1.0, 1e8, 1e30])
def test_products_over_rows_follow_the_weights(hidden):
    # sum over j of w_j v_j as the kernels take it: V's rows under scales of their own, their factors in
    # the weights, which are split under one scale of theirs.  A row of weight 0 costs nothing.
    g = np.random.Generator(np.random.PCG64(5))
    w, V = g.random((16, 32)), g.standard_normal((32, 64))
    w[:, 31] = 0
    V[31] *= hidden
    V = V.astype(np.float32).astype(np.float64)
    w = w.astype(np.float32).astype(np.float64)
    factor = 2.0 ** (np.floor(np.log2(np.abs(V).max(1))) - 13)
    vh, vl = (np.stack(t) * 1.0 for t in zip(*(fp16_terms(r, np.abs(r).max()) for r in V)))
    u = w * factor
    terms = [fp16_terms(r, r.max()) for r in u]
    uh, ul = (np.stack(t) for t in zip(*terms))
    vh, vl = vh / factor[:, None], vl / factor[:, None]
    got = uh @ vh + uh @ vl + ul @ vh
    want, size = w @ V, np.abs(w) @ np.abs(V)
    # a term: 2^-23 of either factor (2^-38 of the largest where it is that much smaller), 2^-22 dropped
    assert np.all(np.abs(got - want) <= 2.0 ** -21 * size + 2.0 ** -36 * w.max() * np.abs(V[:31]).max() * 32)
