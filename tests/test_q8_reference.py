"""The 8-bit moments' definition itself, on the CPU: range, error, bias, and
that a state read out and stored again keeps its values."""
import numpy as np
import pytest

from tests import tensors_reference as ref


def values(rng, n, spread):
    return (rng.standard_normal(n) * np.exp2(rng.uniform(-spread, 0, n))).astype(np.float32)


@pytest.mark.parametrize("name,spread", [("m", 0), ("m", 12), ("v", 0), ("v", 30)])
def test_error_is_below_one_step(name, spread):
    rng = np.random.default_rng(1)
    for scale in (1.0, 1e-20, 1e-38, 3e37, 1e-44):
        x = (values(rng, 5000, spread) * np.float32(scale)).astype(np.float32)
        if name == "v":
            x = np.abs(x)
        y = ref.stored(x, name, 3, 77)
        most = np.repeat(np.maximum.reduceat(np.abs(x), np.arange(0, x.size, 256)), 256)[:x.size].astype(np.float64)
        # a step is at most 1/8 of the value (3 fraction bits), or of the least normal code: 2^-(exponents - 1) of
        # the top binade, which the block's largest value is in or just below (the lowest binade that a scale byte can
        # name is 2^-127); binary32's own least step besides
        floor = np.maximum(most, 2.0 ** -127) * 2.0 / 2.0 ** (14 if name == "m" else 30)
        step = np.maximum(np.abs(x.astype(np.float64)), floor) / 8 + 2.0 ** -149
        assert (np.abs(y.astype(np.float64) - x) <= step).all(), scale
        if name == "v":
            assert ((y > 0) == (x > 0)).all()


@pytest.mark.parametrize("name", ["m", "v"])
def test_values_survive_another_encoding(name):
    rng = np.random.default_rng(2)
    for scale in (1.0, 1e-30):
        x = (values(rng, 20000, 25) * np.float32(scale)).astype(np.float32)
        if name == "v":
            x = np.abs(x)
        y = ref.stored(x, name, 0, 5)
        for key in (5, 6, 123456789):
            assert np.array_equal(ref.stored(y, name, 1, key).view(np.uint32), y.view(np.uint32))


def test_rounding_is_unbiased():
    """The mean over many keys; a code step is 1/8 here, so the mean of N
    draws has a deviation of at most 1/16 / sqrt(N); 5 of them."""
    x = np.full(256, 1.01, np.float32)
    x[0] = 1.75
    x[1:100] = np.linspace(1.0, 1.75, 99, dtype=np.float32)
    total, N = np.zeros((2, 256)), 4000
    for key in range(N):
        total[0] += ref.stored(x, "m", 0, key)
        total[1] += ref.stored(x, "v", 0, key)
    assert np.abs(total / N - x).max() <= 5 / 16 / np.sqrt(N)


@pytest.mark.parametrize("name", ["m", "v"])
def test_edges(name):
    z = np.zeros(300, np.float32)
    assert not ref.stored(z, name, 0, 1).any()
    codes, e = ref.encode(z, name, ref.words(300, 0, 1))
    assert not codes.any() and not e.any()      # zero bytes hold zero moments
    for bad in (np.inf, np.nan, 3.3e38):
        x = np.ones(600, np.float32)
        x[300] = bad
        y = ref.stored(x, name, 0, 9)
        assert np.isnan(y[256:512]).all() and (y[:256] == 1).all() and (y[512:] == 1).all()
    # the top code and a mantissa just above it
    for top in (np.float32(1.875), np.nextafter(np.float32(1.875), np.float32(2)), np.float32(1.9999)):
        for key in range(50):
            y = ref.stored(np.full(256, top, np.float32), name, 0, key)
            assert np.isfinite(y).all() and (np.abs(y - top) <= 0.25).all()


@pytest.mark.parametrize("name", ["m", "v"])
def test_the_largest_value(name):
    """1.875 * 2^127 is the top code of the largest scale; anything above it makes its block NaN."""
    top = np.uint32(0x7F700000)
    for key in range(20):
        assert (ref.stored(np.full(256, top.view(np.float32)), name, 0, key) == top.view(np.float32)).all()
        assert np.isnan(ref.stored(np.full(256, (top + 1).view(np.float32)), name, 0, key)).all()


def test_one_moment_moves_where_rounding_to_nearest_would_not():
    """beta2 = 0.999 and a squared gradient that falls to a quarter: the mean of
    the stored second moments follows the exact one.  Each store adds at most
    a binary64-free error of one step times a fair coin: relative deviation of
    one element at most sqrt(step/2) = 0.25 (the variance step * |change| adds up
    to step/2 over the averaging window), of the mean of 4096 at most 0.004; 5
    of them."""
    n, b2 = 4096, np.float32(0.999)
    v = ref.stored(np.ones(n, np.float32), "v", 0, 0)
    exact = 1.0
    for t in range(1, 1501):
        v = ref.stored(b2 * v + np.float32(1) * (1 - b2) * np.float32(0.25), "v", 0, ref.key_of(3, t))
        exact = 0.999 * exact + 0.001 * 0.25
    assert abs(v.mean() - exact) <= 5 * 0.25 / np.sqrt(n) * exact
