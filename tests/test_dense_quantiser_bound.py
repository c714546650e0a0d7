"""The quantiser's fast path on the CPU: x / s as the fp32 product x (1 / s) is
off by less than 1.15e-5 for |x / s| <= 127: 127 2^-24 from the reciprocal's
rounding and 2^-18, half a step of a product between 64 and 128. It decides
where it lies 2e-5 and more from a half-integer."""
import numpy as np

BOUND = 127.5 * 2.0 ** -24 + 2.0 ** -18      # 127.5: the quotient of a row's largest value, s being rounded
MARGIN = 0.5 - float(np.float32(0.49998))


def errors(m, x):
    s = m / np.float32(127)
    t = x * (np.float32(1) / s)
    assert t.dtype == np.float32
    return np.abs(t.astype(np.float64) - x.astype(np.float64) / s.astype(np.float64))


def test_the_bound_holds_and_is_nearly_reached():
    assert BOUND < 1.15e-5 < MARGIN
    rng = np.random.default_rng(3)
    worst = 0.0
    for _ in range(20):
        m = (1 + rng.random(1 << 19)).astype(np.float32)
        x = (m * (1 - rng.random(1 << 19) ** 3 / 2)).astype(np.float32)
        worst = max(worst, errors(m, x).max())
    assert 127 * 2.0 ** -24 < 1.05e-5 < worst < BOUND        # one rounding alone would be below 7.6e-6
    assert errors(np.float32([1.9843475]), np.float32([1.9786434]))[0] > 1.1e-5


def test_codes_of_the_fast_path_are_those_of_the_exact_quotient():
    rng = np.random.default_rng(4)
    m = (1 + rng.random(1 << 16)).astype(np.float32)
    s = m / np.float32(127)
    n = rng.integers(-127, 127, 1 << 16)
    half = (n + 0.5) * s.astype(np.float64)              # exact: 24 and 8 bits
    for ulps in range(-6, 7):
        x = half.astype(np.float32)
        x = (x.view(np.int32) + ulps).view(np.float32)
        t = x * (np.float32(1) / s)
        near = np.rint(t)
        fast = np.abs(t - near) < np.float32(0.49998)
        exact = np.where(x.astype(np.float64) > half, n + 1, np.where(x.astype(np.float64) < half, n, n + (n & 1)))
        assert (near[fast] == exact[fast]).all()
        assert fast.any() or abs(ulps) < 3               # nearer than that the quotient decides
