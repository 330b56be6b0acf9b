"""That the inputs of the GPU tests of the microscaled operators show what they are made to show (no GPU): each mistake
is made here, in the oracle, and has to move the results past what the GPU tests allow."""
import numpy as np

import mx_cases as C
import mx_reference as R


def test_wide_products_need_the_split():
    """Cut to the instruction's 13 bits the products lose terms in nearly every output; with x split at 2, none."""
    for rows, k, d in ((7, 264, 40), (33, 136, 24), (5, 1416, 16)):
        x, w = C.wide_products(rows, k, d, rows + k)
        codes = R.codes_under(x, np.full((rows, -(-k // 32)), 127, np.uint8), R.E4M3)
        assert (R.grid(R.E4M3)[codes & 127] == np.abs(x)).all()   # held exactly
        want = x @ w.T
        assert (want * 2 ** 10 % 1 == 0).all() and np.abs(want).max() < 2 ** 14
        high = np.where(np.abs(x) >= 2, x, 0)
        np.testing.assert_array_equal(C.instruction(high, w) + C.instruction(x - high, w), want)
        assert (C.instruction(x, w) != want).mean() > 0.95


def test_split_a_binade_lower_shows():
    x, w = C.wide_products(33, 264, 40, 3)
    high = np.where(np.abs(x) >= 1, x, 0)
    assert (C.instruction(high, w) + C.instruction(x - high, w) != x @ w.T).any(1).mean() > 0.5


def test_squares_summed_in_32_bits_show():
    """A norm whose squares are summed in fp32 leaves the bound of the norm's precision tests."""
    g = np.random.default_rng(1)
    x = g.standard_normal((16, 4096)).astype(np.float32)
    _, want = R.norm(x.astype(np.float64), None, np.ones(4096), 0.0)
    mean = np.float32(1 / 4096) * np.cumsum((x * x).reshape(16, 64, 64), -1, dtype=np.float32)[..., -1].sum(-1, dtype=np.float32)
    got = (x / np.sqrt(mean.astype(np.float64))[:, None]).astype(np.float32)
    near = 2.0 ** -40
    off = np.abs(got - want) > (2.0 ** -24 * (1 + near) + near) * np.abs(want)
    assert off.any(1).mean() > 0.5
