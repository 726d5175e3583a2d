"""What the limits of linear_states are for: plainer forms of the recurrence exceed them."""
import numpy as np
import pytest

from linear_states import (TENSOR, WEAK, large_parts_first, numbers, off, one_decay, one_sum, state64, two_parts,
                           walked)


@pytest.mark.parametrize("g", WEAK)
def test_one_decay_a_token_would_exceed_the_limits(g):
    n = 4000
    g = np.full(n, float(np.float32(g)))
    assert abs(np.float64(np.float32(np.exp(g[0]))) / np.exp(g[0]) - 1) > 0.9 * 2.0 ** -25
    x = numbers(1, n)
    assert off(one_decay(x[0], x[1], g, x[2]), state64(x[0], x[1], g, x[2])) > 3 * max(walked(n), TENSOR)


@pytest.mark.parametrize("n", [65, 517, 3000])
def test_two_parts_would_exceed_the_limit(n):
    g = -np.random.default_rng(2).exponential(0.02, n)
    x = numbers(3, n)
    assert off(two_parts(x[0], x[1], g, x[2]), state64(x[0], x[1], g, x[2])) > 3 * TENSOR


def test_one_sum_would_exceed_the_limit():
    """Tokens of one direction, so that the sums grow and what is cut off adds up."""
    n = 960
    g = np.full(n, -1e-4)
    k, v, first = numbers(4, n)
    k, v = np.abs(k), np.abs(v)
    assert off(one_sum(k, v, g, first), state64(k, v, g, first)) > 1.5 * TENSOR


def test_large_parts_first_would_exceed_the_limit():
    n = 704
    g = np.full(n, WEAK[1])
    k, v, first = numbers(4, n)
    k, v = np.abs(k), np.abs(v)
    assert off(large_parts_first(k, v, g, first), state64(k, v, g, first)) > 1.4 * TENSOR
