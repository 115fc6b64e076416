"""The oracle's bound on the kernels' roundings is a bound on what they may lose,
too: a result without the keys under a dominant one does not pass (CPU)."""
import math

import numpy as np
import pytest

from oracle.page_scaled_fp64 import page_scaled_oracle


@pytest.mark.parametrize("n", [1024, 8192])
@pytest.mark.parametrize("weight", [0.5, 0.8])
def test_losing_all_other_keys_is_outside_the_bound(n, weight):
    rng = np.random.default_rng(n)
    pages = n // 16
    q, k = np.zeros((1, 1, 8)), np.zeros((pages, 16, 1, 8))
    v = 1.0 + rng.standard_normal((pages, 16, 1, 8))
    k[0, 0], v[0, 0] = 0.0, 0.0
    k[0, 0, 0, 0] = 1.0
    q[0, 0, 0] = math.log(weight / (1 - weight) * (n - 1))
    one = np.ones((pages, 1))
    out, tol = page_scaled_oracle(q, k, v, one, one, np.arange(pages)[None], np.array([0, 1]), np.array([n]), 1.0)
    # Q's two terms may move the logit of the dominant key (at most 10.4) by 2^-8 of
    # it: e^(2 * 0.041) - 1 = 8.5 % of sum w |v|, which is 1.2 times |out| here
    assert (tol < 0.2 * np.abs(out)).all()
    assert (np.abs(0.0 - out) > tol).all() and (np.abs(0.75 * out - out) > tol).all()
