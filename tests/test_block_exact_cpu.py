"""The operands that tell fp32 sums from those of the 8-bit matrix instruction: exact in fp32 in any
order, and something else with that instruction's sums (planted here, in the reference)."""

import numpy as np
import pytest

import block_ref as R
from block_exact_ref import exact_operands, f32_bound, truncated


@pytest.mark.parametrize("d_in", [16, 144, 272, 384])
def test_fp32_sums_are_exact_and_truncation_shows(d_in):
    rng = np.random.default_rng(d_in)
    x, W = exact_operands(rng, 7, d_in, 9)
    p = R.decode(x)[:, None, :] * R.decode(W)[None, :, :]
    ref = p.sum(2)
    unit = 2.0**-6
    assert (p / unit == np.round(p / unit)).all() and np.abs(p).sum(2).max() / unit < 2.0**24
    for _ in range(5):
        total = np.zeros(ref.shape, dtype=np.float32)
        for k in rng.permutation(d_in):
            total += p[:, :, k].astype(np.float32)
        assert np.array_equal(total, ref)
    assert (truncated(x, W) != ref).mean() > 0.5


def test_the_bound_of_few_terms_tells_them_apart():
    """16 terms, the small products 2^2, below the last place (2^3) that is kept: what truncation loses of them
    is far more than the bound of fp32 sums."""
    rng = np.random.default_rng(2)
    x, W = exact_operands(rng, 30, 16, 40, small=64)
    one = np.ones((1, 30)), np.ones((1, 1))
    ref, mag, _ = R.linear(x, one[0], W, one[1])
    off = np.abs(truncated(x, W) - ref) > f32_bound(ref, mag, 16)
    assert off.mean() > 0.5
