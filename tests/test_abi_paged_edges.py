"""Edges of the calls on the 8-bit paged cache and of the rotary frequencies that need no GPU."""
import math

import numpy as np
import pytest

import exact_io_aware_55_b200 as fa


@pytest.mark.parametrize("scaling,high", [("yarn", 32.0), ("bands", 4.0)])
def test_rope_frequencies_default_edges_are_the_scaling_s_own(scaling, high):
    """Without low and high: 1 and 32 turns for the ramp over pairs, 1 and 4 for the bands."""
    rot, base, factor, length = 128, 10000.0, 8.0, 4096.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    if scaling == "yarn":
        pair = lambda t: rot * math.log(length / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        first, last = math.floor(pair(high)), math.ceil(pair(1.0))
        keep = 1 - np.clip((i - first) / (last - first), 0, 1)
    else:
        keep = np.clip((length * f / (2 * math.pi) - 1) / (high - 1), 0, 1)
    got, _ = fa.rope_frequencies(rot, base, scaling, factor, length, device="cpu")
    assert np.allclose(got.numpy(), f / factor * (1 - keep) + f * keep, rtol=1e-13)
    same, _ = fa.rope_frequencies(rot, base, scaling, factor, length, 1.0, high, device="cpu")
    assert np.array_equal(got.numpy(), same.numpy())
