"""Scales that the attention of drafted tokens refuses or takes, checked on the
host: the refusal comes before the workspace's, so a missing workspace tells
a scale that was taken. No GPU."""
import numpy as np
import pytest

from long_context_prefill_dhsa_b200 import binding, build

FAKE = 1 << 20   # a non-null, aligned stand-in pointer; never dereferenced
INVALID, WORKSPACE = 1, 5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("scale,weights,want", [
    (2.3e38, False, WORKSPACE), (2.4e38, False, INVALID), (3.4e38, False, INVALID), (np.inf, False, INVALID),
    (1e-45, False, WORKSPACE), (0.0, False, INVALID), (-0.0, False, INVALID), (np.nan, False, INVALID),
    (1e-30, True, WORKSPACE), (9e-31, True, INVALID), (1e30, True, WORKSPACE), (1.1e30, True, INVALID),
])
def test_scales(lib, scale, weights, want):
    w = FAKE if weights else None
    got = lib.dhsa_tree_attn(FAKE, FAKE, None, FAKE, None, 1, 2, 1, 1, 50, 128, FAKE, None, None, scale, FAKE + 4096,
                             None, w, w, None, 0, None)
    assert got == want


def test_scales_that_are_taken_are_finite_in_powers_of_two():
    """The kernel multiplies by scale * log2(e) in fp32: inf there would make 0 * inf of the best score's difference."""
    log2e = np.float32(1.4426950408889634)
    assert np.isfinite(np.float32(2.3e38) * log2e)
    with np.errstate(over="ignore"):
        assert not np.isfinite(np.float32(2.4e38) * log2e)
