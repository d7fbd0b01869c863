"""Which elements the routed experts' kernels touch, replayed on the host from
their own index arithmetic (no GPU)."""
import numpy as np
import pytest

import blockwise_scaled_fp8_gb300 as B
from blockwise_scaled_fp8_gb300 import buildlib as bbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    bbuild.build()


# Widths whose rows share a CTA (up to 1024 columns at eight an access, 512 at four, 256 at two, 128 at one), have one
# to themselves, and need several; token counts that leave the last CTA partly empty
WIDTHS = [(0, N) for N in (1, 3, 64, 101, 128, 129, 300)] + [(1, N) for N in (2, 130, 256, 258, 600)] + \
    [(2, N) for N in (4, 260, 512, 516, 1100)] + [(3, N) for N in (8, 24, 256, 512, 1000, 1024, 1032, 2048, 4096, 5000)]


@pytest.mark.parametrize("log_vec,N", WIDTHS)
@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 9, 32])
def test_combine_touches_each_element_once(log_vec, N, k):
    vec = 1 << log_vec
    sides = max(256 // -(-N // vec), 1)
    for T in sorted({1, 5, 40, 97, max(sides - 1, 1), sides, sides + 1, 3 * sides + 2}):
        y, slots, oob = B.debug_write_counts(7, T, N, k, log_vec << 4)
        assert oob == 0, (T, oob)
        assert y.shape == (T, N) and np.all(y == 1)
        assert slots.shape == (T, k) and np.all(slots >= 1)


def test_combine_replay_refuses_what_no_launch_has():
    for bad in ((4, 9, 2, 1 << 4), (4, 8, 0, 0), (4, 8, 33, 0)):
        with pytest.raises(B.Bfp8Error, match="out of range"):
            B.debug_write_counts(7, *bad)
