"""Calls of the routed experts whose answers would be wrong are refused before
anything runs (host logic; no GPU)."""
import pytest
import torch

import blockwise_scaled_fp8_gb300 as B
from blockwise_scaled_fp8_gb300 import buildlib as bbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    bbuild.build()


def _plan(T, k, E, align):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    return B.MoePlan(i(E + 1), i(T, k), i(B.moe_plan_rows(T, k, E, align)), i(E))


def _quantised(E, N, K):
    """The shapes that quant_weight(w.reshape(E * N, K)) returns."""
    return (torch.zeros(E * N, -(-K // 16) * 16, dtype=torch.uint8), torch.zeros(-(-E * N // 128), -(-K // 128)))


# The stacked weight's tiles straddle experts; the count of its rows of scales is that of whole tiles an expert in the
# first three
@pytest.mark.parametrize("E,N", [(2, 1000), (5, 1000), (8, 120), (4, 200), (3, 1)])
def test_decoding_refuses_tiles_that_straddle_experts(E, N):
    qw, sw = _quantised(E, N, 256)
    with pytest.raises(ValueError, match="multiple of 128"):
        B.moe_experts_decode(torch.zeros(4, 256, dtype=torch.bfloat16), qw, sw, _plan(4, 2, E, 1), torch.zeros(4, 2), N)
