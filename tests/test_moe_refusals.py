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


@pytest.mark.parametrize("columns", [120, 250, 304])
def test_training_forward_refuses_another_width_of_tokens(columns):
    """Fewer columns than the weights' (their codes' padding would be read) and more."""
    w = torch.zeros(4, 128, 256 if columns > 128 else 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=f"x has {columns} features"):
        B.moe_experts_fwd(torch.zeros(8, columns, dtype=torch.bfloat16), w, _plan(8, 2, 4, 128), torch.zeros(8, 2))


@pytest.mark.parametrize("columns,K", [(128, 256), (256, 512), (300, 256), (1024, 896)])
def test_decoding_refuses_another_width_of_tokens(columns, K):
    qw, sw = _quantised(4, 128, K)
    with pytest.raises(ValueError, match=f"x has {columns} features"):
        B.moe_experts_decode(torch.zeros(8, columns, dtype=torch.bfloat16), qw, sw, _plan(8, 2, 4, 1), torch.zeros(8, 2), 128)


def test_decoding_takes_padded_codes_or_scales():
    """Row strides beyond the weight's width are no other width: these fail at the tensors' device only."""
    qw, sw = _quantised(4, 128, 200)
    for q, s in ((torch.zeros(512, 256, dtype=torch.uint8), sw), (qw, torch.zeros(4, 5))):
        with pytest.raises(ValueError, match="x must be"):
            B.moe_experts_decode(torch.zeros(8, 200, dtype=torch.bfloat16), q, s, _plan(8, 2, 4, 1), torch.zeros(8, 2), 128)


@pytest.mark.parametrize("T,k,E,align", [(64, 2, 8, 1), (256, 4, 8, 1), (128, 1, 2, 64), (130, 3, 16, 32), (512, 2, 4, 8)])
def test_training_forward_refuses_plans_whose_experts_start_off_a_block(T, k, E, align):
    """Also where the rows in all happen to be a multiple of 128."""
    w = torch.zeros(E, 128, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiples of 128"):
        B.moe_experts_fwd(torch.zeros(T, 128, dtype=torch.bfloat16), w, _plan(T, k, E, align), torch.zeros(T, k))


@pytest.mark.parametrize("T,k,E,align", [(64, 2, 8, 128), (1, 1, 1, 128), (300, 2, 4, 256), (128, 1, 1, 1), (3, 2, 1024, 128)])
def test_training_forward_takes_every_plan_on_blocks(T, k, E, align):
    """One expert starts on a block whatever the alignment; these fail at the tensors' device only."""
    w = torch.zeros(E, 128, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be"):
        B.moe_experts_fwd(torch.zeros(T, 128, dtype=torch.bfloat16), w, _plan(T, k, E, align), torch.zeros(T, k))
