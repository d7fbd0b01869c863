"""The weight-gradient GEMM that quantises X itself, call after call: the bits
of the two-launch path every time (its raw tiles are refilled by asynchronous
copies while other warps still work on the values read from them)."""
import pytest

from gpu_util import torch

import blockwise_scaled_fp8_gb300 as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    yield
    B.check_device_errors()


@pytest.mark.parametrize("M,N,K,calls", [(4096, 4096, 8192, 1000), (1024, 4096, 16384, 500), (512, 2048, 4096, 1000)])
def test_wgrad_xq_repeats_the_two_launch_path(M, N, K, calls):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    dy, x = (torch.randn(K, n, generator=g, device="cuda").bfloat16() for n in (M, N))
    qa, sa = B.quant_lhs(dy, transposed=True)
    qb, sb = B.quant_rhs(x)
    ref = B.gemm_1x128_128x1(qa, sa, qb, sb, K, M=M, N=N).view(torch.int16)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(calls):
        B.gemm_1x128_128x1_xq(qa, sa, x, out=out, M=M)
        wrong += (out.view(torch.int16) != ref).any()
    assert int(wrong) == 0, f"{int(wrong)} of {calls} calls differ"
