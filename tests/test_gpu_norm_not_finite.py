"""The norm's gradient of gradients that are not finite: infinities and NaN come out where the formula has them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64


def kinds(v):
    """0 finite, +-1 infinities, 2 NaN."""
    return torch.where(v.isnan(), 2, torch.where(v.isinf(), v.sign().nan_to_num(), torch.zeros_like(v))).to(torch.int32)


@pytest.mark.parametrize("T,K", [(3, 64), (700, 1000), (1300, 1003), (2000, 4096), (90, 16384)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_gradients_that_are_not_finite(T, K, value):
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, w, dy = n(T, K).to(bf16), 1 + 0.1 * n(K), n(T, K).to(bf16)
    h[h == 0] = 1
    r, k = T // 2, K // 3
    dy[r, k] = value
    rstd = B.rms_norm_quant(h, w).rstd
    dx, dw = B.rms_norm_bwd(dy, h, w, rstd)
    B.check_device_errors()
    norm, grad = h.to(f64) * rstd.to(f64)[:, None], dy.to(f64) * w.to(f64)
    ref = rstd.to(f64)[:, None] * (grad - norm * (grad * norm).mean(1, keepdim=True))
    assert torch.equal(kinds(dw), kinds((dy.to(f64) * norm).sum(0)))
    assert torch.equal(kinds(dx.float()), kinds(ref))


def test_a_sum_that_passes_fp32():
    """Terms of one sign whose sum no fp32 holds: infinite, as a plain sum of them in fp32 is."""
    T, K = 64, 256
    h = torch.ones(T, K, device="cuda", dtype=bf16)
    w = torch.ones(K, device="cuda")
    dy = torch.zeros(T, K, device="cuda", dtype=bf16)
    dy[:, 5], dy[:, 9] = 3e38, -3e38
    _, dw = B.rms_norm_bwd(dy, h, w, B.rms_norm_quant(h, w).rstd)
    assert float(dw[5]) == float("inf") and float(dw[9]) == float("-inf") and float(dw[6]) == 0
