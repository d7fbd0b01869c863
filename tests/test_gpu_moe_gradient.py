"""The router's gradient where its terms are extreme, against the 64-bit formula."""
import numpy as np
import pytest

import moe_gradient_reference as gref
import moe_reference as ref
from gpu_util import torch

import blockwise_scaled_fp8_gb300 as B

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
F32_LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    yield
    B.check_device_errors()


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_at_the_sum_floor(score, renorm):
    rows, bias = gref.FLOOR_ROWS[score]
    logits = torch.tensor(rows, device="cuda")
    bias = None if bias is None else torch.tensor(bias, device="cuda")
    T, k, scale = len(rows), 2, 1.5
    dw = torch.randn(T, k, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    idx, w = B.moe_route(logits, k, score=score, bias=bias, renormalize=renorm, scale=scale)
    ln, ix = _f64(logits), idx.cpu().numpy()
    p, _ = ref.scores(ln, score, F32_LOWEST)
    wref = ref.weights(p, ix, renorm, scale)
    # a score: exp within 2 ulps, its argument |l| EPS at most 90; a sum, two divisions, a product
    tol = (90 + 2 * 2 + 4 + 8) * EPS
    assert np.all(np.abs(_f64(w) - wref) <= tol * np.abs(wref) + 1e-37)
    got = _f64(B.moe_route_bwd(logits, idx, w, dw, score=score, renormalize=renorm, scale=scale))
    want = gref.route_grad(p, ix, _f64(dw), score, renorm, scale)
    # each element: a few terms of this size, each with the weights' error
    pe = np.take_along_axis(p, ix, 1)
    size = scale * np.abs(_f64(dw)).max(1) * (pe.max(1) / np.maximum(pe.sum(1), ref.SUM_FLOOR) if renorm else pe.max(1))
    assert np.all(np.abs(got - want) <= 4 * tol * size[:, None] + 1e-37)


def test_gradient_of_weights_below_the_normal_range():
    """A scale so small that the weights lose bits, dw as large: the scores come from the logits, not from the weights."""
    T, E, k, scale = 16, 512, 4, 2.0 ** -140
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = 0.3 * torch.randn(T, E, generator=g, device="cuda")
    dw = 2.0 ** 100 * torch.randn(T, k, generator=g, device="cuda")
    idx, w = B.moe_route(logits, k, renormalize=False, scale=scale)
    got = _f64(B.moe_route_bwd(logits, idx, w, dw, renormalize=False, scale=scale))
    ix = idx.cpu().numpy()
    p, _ = ref.scores(_f64(logits), "softmax", F32_LOWEST)
    want = gref.route_grad(p, ix, _f64(dw), "softmax", False, scale)
    # scores: exp of arguments below 4, a sum of E / 32 + 5 additions, a quotient, products
    tol = (4 + 2 * 2 + E / 32 + 5 + 8) * EPS
    size = scale * np.abs(_f64(dw)).max(1) * np.take_along_axis(p, ix, 1).max(1)
    assert np.all(np.abs(got - want) <= 4 * tol * size[:, None] + 1e-37)
