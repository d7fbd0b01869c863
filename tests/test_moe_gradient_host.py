"""The 64-bit form of the router's gradient against differences of the 64-bit
weights, where the chosen scores' sum is below its floor and above (CPU)."""
import numpy as np
import pytest

import moe_gradient_reference as gref
import moe_reference as ref


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_at_the_sum_floor(score, renorm):
    rows, bias = gref.FLOOR_ROWS[score]
    l, k, h = np.array(rows), 2, 1e-5
    dw = np.random.default_rng(0).normal(size=(len(rows), k))
    p, ok = ref.scores(l, score, -3e38)
    idx, _ = ref.choose(p, ok, l, score, bias, k, 1, 1, 1)
    S = np.take_along_axis(p, idx, 1).sum(1)
    assert (S < ref.SUM_FLOOR).any() and (S > ref.SUM_FLOOR).any()
    grad = gref.route_grad(p, idx, dw, score, renorm, 1.5)
    loss = lambda m: (dw * ref.weights(ref.scores(m, score, -3e38)[0], idx, renorm, 1.5)).sum(1)
    for e in range(l.shape[1]):
        step = h * np.eye(l.shape[1])[e]
        # h^2 / 6 times a third derivative below 20, 64-bit cancellation 1e-15 / h
        assert np.allclose(grad[:, e], (loss(l + step) - loss(l - step)) / (2 * h), rtol=0, atol=1e-9 + 1e-10)
