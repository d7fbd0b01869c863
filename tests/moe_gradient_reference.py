"""The router's gradient in 64 bits, with the floor of the chosen scores' sum:
w = scale p / max(sum p, floor), whose denominator is a constant below the
floor."""
import numpy as np

from moe_reference import SUM_FLOOR


def route_grad(p, idx, dw, score, renormalize, scale):
    """d(sum dw w) / d logits of p [T, E], idx and dw [T, k]."""
    out = np.zeros(p.shape)
    for t in range(p.shape[0]):
        on = idx[t] >= 0
        e = idx[t][on]
        d, pe = scale * dw[t][on], p[t, e]
        if renormalize:
            S = pe.sum()
            d = (d - (d * pe).sum() / S) / S if S > SUM_FLOOR else d / SUM_FLOOR
        if score == "sigmoid":
            out[t, e] = d * pe * (1 - pe)
        else:
            out[t] = -p[t] * (d * pe).sum()
            out[t, e] += d * pe
    return out


# Rows of logits [E] (with a softmax's bias [E], or None) whose chosen scores sum to less than the floor, to more, and
# to nearly it
FLOOR_ROWS = {
    "sigmoid": ([[-47.0, -47.3, -90.0, -60.0], [-47.0, -46.9, -48.0, -47.5], [-45.0, -45.2, -46.0, -44.9],
                 [-80.0, -79.0, -81.0, -82.0], [-46.0, 1.0, -47.0, -48.0], [-46.7, -47.0, -47.1, -47.2]], None),
    "softmax": ([[0.0, -48.0, -47.5, -49.0], [0.0, -46.0, -60.0, -47.2], [0.0, -44.0, -45.0, -44.5],
                 [0.0, -70.0, -71.0, -70.5]], [-10.0, 0.0, 0.0, 0.0]),
}
