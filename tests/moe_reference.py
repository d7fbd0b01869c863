"""Plain 64-bit forms of the mixture-of-experts operators, one token, row or
group at a time, shared by the CPU and GPU tests."""
import numpy as np

SUM_FLOOR = 1e-20
E4M3_MAX, AMAX_FLOOR = 448.0, 1e-12


def scores(logits, score, lowest):
    """(p, eligible) of logits [T, E] (values as the kernel reads them)."""
    l = np.asarray(logits, np.float64)
    with np.errstate(invalid="ignore"):
        ok = l > lowest
    l = np.where(ok, np.minimum(l, -lowest), -np.inf)
    p = np.zeros_like(l)
    for t in range(l.shape[0]):
        if not ok[t].any():
            continue
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                p[t] = np.where(ok[t], 1 / (1 + np.exp(-l[t])), 0)
        else:
            e = np.exp(l[t] - l[t].max())
            p[t] = e / e.sum()
    return p, ok


def choose(p, ok, logits, score, bias, k, groups, top_groups, group_top):
    """idx [T, k], and the values [T, E] that were compared (-inf: not eligible)."""
    T, E = p.shape
    c = p if bias is None else p + np.asarray(bias, np.float64)
    order_by_logit = score == "softmax" and bias is None
    with np.errstate(invalid="ignore"):
        ok = ok & (c > -np.inf)
    value = np.where(ok, np.asarray(logits, np.float64) if order_by_logit else c, -np.inf)
    idx = np.full((T, k), -1, np.int32)
    for t in range(T):
        if groups > 1:
            S = E // groups
            gs = []
            for g in range(groups):
                v = np.sort(c[t, g * S:(g + 1) * S][ok[t, g * S:(g + 1) * S]])[::-1][:group_top]
                gs.append(v.sum() if v.size else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept or gs[g] == -np.inf:
                    value[t, g * S:(g + 1) * S] = -np.inf
        best = sorted((e for e in range(E) if value[t, e] > -np.inf), key=lambda e: (-value[t, e], e))[:k]
        idx[t, :len(best)] = best
    return idx, value


def weights(p, idx, renormalize, scale):
    w = np.where(idx >= 0, np.take_along_axis(p, np.maximum(idx, 0), 1), 0.0)
    if renormalize:
        w = w / np.maximum(w.sum(1, keepdims=True), SUM_FLOOR)
    return scale * w


def route_grad(p, idx, dw, score, renormalize, scale):
    """d(sum dw w) / d logits, by the formulas."""
    T, E = p.shape
    out = np.zeros((T, E))
    for t in range(T):
        j = idx[t] >= 0
        e = idx[t][j]
        d, pe = scale * dw[t][j], p[t, e]
        if renormalize:
            S = max(pe.sum(), SUM_FLOOR)
            d = (d - (d * pe).sum() / S) / S
        if score == "sigmoid":
            out[t, e] = d * pe * (1 - pe)
        else:
            out[t] = -p[t] * (d * pe).sum()
            out[t, e] += d * pe
    return out


def plan(idx, E, align, R):
    """(offs, row, src, counts) by appending slots to their experts' lists."""
    T, k = idx.shape
    lists = [[] for _ in range(E)]
    for slot, e in enumerate(idx.reshape(-1)):
        if 0 <= e < E:
            lists[e].append(slot)
    offs, src, row = [0], np.full(R, -1, np.int32), np.full(T * k, -1, np.int32)
    for e in range(E):
        for i, slot in enumerate(lists[e]):
            src[offs[e] + i] = slot
            row[slot] = offs[e] + i
        offs.append(offs[e] + -(-len(lists[e]) // align) * align)
    return np.array(offs, np.int32), row.reshape(T, k), src, np.array([len(v) for v in lists], np.int32)


def gathered(x, src, k, weight=None):
    """X [R, K] of the dispatch in 64 bits."""
    out = np.zeros((src.size, x.shape[1]))
    on = src >= 0
    out[on] = np.asarray(x, np.float64)[src[on] // k]
    if weight is not None:
        out[on] *= np.asarray(weight, np.float64).reshape(-1)[src[on]][:, None]
    return out


def combine(ye, row, w):
    T, k = row.shape
    y = np.zeros((T, ye.shape[1]))
    for t in range(T):
        for j in range(k):
            if row[t, j] >= 0:
                y[t] += (1.0 if w is None else w[t, j]) * ye[row[t, j]]
    return y


def combine_grad(dy, ye, row, src, w):
    T, k = row.shape
    dw, dye = np.zeros((T, k)), np.zeros(ye.shape)
    for t in range(T):
        for j in range(k):
            if row[t, j] >= 0:
                dw[t, j] = dy[t] @ ye[row[t, j]]
    for r, slot in enumerate(src):
        if slot >= 0:
            dye[r] = w.reshape(-1)[slot] * dy[slot // k]
    return dye, dw
