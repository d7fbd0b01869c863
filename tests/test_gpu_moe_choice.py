"""The router's choice token by token against the 64-bit form: the same expert,
unless what is compared lies closer together than fp32 scores can tell."""
import numpy as np
import pytest

import moe_reference as ref
from gpu_util import torch

import blockwise_scaled_fp8_gb300 as B

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
LOWEST = {torch.bfloat16: float(torch.finfo(torch.bfloat16).min), torch.float32: float(torch.finfo(torch.float32).min)}


def check_choice(got, want, value, groups, top_groups, group_score, tol_v, tol_g):
    """got, want [k]; value [E]: what is compared within the kept groups (-inf: not eligible); group_score [groups].
    Returns whether the token's groups were near each other."""
    S = value.size // groups
    live = np.sort(group_score[group_score > -np.inf])[::-1]
    edge = live[top_groups - 1] if live.size > top_groups else -np.inf
    with np.errstate(invalid="ignore"):           # groups without an expert
        off = np.abs(group_score - edge)
    near = bool(((off > 0) & (off <= tol_g)).any())
    if not near:  # the kept groups are certain
        for a, b in zip(got, want):
            if a != b:
                assert a >= 0 and b >= 0 and 0 < abs(value[a] - value[b]) <= tol_v, (got, want)
        return False
    chosen = got[got >= 0]
    of = chosen // S
    assert len(set(of)) <= top_groups
    assert (group_score[of] >= edge - tol_g).all()
    certain = np.repeat(group_score > edge + tol_g, S)
    left = np.ones(value.size, bool)
    left[chosen] = False
    best_left = value[certain & left].max(initial=-np.inf)
    assert best_left <= (value[chosen].min() + tol_v if chosen.size == got.size else -np.inf)
    assert (np.diff(value[chosen]) <= tol_v).all()
    return True


def group_scores(c, ok, groups, group_top):
    v = np.where(ok, c, -np.inf).reshape(c.shape[0], groups, -1)
    top = -np.sort(-v, axis=2)[:, :, :group_top]
    score = np.where(top > -np.inf, top, 0).sum(2)
    return np.where(top[:, :, 0] > -np.inf, score, -np.inf)


# T, E, k, score, bias, groups, top_groups, group_top
CASES = [(600, 160, 6, "softmax", False, 8, 3, 1), (600, 160, 8, "softmax", False, 8, 3, 2),
         (400, 256, 8, "sigmoid", True, 8, 4, 2), (400, 256, 8, "sigmoid", False, 8, 4, 1),
         (500, 96, 5, "sigmoid", True, 3, 2, 2), (500, 96, 5, "softmax", True, 6, 2, 2),
         (60, 1024, 32, "softmax", False, 32, 17, 2), (300, 32, 8, "sigmoid", True, 32, 9, 2),
         (300, 64, 6, "softmax", False, 1, 1, 1), (300, 64, 6, "sigmoid", True, 1, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k,score,with_bias,groups,top_groups,group_top", CASES)
def test_choice_token_by_token(T, E, k, score, with_bias, groups, top_groups, group_top, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E + k + groups)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(dtype)
    logits[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -float("inf")
    logits[1] = 0.25                                  # equal everywhere: the lowest groups, the lowest experts
    logits[2, E // 2:] = -float("inf")
    logits[3] = -float("inf")
    bias = None
    if with_bias:
        bias = 0.1 * torch.randn(E, generator=g, device="cuda")
        bias[E // 3] = -float("inf")
    idx, _ = B.moe_route(logits, k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top)
    got, ln, bn = idx.cpu().numpy(), logits.float().cpu().numpy(), None if bias is None else bias.cpu().numpy()
    p, ok = ref.scores(ln, score, LOWEST[dtype])
    want, _ = ref.choose(p, ok, ln, score, bn, k, groups, top_groups, group_top)
    by_logit = score == "softmax" and not with_bias
    with np.errstate(invalid="ignore"):
        c = p if bn is None else p + bn.astype(np.float64)
        ok = ok & (c > -np.inf)
    value = np.where(ok, ln.astype(np.float64) if by_logit else c, -np.inf)
    # A score: exp (2 ulps, and its argument's rounding, below 24 here), a sum of E / 32 + 5 terms, a division and the
    # bias, all of values below 1.5; a group's: two of them and their sum.
    tol_v = 0.0 if by_logit else (2 * 2 + 24 + E / 32 + 5 + 2 + 2) * EPS
    tol_g = 2 * 1.5 * (2 * 2 + 24 + E / 32 + 5 + 2 + 2) * EPS
    gs = group_scores(c, ok, groups, group_top) if groups > 1 else np.zeros((T, 1))
    near = sum(check_choice(got[t], want[t], value[t], groups, top_groups, gs[t], tol_v, tol_g) for t in range(T))
    assert near <= T // 4                             # nearly every token's groups are certain
