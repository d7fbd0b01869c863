"""Values of the routed experts' operators at the edges of their types, and to
the last bit where the method fixes it."""
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ router

@pytest.mark.parametrize("E", [8, 64, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_infinity_counts_as_the_types_largest_value(E, dtype):
    big = torch.finfo(dtype).max
    logits = torch.zeros(3, E, dtype=dtype, device="cuda")
    logits[0, 3], logits[0, 5] = float("inf"), big
    logits[1, 2], logits[1, 6] = big, float("inf")
    logits[2, 1] = logits[2, 4] = float("inf")
    at = torch.tensor([[3, 5], [2, 6], [1, 4]], device="cuda")
    idx, w = B.moe_route(logits, 2, renormalize=False)
    assert torch.equal(idx.long(), at) and bool((w == 0.5).all())
    dw = torch.tensor([[1.0, 3.0]], device="cuda").repeat(3, 1)
    for renorm in (False, True):
        idx, w = B.moe_route(logits, 2, renormalize=renorm)
        dl = B.moe_route_bwd(logits, idx, w, dw, renormalize=renorm).float()
        want = torch.zeros(3, E, device="cuda").scatter_(1, at, torch.tensor([[-0.5, 0.5]], device="cuda").repeat(3, 1))
        assert torch.equal(dl, want)


@pytest.mark.parametrize("E", [32, 20, 128])
def test_route_softmax_of_fp32_logits_by_the_full_exponential(E):
    """Weights that are not renormalised, bit for bit: exp(l - max) / sum, the sum lane by lane and over the lanes in
    pairs."""
    g = _gen(E)
    logits = 3 * torch.randn(2000, E, generator=g, device="cuda")
    idx, w = B.moe_route(logits, 4, renormalize=False)
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    lanes = torch.zeros(2000, -(-E // 32) * 32, device="cuda")
    lanes[:, :E] = e
    lanes = lanes.view(2000, 32, -1)
    s = torch.zeros(2000, 32, device="cuda")
    for i in range(lanes.shape[2]):
        s = s + lanes[:, :, i]
    for o in (16, 8, 4, 2, 1):
        s = s + s[:, torch.arange(32, device="cuda") ^ o]
    assert torch.equal(w, e.gather(1, idx.long()) / s[:, :1])


# ------------------------------------------------------------------ dispatch

def _plan(g, T, k, E, align=128, empty=0.1):
    idx = torch.argsort(torch.rand(T, E, generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32)
    idx[torch.rand(T, generator=g, device="cuda") < empty] = -1
    return B.moe_plan(idx.contiguous(), E, align=align)


def _codes(X):
    """Codes and scales of the 1x128 groups of X [A, C], fp32, by IEEE quotients (C a multiple of 128)."""
    v = X.view(X.shape[0], -1, 128)
    amax = v.abs().amax(2)
    s = amax.clamp_min(1e-12) / torch.full_like(amax, 448.0)
    q = (v / s[:, :, None].expand_as(v)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(X.shape).view(torch.uint8), s.t()


@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_codes_are_those_of_the_quotient(weighted):
    g = _gen(3)
    T, k, E, K = 2048, 4, 16, 1024
    plan = _plan(g, T, k, E)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05 if weighted else None
    q, s, qc, sc = B.moe_dispatch(x, plan, weight=w)
    src = plan.src.long()
    X = x.float()[src.clamp_min(0) // k]
    if weighted:
        X = X * w.reshape(-1)[src.clamp_min(0)][:, None]
    X = torch.where((src >= 0)[:, None], X, torch.zeros((), device="cuda"))
    R = src.numel()
    for codes, scales, (want_q, want_s) in ((q[:, :K], s[:, :R], _codes(X)), (qc[:, :R], sc[:, :K], _codes(X.t().contiguous()))):
        assert torch.equal(scales, want_s)
        assert torch.equal(codes, want_q), f"{int((codes != want_q).sum())} of {codes.numel()} codes differ"


def test_dispatch_of_values_that_are_not_finite():
    """The same bytes as quantising the gathered rows, but for the sign of NaN codes, where a group holds infinities or
    NaN."""
    g = _gen(4)
    T, k, E, K = 200, 2, 4, 384
    plan = _plan(g, T, k, E)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    x[3, 5], x[7, 130], x[9, 200], x[20, :128] = float("inf"), -float("inf"), float("nan"), float("nan")
    x[30], x[40, ::2] = float("inf"), -float("nan")
    src = plan.src.long()
    xg = torch.where((src >= 0)[:, None], x[src.clamp_min(0) // k], torch.zeros((), dtype=x.dtype, device="cuda"))
    for got, want in zip(B.moe_dispatch(x, plan), B.quant_dual(xg.contiguous())):
        if got.dtype == torch.uint8:
            n = K if got.shape[0] == src.numel() else src.numel()
            a, b = (torch.where((t[:, :n] & 0x7F) == 0x7F, 0x7F, t[:, :n]) for t in (got, want))
            assert torch.equal(a, b) and bool((a == 0x7F).any()) and not bool((a == 0x7F).all())
        else:
            a, b = got[:want.shape[0], :want.shape[1]], want
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("N", [64, 1000, 4096])
@pytest.mark.parametrize("k", [1, 2, 3, 6, 9])
def test_combine_gradient_of_slots_without_a_row_is_zero(N, k):
    """Whatever dy and the weight hold there."""
    g = _gen(N + k)
    T, E = 33, 12
    idx = torch.argsort(torch.rand(T, E, generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32)
    idx[torch.rand(T, k, generator=g, device="cuda") < 0.3] = -1
    idx[5] = idx[6] = idx[7] = -1
    plan = B.moe_plan(idx.contiguous(), E, align=16)
    ye, dy = (torch.randn(n, N, generator=g, device="cuda").bfloat16() for n in (plan.src.numel(), T))
    dy[5], dy[6, 0], dy[8, 1] = float("inf"), float("nan"), -float("inf")
    w = torch.randn(T, k, generator=g, device="cuda")
    w[idx < 0] = float("nan")
    none = plan.row < 0
    y = B.moe_combine(ye, plan, w)
    assert bool(y.isfinite().all()) and not y[5].any()
    results = [B.moe_combine_bwd(dy, ye, plan, w, with_dye=d) for d in (True, False)]
    for dye, dw in results:
        assert not dw[none].any()
        assert not dw[none].isnan().any()
        if dye is not None:
            assert not dye[plan.src < 0].any()
    a, b = results[0][1], results[1][1]
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
