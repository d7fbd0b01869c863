"""Mixture-of-experts operators against their 64-bit forms (moe_reference.py),
and the dispatch and the routed product against the entries they replace."""
import ctypes

import numpy as np
import pytest

import moe_reference as ref
import oracle as O
from gpu_util import assert_gemm_close, torch

import blockwise_scaled_fp8_gb300 as B

pytestmark = pytest.mark.gpu

BF16_LOWEST = float(np.float32(np.uint32(0xFF7F0000).view(np.float32)))
F32_LOWEST = float(np.finfo(np.float32).min)
EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    O.build()
    yield
    B.check_device_errors()


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------ router

# T, E, k, score, bias, groups, top_groups, group_top, renormalize, scale
ROUTE = [
    (1, 64, 6, "softmax", False, 1, 1, 1, True, 1.0),
    (1, 1, 1, "sigmoid", False, 1, 1, 1, False, 1.0),
    (33, 8, 2, "softmax", False, 1, 1, 1, True, 1.0),
    (70, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (70, 160, 8, "softmax", False, 8, 3, 2, True, 1.0),
    (65, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (65, 96, 5, "sigmoid", True, 3, 2, 2, False, 1.0),
    (40, 100, 4, "softmax", True, 1, 1, 1, True, 1.0),
    (40, 37, 32, "sigmoid", False, 1, 1, 1, True, 1.0),
    (9, 1024, 32, "softmax", False, 32, 17, 2, True, 1.0),
    (9, 500, 3, "sigmoid", True, 1, 1, 1, True, 1.0),
    (17, 32, 8, "sigmoid", True, 32, 9, 2, True, 1.0),   # groups of one expert
]


def _masked_logits(g, T, E, dtype):
    """Logits with every kind of mask: some experts, whole rows, few experts left."""
    l = 2 * _randn(g, T, E, dtype=dtype)
    l[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -float("inf")
    if T > 8:
        l[1] = -float("inf")
        l[2] = torch.finfo(dtype).min
        l[3] = float("nan")
        l[4, 1:] = -float("inf")       # one expert left
        l[5, 0] = float("inf")         # one expert without bound
        l[6] = 0.25                    # all equal: the lowest indices
        l[7, ::2] = -0.0
        l[7, 1::2] = 0.0               # the zeros are equal
    return l


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", ROUTE)
def test_route_and_gradient(case, dtype):
    T, E, k, score, with_bias, groups, top_groups, group_top, renorm, scale = case
    g = _gen(T * 7 + E + k)
    logits = _masked_logits(g, T, E, dtype)
    bias = 0.1 * _randn(g, E) if with_bias else None
    if with_bias and E > 8:
        bias[E // 2] = -float("inf")   # an expert switched off
    how = dict(score=score, renormalize=renorm, scale=scale)
    idx, w = B.moe_route(logits, k, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top, **how)
    lowest = BF16_LOWEST if dtype == torch.bfloat16 else F32_LOWEST
    ln = logits.float().cpu().numpy()
    bn = None if bias is None else bias.cpu().numpy()
    p, ok = ref.scores(ln, score, lowest)
    want, value = ref.choose(p, ok, ln, score, bn, k, groups, top_groups, group_top)
    got = idx.cpu().numpy()
    # where the choices differ the compared values are as good as equal: fp32
    # scores are within 4 EPS of 1 of the 64-bit ones (groups: sums of two)
    for t, j in np.argwhere(got != want):
        a, b = got[t, j], want[t, j]
        assert a >= 0 and b >= 0, (t, j, a, b)
        assert not (score == "softmax" and not with_bias and groups == 1), (t, j, a, b)
        if groups == 1:
            assert abs(value[t, a] - value[t, b]) <= 8 * EPS, (t, j, a, b)
    assert (got != want).mean() <= 0.01 or groups == 1
    for t in range(T):
        live = got[t][got[t] >= 0]
        assert len(set(live)) == len(live) and np.all(got[t][len(live):] == -1)
    # weights: exp within 2 ulps, its argument's subtraction |l - max| EPS (below 40 EPS for what is chosen
    # here), a sum of E / 32 + 5 additions, two divisions and a product
    wref = ref.weights(p, got, renorm, scale)
    tol = (40 + 8 + E / 32 + 5 + 8) * EPS
    assert np.all(np.abs(_f64(w) - wref) <= tol * np.abs(wref) + 1e-37)

    dw = _randn(g, T, k)
    dl = B.moe_route_bwd(logits, idx, w, dw, **how)
    assert dl.dtype == dtype and dl.shape == logits.shape
    dref = ref.route_grad(p, got, _f64(dw), score, renorm, scale)
    # every term carries the weights' error: relative to the row's largest dw scale p (/ S), plus the output's rounding
    pe = np.where(got >= 0, np.take_along_axis(p, np.maximum(got, 0), 1), 0.0)
    size = scale * np.abs(_f64(dw)).max(1) * (pe.max(1) / np.maximum(pe.sum(1), 1e-20) if renorm else pe.max(1))
    out_eps = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    bound = out_eps * np.abs(dref) + 4 * tol * size[:, None] + 1e-37
    assert np.all(np.abs(_f64(dl) - dref) <= bound)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_gradient_against_differences(score, renorm):
    T, E, k, scale, h = 5, 24, 4, 1.5, 1e-5
    g = _gen(3)
    logits, dw = _randn(g, T, E), _randn(g, T, k)
    idx, w = B.moe_route(logits, k, score=score, renormalize=renorm, scale=scale)
    dl = _f64(B.moe_route_bwd(logits, idx, w, dw, score=score, renormalize=renorm, scale=scale))
    ln, dn, ix = _f64(logits), _f64(dw), idx.cpu().numpy()

    def loss(l):
        p, _ = ref.scores(l, score, F32_LOWEST)
        return (dn * ref.weights(p, ix, renorm, scale)).sum(1)

    for e in range(E):
        step = np.zeros(E)
        step[e] = h
        diff = (loss(ln + step) - loss(ln - step)) / (2 * h)
        # central differences: h^2 / 6 times a third derivative below 10, 64-bit cancellation 1e-16 / h; fp32 kernel
        assert np.all(np.abs(dl[:, e] - diff) <= 1e-9 + 1e-10 + 1e-5)


def test_route_strided_logits_and_stream():
    g = _gen(5)
    wide = _randn(g, 50, 91, dtype=torch.bfloat16)
    logits = wide[:, 3:80]                       # odd width, odd offset, row stride 91
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        idx, w = B.moe_route(logits, 5)
        dl = B.moe_route_bwd(logits, idx, w, torch.ones_like(w))
    torch.cuda.current_stream().wait_stream(side)
    idx2, w2 = B.moe_route(logits.contiguous(), 5)
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    assert torch.equal(dl, B.moe_route_bwd(logits.contiguous(), idx2, w2, torch.ones_like(w)))


# ------------------------------------------------------------------ plan

# T, k, E, align
PLANS = [(1, 1, 1, 1), (1, 8, 64, 1), (48, 8, 256, 1), (33, 3, 7, 128), (1000, 6, 160, 128), (4100, 2, 8, 16),
         (20000, 8, 256, 128), (20000, 1, 1024, 1), (70000, 4, 3, 64)]


@pytest.mark.parametrize("T,k,E,align", PLANS)
def test_plan(T, k, E, align):
    rng = np.random.default_rng(T + k + E)
    idx = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    if T > 30:
        idx[5:9] = -1
        idx[10] = E + 3                              # out of range: goes nowhere
        idx[11] = -7
        idx[12:30] = E // 2                          # one expert liked by many, a token's choices all equal
    p = B.moe_plan(torch.from_numpy(idx).cuda(), E, align=align)
    assert p.src.numel() == B.moe_plan_rows(T, k, E, align)
    offs, row, src, counts = ref.plan(idx, E, align, p.src.numel())
    assert np.array_equal(p.offs.cpu().numpy(), offs)
    assert np.array_equal(p.counts.cpu().numpy(), counts)
    assert np.array_equal(p.row.cpu().numpy(), row)
    assert np.array_equal(p.src.cpu().numpy(), src)


def test_plan_of_no_tokens():
    p = B.moe_plan(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert p.src.numel() == 0 and p.row.shape == (0, 4)
    assert not p.offs.any() and not p.counts.any()


# ------------------------------------------------------------------ dispatch

def _routed(seed, T, k, E, align, empty=0.1):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)]).astype(np.int32)
    idx[idx >= E] = -1
    idx[rng.random(T) < empty] = -1
    return B.moe_plan(torch.from_numpy(idx).cuda(), E, align=align)


# T, k, E, align, K
DISPATCH = [(1, 1, 1, 1, 128), (5, 2, 3, 128, 256), (130, 2, 8, 128, 384), (300, 8, 16, 128, 520), (77, 3, 5, 1, 1000),
            (64, 6, 40, 16, 136), (700, 4, 8, 128, 1288), (50, 2, 4, 128, 8)]


@pytest.mark.parametrize("cols", [True, False])
@pytest.mark.parametrize("T,k,E,align,K", DISPATCH + [(41, 2, 4, 128, 101), (90, 3, 6, 8, 1)])
def test_dispatch_equals_quantising_the_gathered_rows(T, k, E, align, K, cols):
    plan = _routed(T + K, T, k, E, align)
    g = _gen(K)
    x = _randn(g, T, K, dtype=torch.bfloat16)
    q, s, qc, sc = B.moe_dispatch(x, plan, cols=cols)
    src = plan.src.long()
    xg = torch.where((src >= 0)[:, None], x[src.clamp_min(0) // k], torch.zeros((), dtype=x.dtype, device="cuda"))
    R, Kb = src.numel(), -(-K // 128)
    q2, s2, qc2, sc2 = B.quant_dual(xg.contiguous())
    assert torch.equal(q[:, :K], q2[:, :K])
    assert torch.equal(s[:Kb, :R], s2[:Kb, :R])
    if cols:
        assert torch.equal(qc[:, :R], qc2[:, :R])
        assert torch.equal(sc[:, :K], sc2[:, :K])
    else:
        assert qc is None and sc is None


def _check_codes(codes, scale, value):
    """Codes [G, n] of groups with one scale [G] each, against the 64-bit values."""
    amax = np.maximum(np.abs(value).max(1), ref.AMAX_FLOOR)
    # the scale: a product and a division, each within half an ulp of its operands'
    assert np.all(np.abs(scale - amax / ref.E4M3_MAX) <= 4 * EPS * amax / ref.E4M3_MAX)
    v = value / scale[:, None]
    half = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 4)  # half a step of e4m3 at |v|
    assert np.all(np.abs(codes - v) <= half + 8 * EPS * np.abs(v))


@pytest.mark.parametrize("T,k,E,align,K", DISPATCH[:-1] + [(41, 2, 4, 128, 101)])
def test_dispatch_with_weights(T, k, E, align, K):
    plan = _routed(T + K + 1, T, k, E, align)
    g = _gen(K + 1)
    x = _randn(g, T, K, dtype=torch.bfloat16)
    w = _randn(g, T, k)                              # both signs
    w[0, 0] = 0.0
    q, s, qc, sc = B.moe_dispatch(x, plan, weight=w)
    X = ref.gathered(_f64(x), plan.src.cpu().numpy(), k, _f64(w))
    R = X.shape[0]
    code = lambda t, n: _f64(t[:, :n].contiguous().view(torch.float8_e4m3fn))
    cr, cc = code(q, K), code(qc, R)
    sr, sct = _f64(s), _f64(sc)
    for kb in range(-(-K // 128)):
        b = slice(128 * kb, min(128 * kb + 128, K))
        _check_codes(cr[:, b], sr[kb], X[:, b])
    for rb in range(-(-R // 128)):
        b = slice(128 * rb, min(128 * rb + 128, R))
        _check_codes(cc[:, b], sct[rb, :K], X[b].T)


def test_dispatch_strided_input_and_write_bounds():
    """Through the ABI: padded rows of x, padded outputs inside guard bands."""
    T, k, E, K = 60, 3, 5, 200
    plan = _routed(2, T, k, E, 128)
    R = plan.src.numel()
    g = _gen(8)
    wide = _randn(g, T, 240, dtype=torch.bfloat16)
    guard, ldq, ldc, lds, ldsc = 4096, 224, R + 32, R + 5, K + 3
    def guarded(rows, ld, dtype, fill):
        flat = torch.full((rows * ld + 2 * guard,), fill, dtype=dtype, device="cuda")
        return flat, flat[guard:guard + rows * ld].view(rows, ld)
    qf, q = guarded(R, ldq, torch.uint8, 0xA5)
    cf, qc = guarded(K, ldc, torch.uint8, 0xA5)
    sf, s = guarded(2, lds, torch.float32, -7.0)
    tf, sc = guarded(R // 128, ldsc, torch.float32, -7.0)
    vp = lambda t: ctypes.c_void_p(t.data_ptr())
    for off in (0, 3):                               # 16-byte aligned rows, and not
        x = wide[:, off:off + K]
        st = B.lib().bfp8_moe_dispatch(vp(x), T, K, 240, vp(plan.src), R, k, None, vp(q), ldq, vp(s), lds, vp(qc), ldc,
                                       vp(sc), ldsc, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == B.BFP8_OK
        ql, sl, qcl, scl = B.moe_dispatch(x.contiguous(), plan)
        assert torch.equal(q[:, :K], ql[:, :K]) and torch.equal(qc[:, :R], qcl[:, :R])
        assert torch.equal(s[:, :R], sl) and torch.equal(sc[:, :K], scl[:, :K])
        for flat, body, cols, fill in ((qf, q, K, 0xA5), (cf, qc, R, 0xA5), (sf, s, R, -7.0), (tf, sc, K, -7.0)):
            assert bool((flat[:guard] == fill).all()) and bool((flat[-guard:] == fill).all())
            assert bool((body[:, cols:] == fill).all())


# ------------------------------------------------------------------ combine

# T, k, E, align, N
COMBINE = [(1, 1, 1, 1, 1), (1, 8, 64, 1, 4096), (48, 8, 256, 1, 2048), (130, 2, 8, 128, 384), (33, 11, 40, 16, 1001),
           (57, 32, 40, 1, 520), (9, 3, 4, 128, 7000)]


@pytest.mark.parametrize("T,k,E,align,N", COMBINE)
def test_combine_and_gradient(T, k, E, align, N):
    plan = _routed(T + N, T, k, E, align, empty=0.2 if T > 1 else 0.0)
    R = plan.src.numel()
    g = _gen(N)
    ye, dy = _randn(g, R, N, dtype=torch.bfloat16), _randn(g, T, N, dtype=torch.bfloat16)
    w = _randn(g, T, k)
    ye[plan.src < 0] = float("nan")                  # padding is never read
    row, src = plan.row.cpu().numpy(), plan.src.cpu().numpy()
    yn, wn, dn = np.nan_to_num(_f64(ye)), _f64(w), _f64(dy)
    for ww in (w, None):
        y = _f64(B.moe_combine(ye, plan, ww))
        want = ref.combine(yn, row, None if ww is None else wn)
        size = ref.combine(np.abs(yn), row, None if ww is None else np.abs(wn))
        # k fused products in fp32, one rounding to bf16 (8 significant bits: at most 2^-8 relative)
        assert np.all(np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2 * EPS * size + 1e-38)
    dye, dw = B.moe_combine_bwd(dy, ye, plan, w)
    none, dw2 = B.moe_combine_bwd(dy, ye, plan, w, with_dye=False)
    assert none is None and torch.equal(dw, dw2)
    dye_ref, dw_ref = ref.combine_grad(dn, yn, row, src, wn)
    assert np.all(np.abs(_f64(dye) - dye_ref) <= (2.0 ** -8 + EPS) * np.abs(dye_ref) + 1e-38)
    size = ref.combine_grad(np.abs(dn), np.abs(yn), row, src, wn)[1]
    # the longest chain of additions of a dot product: one thread's share, then the tree over the CTA
    chain = N / 32 + 8 + 16
    assert np.all(np.abs(_f64(dw) - dw_ref) <= chain * EPS * size + 1e-38)


# Rows of one to eight column classes and more, shared CTAs, one to several tokens a thread, k past eight
@pytest.mark.parametrize("N", [1, 8, 24, 256, 264, 500, 1024, 1026, 1536, 1544, 2304])
@pytest.mark.parametrize("T,k,E,align", [(1, 1, 3, 1), (33, 2, 5, 128), (70, 3, 8, 1), (19, 4, 6, 16), (40, 9, 12, 1)])
def test_combine_narrow_rows_and_batches(T, k, E, align, N):
    test_combine_and_gradient(T, k, E, align, N)


def test_combine_gradients_against_differences():
    """The combine is linear in ye and in w, so a whole unit step is its derivative."""
    T, k, E, N = 6, 2, 3, 16
    plan = _routed(4, T, k, E, 1, empty=0.0)
    rng = np.random.default_rng(0)
    R = plan.src.numel()
    ye = torch.from_numpy(rng.integers(-4, 5, (R, N))).to(torch.bfloat16).cuda()   # whole numbers: exact in bf16
    dy = torch.from_numpy(rng.integers(-4, 5, (T, N))).to(torch.bfloat16).cuda()
    w = torch.from_numpy(rng.integers(-2, 3, (T, k))).float().cuda()
    dye, dw = B.moe_combine_bwd(dy, ye, plan, w)
    loss = lambda a, b: float((B.moe_combine(a, plan, b).double() * dy.double()).sum())
    base = loss(ye, w)
    for t in range(T):
        for j in range(k):
            w1 = w.clone()
            w1[t, j] += 1
            assert loss(ye, w1) - base == float(dw[t, j])
    for r in range(R):
        y1 = ye.clone()
        y1[r, r % N] += 1
        assert loss(y1, w) - base == float(dye[r, r % N])


def test_combine_strided():
    plan = _routed(6, 40, 3, 8, 1)
    R = plan.src.numel()
    g = _gen(1)
    ye, dy, w = _randn(g, R, 300, dtype=torch.bfloat16)[:, 5:265], _randn(g, 40, 301, dtype=torch.bfloat16)[:, 1:261], \
        _randn(g, 40, 3)
    out = torch.zeros(40, 270, dtype=torch.bfloat16, device="cuda")
    B.moe_combine(ye, plan, w, y=out[:, 3:263])
    assert torch.equal(out[:, 3:263], B.moe_combine(ye.contiguous(), plan, w))
    assert not out[:, :3].any() and not out[:, 263:].any()
    a, b = B.moe_combine_bwd(dy, ye, plan, w), B.moe_combine_bwd(dy.contiguous(), ye.contiguous(), plan, w)
    assert torch.equal(a[0], b[0])
    size = (dy.float().abs() @ ye.float().abs().t()).max().item()
    assert float((a[1] - b[1]).abs().max()) <= 2 * (260 / 32 + 24) * EPS * size


# ------------------------------------------------------------------ routed product

def _codes(rng, shape):
    c = rng.integers(0, 256, size=shape, dtype=np.uint8)
    c[(c & 0x7F) == 0x7F] = 0x00  # no NaN codes
    return c


# T, k, E, align, N, K
PRODUCT = [(1, 1, 1, 1, 16, 128), (1, 8, 64, 1, 256, 512), (4, 2, 8, 1, 130, 208), (32, 4, 8, 1, 384, 1024),
           (100, 2, 3, 1, 200, 300), (60, 2, 4, 128, 136, 640), (7, 3, 5, 1, 1, 1), (20, 6, 300, 1, 64, 130),
           (17, 1, 1, 1, 2056, 96)]


@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("T,k,E,align,N,K", PRODUCT)
def test_routed_product(T, k, E, align, N, K, gathered):
    rng = np.random.default_rng(T + N + K)
    plan = _routed(T + K, T, k, E, align, empty=0.1 if T > 1 else 0.0)
    R = plan.src.numel()
    rows = T if gathered else R
    Kb, Nb, lda = -(-K // 128), -(-N // 128), -(-K // 16) * 16 + 16
    qa, qb = _codes(rng, (rows, lda)), _codes(rng, (E * N, lda))
    qa[:, K:] = 0x7F                                  # padding that would show: NaN codes
    qb[:, K:] = 0x7F
    sa = rng.uniform(0.01, 2.0, (Kb, rows + 3)).astype(np.float32)
    sb = rng.uniform(0.01, 2.0, (E * Nb, Kb + 1)).astype(np.float32)
    sa[:, rows:] = np.nan
    cu = lambda a: torch.from_numpy(a).cuda()
    guard, ldc, sent = 4096, N + 8, 0x7FC1
    flat = torch.full((R * ldc + 2 * guard,), sent, dtype=torch.int16, device="cuda")
    out = flat[guard:guard + R * ldc].view(torch.bfloat16).view(R, ldc)
    B.gemm_routed_1x128_128x128(cu(qa), cu(sa), cu(qb), cu(sb), plan, N, K, gathered=gathered, out=out)
    offs, src = plan.offs.cpu().numpy(), plan.src.cpu().numpy()
    end = offs[E]
    inside = np.arange(R) < end
    a_of = np.where(src >= 0, src // k, 0) if gathered else np.arange(R)
    qg, sg = qa[a_of].copy(), np.ascontiguousarray(sa[:, a_of])
    if gathered:
        qg[src < 0] = 0
    want = O.moe_gemm_fwd(np.ascontiguousarray(qg[:, :K]), sg, np.ascontiguousarray(qb[:, :K]),
                          np.ascontiguousarray(sb[:, :Kb]), offs, N, K)
    assert_gemm_close(_f64(out[:end, :N]), want[inside], f"routed product {T},{k},{E},{N},{K}")
    h = flat.cpu().numpy()
    body = h[guard:guard + R * ldc].reshape(R, ldc)
    assert np.all(h[:guard] == sent) and np.all(h[-guard:] == sent) and np.all(body[:, N:] == sent)
    assert np.all(body[end:] == sent)


# Batches whose tiles are few, split over 8, 4 and 2 CTAs with 16, 32 and 64 tokens a walk, and
# experts of several walks of 32 and 64 (the same check as above)
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("T,k,E,align,N,K", [
    (3, 1, 2, 1, 100, 1024), (4, 2, 8, 1, 500, 1100), (8, 2, 8, 1, 1000, 2000), (14, 1, 1, 1, 257, 1024),
    (30, 1, 2, 1, 300, 1100), (60, 1, 1, 1, 9728, 1024), (33, 1, 2, 1, 136, 2048), (300, 2, 4, 1, 2500, 272),
    (150, 3, 6, 16, 640, 400)])
def test_routed_product_splits_and_walks(T, k, E, align, N, K, gathered):
    test_routed_product(T, k, E, align, N, K, gathered)


def test_routed_product_refuses_wrong_types_and_outputs():
    plan = _routed(1, 4, 2, 3, 1, empty=0.0)
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    ok = dict(qa=e8(4, 256), sa=f(2, 4), qb=e8(3 * 8, 256), sb=f(3, 2), plan=plan, N=8, K=256)
    f8 = torch.float8_e4m3fn
    B.gemm_routed_1x128_128x128(**{**ok, "qa": ok["qa"].view(f8), "qb": ok["qb"].view(f8)}, out=bf(9, 24))
    for name, bad in (("codes", dict(qa=bf(4, 256))), ("codes", dict(qb=bf(24, 256))), ("scales", dict(sa=bf(2, 4))),
                      ("scales", dict(sb=f(3, 2).double())), ("CUDA", dict(sa=torch.zeros(2, 4))),
                      ("out", dict(out=f(8, 8))), ("out", dict(out=bf(7, 8))), ("out", dict(out=bf(8, 7))),
                      ("out", dict(out=bf(8, 8).t())), ("offs", dict(plan=plan._replace(offs=plan.offs.cpu()))),
                      ("offs", dict(plan=plan._replace(offs=plan.offs.long())))):
        with pytest.raises(ValueError, match=name):
            B.gemm_routed_1x128_128x128(**{**ok, **bad})
    ye, dy = bf(8, 16), bf(4, 16)
    with pytest.raises(ValueError, match="offs"):
        B.moe_combine_bwd(dy, ye, plan._replace(offs=plan.offs.cpu()), None)


def test_routed_product_of_no_reduction_is_zero():
    plan = _routed(1, 4, 2, 3, 1, empty=0.0)
    e8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")
    c = B.gemm_routed_1x128_128x128(e8(4, 16), f(1, 4), e8(3 * 8, 16), f(3, 1), plan, 8, 0)
    assert c.shape == (8, 8) and not c.any()


def test_operators_repeat_bit_for_bit():
    g = _gen(11)
    logits, x = _randn(g, 200, 64), _randn(g, 200, 512, dtype=torch.bfloat16)
    def once():
        idx, w = B.moe_route(logits, 4)
        plan = B.moe_plan(idx, 64)
        q = B.moe_dispatch(x, plan, weight=w)
        ye = torch.arange(plan.src.numel(), device="cuda").to(torch.bfloat16)[:, None].expand(-1, 512).contiguous()
        return [idx, w, *plan, q[0], q[1], q[2], q[3][:, :512], B.moe_combine(ye, plan, w),
                *B.moe_combine_bwd(x, ye, plan, w)]
    for a, b in zip(once(), once()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_combine_gradient_without_weights_is_the_dispatch():
    plan = _routed(3, 30, 2, 4, 128)
    g = _gen(4)
    ye, dy = _randn(g, plan.src.numel(), 96, dtype=torch.bfloat16), _randn(g, 30, 96, dtype=torch.bfloat16)
    dye, dw = B.moe_combine_bwd(dy, ye, plan, None)
    one = torch.ones(30, 2, device="cuda")
    dye1, dw1 = B.moe_combine_bwd(dy, ye, plan, one)
    assert torch.equal(dye, dye1) and torch.equal(dw, dw1)
    src = plan.src.long()
    want = torch.where((src >= 0)[:, None], dy[src.clamp_min(0) // 2], torch.zeros((), dtype=dy.dtype, device="cuda"))
    assert torch.equal(dye, want)


def test_routed_product_refuses_wrong_sizes():
    plan = _routed(1, 4, 2, 3, 1, empty=0.0)
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")
    ok = dict(qa=e8(4, 256), sa=f(2, 4), qb=e8(3 * 8, 256), sb=f(3, 2), plan=plan, N=8, K=256)
    B.gemm_routed_1x128_128x128(**ok)
    for bad in (dict(qa=e8(5, 256)), dict(qb=e8(23, 256)), dict(sb=f(2, 2)), dict(sa=f(1, 4)), dict(gathered=False)):
        with pytest.raises(ValueError):
            B.gemm_routed_1x128_128x128(**{**ok, **bad})
    for bad in (dict(K=272), dict(qa=e8(4, 264)), dict(sb=f(3, 1))):
        with pytest.raises((B.Bfp8Error, ValueError)):
            B.gemm_routed_1x128_128x128(**{**ok, **bad})


def test_routed_product_of_one_k_block_takes_any_stride_of_its_single_row_of_scales():
    plan = _routed(1, 4, 2, 3, 1, empty=0.0)
    g = _gen(2)
    qa, qb = (torch.randint(0, 120, (n, 128), generator=g, device="cuda", dtype=torch.uint8) for n in (4, 24))
    sa, sb = torch.rand(4, 1, generator=g, device="cuda"), torch.rand(3, 1, generator=g, device="cuda")
    one = sa.t()                                     # [1, 4], row stride 1
    assert one.stride(0) == 1
    got = B.gemm_routed_1x128_128x128(qa, one, qb, sb, plan, 8, 128)
    want = B.gemm_routed_1x128_128x128(qa, sa.reshape(1, 4).clone(), qb, sb, plan, 8, 128)
    assert torch.equal(got, want)
    with pytest.raises(ValueError, match="unit column"):
        B.gemm_routed_1x128_128x128(qa, torch.rand(4, 2, device="cuda").t(), qb, sb, plan, 8, 128)


# ------------------------------------------------------------------ offsets past 32 bits

def test_more_than_2_31_elements():
    """Sorted buffers and logits of more than 2^32 bytes and 2^31 elements: their last rows are right."""
    T, k, E, K = 70000, 8, 64, 4096                  # 560000 rows and more: 2.3e9 elements
    g = _gen(31)
    logits = _randn(g, T, E)
    idx, w = B.moe_route(logits, k, score="sigmoid")
    plan = B.moe_plan(idx, E)
    R = plan.src.numel()
    assert R * K > 1 << 31
    x = _randn(g, T, K, dtype=torch.bfloat16)
    q, s, qc, sc = B.moe_dispatch(x, plan)
    end = int(plan.offs[E])
    rows = torch.arange(end - 128, end, device="cuda")          # the last expert's last block
    src = plan.src[rows].long()
    xg = torch.where((src >= 0)[:, None], x[src.clamp_min(0) // k], torch.zeros((), dtype=x.dtype, device="cuda"))
    q2, s2, qc2, sc2 = B.quant_dual(xg)
    assert torch.equal(q[rows], q2) and torch.equal(s[:, rows], s2)
    assert torch.equal(qc[:, end - 128:end], qc2) and torch.equal(sc[end // 128 - 1], sc2[0])
    assert not q[end:].any() and not qc[:, end:].any()          # rows of no expert
    del q, s, qc, sc
    ye = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    ye.copy_(torch.arange(R, device="cuda")[:, None] % 251)
    y = B.moe_combine(ye, plan, w)
    dye, dw = B.moe_combine_bwd(x, ye, plan, w)
    t = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    at = plan.row[t].long()
    want = (ye[at].double() * w[t].double()[:, :, None]).sum(1)
    assert float((y[t].double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) + 1e-3
    dref = x[t].double()[:, None, :] * w[t].double()[:, :, None]
    assert float((dye[at].double() - dref).abs().max()) <= 2.0 ** -8 * float(dref.abs().max()) + 1e-6
    assert not dye[end:].any()
    dwref = (x[t].double()[:, None, :] * ye[at].double()).sum(2)
    size = (x[t].double()[:, None, :] * ye[at].double()).abs().sum(2)
    assert bool(((dw[t].double() - dwref).abs() <= (K / 32 + 24) * EPS * size).all())
    del ye, dye, y
    wide = torch.zeros(2200000, 1024, dtype=torch.bfloat16, device="cuda")
    wide[-1] = _randn(g, 1024, dtype=torch.bfloat16)
    i1, w1 = B.moe_route(wide, 4)
    i2, w2 = B.moe_route(wide[-1:], 4)
    assert torch.equal(i1[-1:], i2) and torch.equal(w1[-1:], w2) and bool((i1[0] == torch.arange(4, device="cuda")).all())
