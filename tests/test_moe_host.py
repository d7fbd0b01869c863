"""Host side of the mixture-of-experts operators (no GPU): argument checks
before anything is launched, the plan's row bound, and the 64-bit reference
forms that the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_gb300 as B
import moe_reference as ref
from blockwise_scaled_fp8_gb300 import buildlib as bbuild

NULL = ctypes.c_void_p(None)
P = ctypes.c_void_p(0x10000)      # fake, aligned; never dereferenced
ODD = ctypes.c_void_p(0x10001)
BAD = 1                           # BFP8_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def _built():
    bbuild.build()


def _caller(fn, ok):
    names = list(ok)

    def call(**kw):
        assert not set(kw) - set(names)
        return getattr(B.lib(), fn)(*(kw.get(n, ok[n]) for n in names))
    return call


def test_route_argument_validation():
    call = _caller("bfp8_moe_route", dict(l=P, f32=0, T=4, E=64, ldl=64, bias=NULL, k=6, score=0, groups=8, top=4, gt=2,
                                          renorm=1, scale=1.0, idx=P, w=P, st=NULL))
    for bad in (dict(T=-1), dict(E=0), dict(E=1025, ldl=1025), dict(k=0), dict(k=33), dict(k=65, groups=1, top=1),
                dict(score=2), dict(groups=7), dict(groups=0), dict(groups=64, top=33), dict(top=9), dict(top=0),
                dict(gt=3), dict(gt=0), dict(ldl=63), dict(l=NULL), dict(idx=NULL), dict(w=NULL), dict(l=ODD),
                dict(f32=1, l=ctypes.c_void_p(0x10002)), dict(bias=ODD), dict(top=1, k=9), dict(T=1 << 31)):
        assert call(**bad) == BAD, bad
    assert call(T=0, l=NULL, idx=NULL, w=NULL) == B.BFP8_OK


def test_route_bwd_argument_validation():
    call = _caller("bfp8_moe_route_bwd", dict(l=P, f32=1, T=4, E=64, ldl=64, idx=P, w=P, dw=P, k=6, score=1, renorm=1,
                                              scale=1.0, dl=P, ldd=64, st=NULL))
    for bad in (dict(E=0), dict(k=0), dict(score=-1), dict(ldl=63), dict(ldd=63), dict(dw=NULL), dict(dl=NULL),
                dict(dl=ODD)):
        assert call(**bad) == BAD, bad
    assert call(T=0) == B.BFP8_OK


def test_plan_argument_validation():
    call = _caller("bfp8_moe_plan", dict(idx=P, T=4, k=2, E=8, al=128, offs=P, row=P, src=P, R=1024, counts=P, st=NULL))
    for bad in (dict(T=-1), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(al=0), dict(al=4097), dict(R=1023),
                dict(R=1 << 31), dict(idx=NULL), dict(offs=NULL), dict(row=NULL), dict(src=NULL), dict(counts=NULL),
                dict(src=ODD), dict(T=1 << 30, k=2)):
        assert call(**bad) == BAD, bad


def test_plan_rows_hold_every_choice():
    rng = np.random.default_rng(0)
    for _ in range(300):
        T, k, E = int(rng.integers(0, 40)), int(rng.integers(1, 9)), int(rng.integers(1, 20))
        align = int(rng.choice([1, 2, 16, 128]))
        R = B.moe_plan_rows(T, k, E, align)
        idx = rng.integers(-1, E, size=(T, k)).astype(np.int32)
        offs, row, src, counts = ref.plan(idx, E, align, R)
        assert offs[-1] <= R and R % align == 0
        assert R == B.lib().bfp8_moe_plan_rows(T, k, E, align)
        assert np.array_equal(np.sort(src[src >= 0]), np.flatnonzero(idx.reshape(-1) >= 0))
    # the bound is reached: each slot its own expert
    assert B.moe_plan_rows(3, 1, 8, 128) == 3 * 128
    assert B.moe_plan_rows(0, 4, 8, 128) == 0
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1 << 31, 1, 1, 1), (1 << 28, 8, 1, 1)):
        with pytest.raises(ValueError, match="out of range"):
            B.moe_plan_rows(*bad)
        assert B.lib().bfp8_moe_plan_rows(*bad) == -1


def test_dispatch_argument_validation():
    call = _caller("bfp8_moe_dispatch", dict(x=P, T=4, K=256, ldx=256, src=P, R=256, k=2, wt=NULL, q=P, ldq=256, s=P,
                                             lds=256, qc=P, ldqc=256, sc=P, ldsc=256, st=NULL))
    for bad in (dict(T=-1), dict(R=-1), dict(K=-1), dict(k=0), dict(x=NULL), dict(src=NULL), dict(q=NULL), dict(s=NULL),
                dict(qc=NULL), dict(sc=NULL), dict(ldx=255), dict(ldq=255), dict(ldq=264), dict(lds=255),
                dict(ldqc=240), dict(ldqc=260), dict(ldsc=255), dict(q=ODD), dict(qc=ODD), dict(x=ODD), dict(wt=ODD)):
        assert call(**bad) == BAD, bad
    assert call(R=0) == B.BFP8_OK
    assert call(K=0) == B.BFP8_OK


def test_combine_argument_validation():
    call = _caller("bfp8_moe_combine", dict(ye=P, ldye=64, R=8, row=P, w=NULL, T=4, k=2, N=64, y=P, ldy=64, st=NULL))
    for bad in (dict(T=-1), dict(N=-1), dict(k=0), dict(ye=NULL), dict(row=NULL), dict(y=NULL), dict(ldye=63),
                dict(ldy=63), dict(ye=ODD), dict(w=ODD), dict(T=1 << 29, N=4096, ldye=4096, ldy=4096)):
        assert call(**bad) == BAD, bad
    assert call(T=0) == B.BFP8_OK
    assert call(N=0) == B.BFP8_OK
    call = _caller("bfp8_moe_combine_bwd", dict(dy=P, lddy=64, ye=P, ldye=64, R=8, offs=P, E=8, row=P, src=P, w=P, T=4, k=2, N=64,
                                                dye=P, lddye=64, dw=P, st=NULL))
    for bad in (dict(T=-1), dict(k=40), dict(dy=NULL), dict(ye=NULL), dict(row=NULL), dict(src=NULL), dict(dw=NULL),
                dict(offs=NULL), dict(E=0), dict(E=1025), dict(lddy=63), dict(lddye=63), dict(ldye=1), dict(dye=ODD), dict(dw=ODD)):
        assert call(**bad) == BAD, bad
    assert call(T=0, dye=NULL) == B.BFP8_OK


def test_routed_product_argument_validation():
    call = _caller("bfp8_gemm_routed_1x128_128x128",
                   dict(qa=P, lda=256, sa=P, ldsa=4, T=4, qb=P, ldb=256, sb=P, ldsb=2, offs=P, E=8, src=P, k=2, c=P, ldc=64,
                        R=8, N=64, K=256, st=NULL))
    for bad in (dict(E=0), dict(E=1025), dict(k=0), dict(T=-1), dict(R=-1), dict(lda=240), dict(lda=260), dict(ldb=264),
                dict(ldsa=3), dict(ldsb=1), dict(ldc=63), dict(qa=NULL), dict(sa=NULL), dict(qb=NULL), dict(sb=NULL),
                dict(offs=NULL), dict(c=NULL), dict(qa=ODD), dict(qb=ODD), dict(src=ODD), dict(T=0),
                dict(E=1024, N=1 << 22, ldc=1 << 22)):
        assert call(**bad) == BAD, bad
    assert call(R=0) == B.BFP8_OK
    assert call(N=0) == B.BFP8_OK


def test_binding_checks_tensors_before_any_device_call():
    f = torch.zeros(4, 8)
    plan = B.MoePlan(*(torch.zeros(s, dtype=torch.int32) for s in (9, (4, 2), 8, 8)))
    with pytest.raises(ValueError, match="logits"):
        B.moe_route(f, 2)                                      # not on a GPU
    with pytest.raises(ValueError, match="T, k"):
        B.moe_plan(torch.zeros(4, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="idx"):
        B.moe_plan(torch.zeros(4, 2, dtype=torch.int64), 8)
    with pytest.raises(ValueError, match="x must"):
        B.moe_dispatch(f, plan)
    with pytest.raises(ValueError, match="ye must"):
        B.moe_combine(f, plan)
    with pytest.raises(ValueError, match="dy must"):
        B.moe_combine_bwd(f, f, plan, f)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    l, dw, h = rng.normal(size=(4, 10)), rng.normal(size=(4, 3)), 1e-5
    p, ok = ref.scores(l, score, -3e38)
    idx, _ = ref.choose(p, ok, l, score, None, 3, 1, 1, 1)
    grad = ref.route_grad(p, idx, dw, score, renorm, 2.0)
    loss = lambda m: (dw * ref.weights(ref.scores(m, score, -3e38)[0], idx, renorm, 2.0)).sum(1)
    for e in range(10):
        step = h * np.eye(10)[e]
        # h^2 / 6 times a third derivative below 20, 64-bit cancellation 1e-15 / h
        assert np.allclose(grad[:, e], (loss(l + step) - loss(l - step)) / (2 * h), rtol=0, atol=1e-9 + 1e-10)
