"""Host side of the norm, the gradients' norm and clipping and the few-token
experts layer (no GPU): argument checks before anything is launched, and the
binding's refusals."""
import ctypes
import os
import subprocess

import pytest
import torch

import blockwise_scaled_fp8_gb300 as B
from blockwise_scaled_fp8_gb300 import buildlib as bbuild

NULL = ctypes.c_void_p(None)
P = ctypes.c_void_p(0x10000)      # fake, aligned; never dereferenced
Y = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10001)
BAD = 1                           # BFP8_ERR_INVALID_ARG
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _built():
    bbuild.build()


def _caller(fn, ok):
    names = list(ok)

    def call(**kw):
        assert not set(kw) - set(names)
        return getattr(B.lib(), fn)(*(kw.get(n, ok[n]) for n in names))
    return call


def test_rms_norm_argument_validation():
    call = _caller("bfp8_rms_norm_quant", dict(x=P, T=4, K=256, ldx=256, r=P, ldr=256, w=P, f32=0, eps=1e-6, h=P, ldh=256,
                                               rstd=P, q=P, ldq=256, s=P, lds=4, qc=P, ldqc=16, sc=P, ldsc=256, y=Y, ldy=256,
                                               st=NULL))
    for bad in (dict(T=-1), dict(K=-1), dict(K=16385, ldx=16385), dict(T=1 << 31), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("inf")), dict(eps=float("nan")), dict(r=NULL), dict(h=NULL), dict(s=NULL), dict(q=NULL),
                dict(sc=NULL), dict(qc=NULL), dict(x=NULL), dict(w=NULL), dict(rstd=NULL), dict(ldx=255), dict(ldr=255),
                dict(ldh=255), dict(ldy=255), dict(ldq=255), dict(ldq=264), dict(lds=3), dict(ldqc=3), dict(ldqc=24),
                dict(ldsc=255), dict(x=ODD), dict(q=ctypes.c_void_p(0x10008)), dict(qc=ctypes.c_void_p(0x10008)),
                dict(s=ODD), dict(w=ODD), dict(f32=1, w=ctypes.c_void_p(0x10002)), dict(y=ODD), dict(h=ODD)):
        assert call(**bad) == BAD, bad
    assert call(T=0, x=NULL) == B.BFP8_OK
    assert call(K=0) == B.BFP8_OK


def test_rows_that_share_memory_are_refused():
    """An output may be an input's rows themselves and otherwise none of its elements."""
    at = lambda element: ctypes.c_void_p(0x100000 + 2 * element)  # noqa: E731
    call = _caller("bfp8_rms_norm_quant", dict(x=at(0), T=4, K=256, ldx=512, r=P, ldr=256, w=P, f32=0, eps=1e-6, h=at(0),
                                               ldh=512, rstd=P, q=NULL, ldq=0, s=NULL, lds=0, qc=NULL, ldqc=0, sc=NULL, ldsc=0,
                                               y=NULL, ldy=256, st=NULL))
    for bad in (dict(ldh=520), dict(h=at(512)), dict(h=at(8)), dict(h=at(255)), dict(h=at(264)), dict(h=at(3 * 512 + 255)),
                dict(x=at(512)), dict(x=at(1791)), dict(h=at(256), ldh=256), dict(T=1, h=at(255)), dict(y=at(0), ldy=512),
                dict(y=at(1)), dict(y=P), dict(r=at(512), ldr=512), dict(h=P, ldh=264)):
        assert call(**bad) == BAD, bad
        assert b"share memory" in B.lib().bfp8_last_error(), bad
    call = _caller("bfp8_rms_norm_bwd", dict(dy=at(0), T=4, K=256, lddy=512, h=P, ldh=256, w=P, f32=1, rstd=P, dh=NULL, lddh=0,
                                             dx=at(0), lddx=512, dw=Y, ws=P, n=1 << 30, st=NULL))
    for bad in (dict(lddx=520), dict(dx=at(512)), dict(dx=at(1)), dict(dx=P, lddx=264), dict(dh=at(255), lddh=512, dy=Y)):
        assert call(**bad) == BAD, bad
        assert b"share memory" in B.lib().bfp8_last_error(), bad


def test_rms_norm_bwd_argument_validation():
    call = _caller("bfp8_rms_norm_bwd", dict(dy=P, T=4, K=256, lddy=256, h=P, ldh=256, w=P, f32=1, rstd=P, dh=P, lddh=256,
                                             dx=P, lddx=256, dw=P, ws=P, n=1 << 30, st=NULL))
    for bad in (dict(T=-1), dict(K=16385), dict(dy=NULL), dict(h=NULL), dict(w=NULL), dict(rstd=NULL), dict(dx=NULL),
                dict(dw=NULL), dict(ws=NULL), dict(lddy=255), dict(ldh=255), dict(lddh=255), dict(lddx=255), dict(dy=ODD),
                dict(dw=ODD), dict(ws=ctypes.c_void_p(0x10008)), dict(w=ctypes.c_void_p(0x10002))):
        assert call(**bad) == BAD, bad
    assert call(K=0) == B.BFP8_OK
    size = B.lib().bfp8_rms_norm_bwd_workspace_size
    assert size(0, 256) == 0 and size(-1, 256) == 0 and size(4, 16385) == 0
    assert size(1, 1) >= 4 and size(100000, 4096) >= 4096 * 4


def test_grad_argument_validation():
    def lists(ptrs, numel, types):
        n = len(ptrs)
        return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*types), n

    L = B.lib()
    A = 0x100000

    def norm(ptrs=(A, 2 * A), numel=(10, 20), types=(0, 1), out=P, ws=P, n=1 << 20):
        p, k, t, c = lists(ptrs, numel, types)
        return L.bfp8_grad_norm(p, k, t, c, out, ws, n, NULL)

    for bad in (dict(ptrs=(None, A)), dict(numel=(-1, 5)), dict(numel=(1 << 40, 5)), dict(types=(3, 0)), dict(types=(-1, 0)),
                dict(ptrs=(A + 2, 2 * A)), dict(ptrs=(A, 2 * A + 1)), dict(out=NULL), dict(ws=NULL), dict(out=ODD),
                dict(ws=ctypes.c_void_p(0x10008))):
        assert norm(**bad) == BAD, bad
    assert L.bfp8_grad_norm(NULL, NULL, NULL, 2, P, P, 1 << 20, NULL) == BAD
    assert L.bfp8_grad_norm(NULL, NULL, NULL, -1, P, P, 1 << 20, NULL) == BAD

    def clip(ptrs, numel, types, out, otypes, max_norm=1.0):
        p, k, t, c = lists(ptrs, numel, types)
        o, _, ot, _ = lists(out, numel, otypes)
        return L.bfp8_clip_grads(p, k, t, c, max_norm, o, ot, P, P, 0, NULL)  # (a workspace too small: nothing is launched)

    def overlap():
        return "shares memory" in L.bfp8_last_error().decode()

    # memory that two of the tensors share: refused, before the workspace is looked at
    for args in (((A, A), (8, 8), (0, 0), (A, A), (0, 0)),                                    # a tensor twice, in place
                 ((A, A + 16), (8, 8), (0, 0), (A, A + 16), (0, 0)),                          # overlapping views
                 ((A, 2 * A), (8, 8), (0, 0), (3 * A, 3 * A + 4), (0, 0)),                    # overlapping outputs
                 ((A, 2 * A), (8, 8), (0, 0), (2 * A, 3 * A), (0, 0)),                        # an output on another input
                 ((A, 2 * A), (8, 8), (1, 0), (A, 2 * A), (0, 0))):                           # in place, wider than it was
        assert clip(*args) == BAD and overlap(), args
    for args in (((A, A), (8, 8), (0, 0), (3 * A, 4 * A), (0, 0)),                            # read twice, written apart
                 ((A, A + 32), (8, 8), (0, 0), (A, A + 32), (0, 0)),                          # neighbours
                 ((A, None), (8, 0), (0, 0), (A, None), (0, 0))):                             # an empty one
        st = clip(*args)
        assert st != B.BFP8_OK and not overlap(), args
    for max_norm in (-1.0, float("nan")):
        assert clip((A,), (8,), (0,), (A,), (0,), max_norm) == BAD and not overlap()
    assert L.bfp8_grad_workspace_size(-1) == 0 and L.bfp8_grad_workspace_size(641) == 2 * L.bfp8_grad_workspace_size(1)


def test_mlp_decode_argument_validation():
    call = _caller("bfp8_moe_mlp_decode",
                   dict(x=P, T=4, K=256, ldx=256, l=P, f32=1, E=8, ldl=8, bias=NULL, k=2, score=0, groups=1, top=1, gt=1,
                        renorm=1, scale=1.0, qgu=P, ldgu=256, sgu=P, ldsgu=2, qd=P, ldd=128, sd=P, ldsd=1, I=128, N=256, y=P,
                        ldy=256, ws=P, n=1 << 20, st=NULL))
    for bad in (dict(T=17), dict(T=-1), dict(K=0), dict(I=0), dict(N=0), dict(I=96), dict(N=200, ldy=256), dict(E=0),
                dict(E=1025, ldl=1025), dict(k=0), dict(k=9), dict(k=33), dict(score=2), dict(groups=3), dict(top=2),
                dict(gt=3), dict(ldl=7), dict(ldx=255), dict(ldy=255), dict(ldgu=240), dict(ldgu=264), dict(ldd=112),
                dict(ldd=136), dict(ldsgu=1), dict(ldsd=0), dict(x=NULL), dict(l=NULL), dict(qgu=NULL), dict(sgu=NULL),
                dict(qd=NULL), dict(sd=NULL), dict(y=NULL), dict(ws=NULL), dict(n=100), dict(x=ODD), dict(y=ODD),
                dict(l=ctypes.c_void_p(0x10002)), dict(bias=ODD), dict(qgu=ctypes.c_void_p(0x10008)),
                dict(qd=ctypes.c_void_p(0x10008)), dict(sd=ODD), dict(ws=ctypes.c_void_p(0x10008)),
                dict(E=1024, ldl=1024, I=1 << 20, ldd=1 << 20, ldsd=1 << 13)):
        assert call(**bad) == BAD, bad
    assert call(T=0, x=NULL, l=NULL) == B.BFP8_OK
    size = B.lib().bfp8_moe_mlp_workspace_size
    assert size(17, 2, 128) == 0 and size(4, 33, 128) == 0 and size(4, 2, 128) >= 4 * 2 * 128 * 4


def test_binding_refuses_what_the_kernels_do_not_take(monkeypatch):
    """Tensors of another type, shape or place are refused by name (on the host: no tensor here is on a GPU)."""
    monkeypatch.setattr(B, "_here", lambda: 0)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256)
    with pytest.raises(ValueError, match="x must be"):
        B.rms_norm_quant(x, w)
    with pytest.raises(ValueError, match="2-D"):
        B.rms_norm_quant(x[0], w)
    with pytest.raises(ValueError, match="dy must be"):
        B.rms_norm_bwd(x, x, w, torch.ones(4))
    with pytest.raises(ValueError, match=r"tensors\[0\]"):
        B.grad_norm([x])
    with pytest.raises(ValueError, match=r"tensors\[0\]"):
        B.clip_grads([x], 1.0)
    with pytest.raises(ValueError, match="logits"):
        B.moe_mlp_decode(x, torch.zeros(4, 8), 2, x, w, x, w, I=64, N=128)
    from blockwise_scaled_fp8_gb300 import module
    with pytest.raises(TypeError, match="bfloat16"):
        module.blockwise_fp8_norm_linear(x.float(), x, w)
    with pytest.raises(ValueError, match="norm_weight"):
        module.blockwise_fp8_norm_linear(x, torch.zeros(8, 256, dtype=torch.bfloat16), torch.ones(8))


def test_dense_tensors():
    t = torch.zeros(3, 4, 5)
    assert B._dense(t) and B._dense(t.permute(2, 0, 1)) and B._dense(t.transpose(0, 1))
    assert not B._dense(t[:, :, ::2]) and not B._dense(t[:, 0].expand(3, 5)[:, :3]) and not B._dense(torch.zeros(1).expand(7))


@pytest.mark.parametrize("stride", [61])
def test_product_scale_quotients(tmp_path, stride):
    """The few-token layer forms s as max(amax, 1e-12) * fl(1/448) and its codes by the quantisers' one-step quotient: the
    codes of RN(x / s) for that s too (near_scale_check.c; stride 1 goes through all 1.07e9 pairs)."""
    root = os.path.dirname(HERE)
    exe = str(tmp_path / "near_scale_check")
    subprocess.run(["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-fno-fast-math", "-fopenmp",
                    os.path.join(HERE, "near_scale_check.c"), os.path.join(root, "oracle", "bfp8_oracle.c"), "-lm", "-o", exe],
                   check=True, capture_output=True, text=True)
    out = subprocess.run([exe, str(stride)], check=True, capture_output=True, text=True).stdout
    fields = dict(kv.split("=") for kv in out.split())
    assert int(fields["tot"]) > 5_000_000 and int(fields["bad"]) == 0
