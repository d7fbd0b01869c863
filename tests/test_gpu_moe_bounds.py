"""The routed experts' kernels write their outputs and nothing beside them, and
what lies behind their inputs does not show: outputs inside sentinels, before,
after and between the rows, inputs as parts of larger buffers."""
import pytest

import moe_reference as ref
from gpu_util import torch

import blockwise_scaled_fp8_gb300 as B

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    yield
    B.check_device_errors()


class Guarded:
    """A [rows, cols] output with row stride ld inside a buffer of sentinels, 300 rows before and after it."""
    PAD = 300

    def __init__(self, rows, cols, ld, dtype):
        self.words = torch.int16 if dtype == torch.bfloat16 else torch.int32
        self.fill = 0x7FC1 if dtype == torch.bfloat16 else 0x7FC0DEAD
        self.flat = torch.full(((rows + 2 * self.PAD) * ld,), self.fill, dtype=self.words, device="cuda")
        self.rows, self.cols, self.ld = rows, cols, ld
        self.out = self._body().view(dtype)[:, :cols]

    def _body(self):
        return self.flat[self.PAD * self.ld:(self.PAD + self.rows) * self.ld].view(self.rows, self.ld)

    def check(self):
        assert bool((self.flat[:self.PAD * self.ld] == self.fill).all()), "written before the output"
        assert bool((self.flat[(self.PAD + self.rows) * self.ld:] == self.fill).all()), "written after the output"
        assert bool((self._body()[:, self.cols:] == self.fill).all()), "written between the rows"


def _behind(t, tail):
    """A copy of t at the start of a larger buffer that goes on with `tail`."""
    return torch.cat([t.reshape(-1), tail.reshape(-1).to(t.dtype)])[:t.numel()].view(t.shape)


def _plan(g, T, k, E, align, empty=0.1):
    idx = torch.argsort(torch.rand(T, max(E, k), generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32)
    idx[(idx >= E) | (torch.rand(T, 1, generator=g, device="cuda") < empty)] = -1
    return B.moe_plan(idx.contiguous(), E, align=align)


# Widths of each access (8, 4, 2 and 1 columns) whose rows share a CTA or do not; token counts beside a full last CTA
@pytest.mark.parametrize("N", [1, 24, 64, 101, 128, 129, 256, 258, 260, 512, 516, 1000, 1024, 1032])
@pytest.mark.parametrize("k", [2, 3, 5, 8, 9, 32])
def test_combine_stays_inside_its_output(N, k):
    vec = next(v for v in (8, 4, 2, 1) if N % v == 0)
    sides = max(256 // -(-N // vec), 1)
    for T in sorted({1, 5, 97, max(sides - 1, 1), sides + 1}):
        g = torch.Generator(device="cuda").manual_seed(1000 * N + 10 * k + T)
        plan = _plan(g, T, k, 40, 1)
        R = plan.src.numel()
        ye = torch.randn(R, N, generator=g, device="cuda").bfloat16()
        w = torch.randn(T, k, generator=g, device="cuda")
        # behind row and w: indices of real rows, and weights
        more = torch.arange(300 * k, device="cuda") % R
        plan = plan._replace(row=_behind(plan.row, more))
        y = Guarded(T, N, N + 8, torch.bfloat16)
        B.moe_combine(ye, plan, _behind(w, torch.ones(300 * k, device="cuda")), y=y.out)
        y.check()
        f = lambda t: t.double().cpu().numpy()
        row = plan.row.cpu().numpy()
        want, size = ref.combine(f(ye), row, f(w)), ref.combine(abs(f(ye)), row, abs(f(w)))
        # k fused products in fp32, one rounding to bf16
        assert (abs(f(y.out) - want) <= 2.0 ** -8 * abs(want) + (k + 1) * 2 * EPS * size + 1e-38).all()


def _call(fn, *args):
    """An entry of the ABI: tensors by their addresses, the current stream."""
    a = [x.data_ptr() if isinstance(x, torch.Tensor) else x for x in args]
    assert getattr(B.lib(), fn)(*a, torch.cuda.current_stream().cuda_stream) == B.BFP8_OK


@pytest.mark.parametrize("with_dye", [True, False])
@pytest.mark.parametrize("N", [1, 24, 101, 128, 258, 260, 1000, 1536, 1544, 4104])
@pytest.mark.parametrize("k", [1, 2, 3, 6, 9, 32])
def test_combine_gradient_stays_inside_its_outputs(N, k, with_dye):
    for T in (1, 37, 70):
        g = torch.Generator(device="cuda").manual_seed(1000 * N + 10 * k + T)
        plan = _plan(g, T, k, 40, 16)
        R = plan.src.numel()
        ye, dy = (torch.randn(n, N, generator=g, device="cuda").bfloat16() for n in (R, T))
        w = torch.randn(T, k, generator=g, device="cuda")
        more = torch.arange(300 * k, device="cuda") % R
        row, src = _behind(plan.row, more), _behind(plan.src, more % (T * k))
        dye, dw = Guarded(R, N, N + 8, torch.bfloat16), Guarded(T, k, k, torch.float32)
        _call("bfp8_moe_combine_bwd", dy, N, ye, N, R, plan.offs, 40, row, src, _behind(w, torch.ones(300 * k, device="cuda")),
              T, k, N, dye.out if with_dye else None, N + 8, dw.out)
        dye.check()
        dw.check()
        want_dye, want_dw = B.moe_combine_bwd(dy, ye, plan, w, with_dye=with_dye)
        assert torch.equal(dw.out, want_dw) and (not with_dye or torch.equal(dye.out, want_dye))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (37, 32), (64, 6), (160, 8), (256, 8), (500, 3), (1024, 32)])
def test_router_stays_inside_its_outputs(E, k, score, dtype):
    f32 = int(dtype == torch.float32)
    for T in (1, 5, 34):
        g = torch.Generator(device="cuda").manual_seed(E + T)
        logits = torch.randn(T, E, generator=g, device="cuda").to(dtype)
        wide = torch.full((T + 8, E + 3), 100.0, dtype=dtype, device="cuda")  # what is beside would be chosen
        wide[:T, :E] = logits
        idx, w = Guarded(T, k, k, torch.int32), Guarded(T, k, k, torch.float32)
        _call("bfp8_moe_route", wide, f32, T, E, E + 3, None, k, score, 1, 1, 1, 1, 1.0, idx.out, w.out)
        idx.check()
        w.check()
        i1, w1 = B.moe_route(logits, k, score="sigmoid" if score else "softmax")
        assert torch.equal(idx.out, i1) and torch.equal(w.out, w1)
        dw, dl = torch.randn(T, k, generator=g, device="cuda"), Guarded(T, E, E + 3, dtype)
        _call("bfp8_moe_route_bwd", wide, f32, T, E, E + 3, i1, w1, dw, k, score, 1, 1.0, dl.out, E + 3)
        dl.check()
        assert torch.equal(dl.out, B.moe_route_bwd(logits, i1, w1, dw, score="sigmoid" if score else "softmax"))


@pytest.mark.parametrize("T,k,E,align", [(1, 1, 1, 1), (1, 8, 64, 1), (33, 3, 7, 128), (150, 7, 160, 16), (4100, 2, 8, 16),
                                         (5000, 8, 1024, 128)])
def test_plan_stays_inside_its_outputs(T, k, E, align):
    g = torch.Generator(device="cuda").manual_seed(T)
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    R = B.moe_plan_rows(T, k, E, align)
    offs, row, src, counts = (Guarded(n, 1, 1, torch.int32) for n in (E + 1, T * k, R, E))
    _call("bfp8_moe_plan", _behind(idx, torch.zeros(4096, device="cuda")), T, k, E, align, offs.out, row.out, src.out, R,
          counts.out)
    want = B.moe_plan(idx, E, align=align)
    for got, part in ((offs, want.offs), (row, want.row), (src, want.src), (counts, want.counts)):
        got.check()
        assert torch.equal(got.out.reshape(-1), part.reshape(-1))
