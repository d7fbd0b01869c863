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
