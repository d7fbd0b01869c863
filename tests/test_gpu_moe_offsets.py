"""Offsets that are no plan's: the routed product refuses decreasing ones on
the device, writes nothing and says so."""
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


# R, N, K and offsets: tiles split over a cluster and not, walks of 16, 32 and 64 rows, the fall at the first, a middle
# and the last expert
@pytest.mark.parametrize("R,N,K,offs", [
    (8, 64, 128, [3, 0, 8, 8]), (16, 256, 1024, [0, 16, 4, 16]), (40, 256, 1024, [0, 10, 40, 39]), (400, 512, 256, [0, 300, 100, 400]),
    (300, 136, 640, [0, 0, 300, -1]), (30, 64, 256, [0] * 600 + [30, 0, 30] + [30] * 400)])
def test_routed_product_refuses_decreasing_offsets(R, N, K, offs):
    g = torch.Generator(device="cuda").manual_seed(R)
    E, k = len(offs) - 1, 1
    code = lambda *s: torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8)
    qa, qb = code(R, K), code(E * N, K)
    sa, sb = (torch.rand(*s, generator=g, device="cuda") for s in ((-(-K // 128), R), (E * -(-N // 128), -(-K // 128))))
    slots = torch.arange(R, dtype=torch.int32, device="cuda")
    plan = B.MoePlan(torch.tensor(offs, dtype=torch.int32, device="cuda"), slots.view(R, k), slots, slots[:0])
    flat = torch.full((3 * R * N,), 0x7FC1, dtype=torch.int16, device="cuda")
    out = flat[R * N:2 * R * N].view(torch.bfloat16).view(R, N)
    B.gemm_routed_1x128_128x128(qa, sa, qb, sb, plan, N, K, out=out)
    with pytest.raises(B.Bfp8Error, match="offsets decreasing"):
        B.check_device_errors()
    assert bool((flat == 0x7FC1).all())
    # offsets past both ends are clamped, as before, and the next call is served
    ok = torch.tensor([-5] + [R + 7] * E, dtype=torch.int32, device="cuda")
    B.gemm_routed_1x128_128x128(qa, sa, qb, sb, plan._replace(offs=ok), N, K, out=out)
    B.check_device_errors()
    whole = torch.tensor([0] + [R] * E, dtype=torch.int32, device="cuda")
    want = B.gemm_routed_1x128_128x128(qa, sa, qb, sb, plan._replace(offs=whole), N, K)
    assert torch.equal(out, want)
    assert bool((flat[:R * N] == 0x7FC1).all()) and bool((flat[2 * R * N:] == 0x7FC1).all())


def test_routed_product_refuses_operands_narrower_than_the_product():
    """Views whose rows lie far enough apart but do not hold the columns: they would be read beyond their width."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    plan = B.MoePlan(torch.tensor([0, 4, 8, 8], dtype=torch.int32, device="cuda"), i(4, 2), i(8), i(3))
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")
    ok = dict(qa=e8(4, 256), sa=f(2, 4), qb=e8(3 * 8, 256), sb=f(3, 2), plan=plan, N=8, K=256)
    B.gemm_routed_1x128_128x128(**ok)
    for bad in (dict(qa=e8(4, 256)[:, :240]), dict(qb=e8(24, 256)[:, :128]), dict(sa=f(2, 8)[:, :3]), dict(sb=f(3, 4)[:, :1])):
        with pytest.raises(ValueError, match="columns"):
            B.gemm_routed_1x128_128x128(**{**ok, **bad})
