"""The norm of many tensors and their clipping, against 64-bit sums."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

f32, bf16, f16, f64 = torch.float32, torch.bfloat16, torch.float16, torch.float64
HALF = {f32: 2.0 ** -24, bf16: 2.0 ** -8, f16: 2.0 ** -11}  # a rounding, of the value
TINY = {f32: 2.0 ** -150, bf16: 2.0 ** -134, f16: 2.0 ** -25}  # .. of the smallest values


def ref_norm(ts):
    return float(torch.stack([t.to(f64).square().sum() for t in ts]).sum().sqrt()) if ts else 0.0


def some(sizes, seed, dtypes=(f32, bf16, f16), offs=(0, 1, 2, 3, 4, 8)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        off = offs[i % len(offs)]
        buf = torch.randn(n + off, generator=g, device="cuda").to(dtypes[i % len(dtypes)])
        out.append(buf[off:])
    return out


# fp32 sums of at most 256 squares, then fp64: the sum within (32 + 5 + 1) roundings, half of them in the root, and its own
NORM_TOL = (38 / 2 + 2) * 2.0 ** -24

SIZES = [[1], [7], [8], [0, 3, 0], [4096], [4097, 1, 16384, 16385, 5], [100003], [5_000_000, 3, 70_001], [1] * 700, [513] * 65,
         [12345] * 64]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm(sizes):
    ts = some(sizes, len(sizes) + max(sizes))
    got = B.grad_norm(ts)
    ref = ref_norm(ts)
    assert got.dtype == f32 and got.dim() == 0
    assert abs(float(got) - ref) <= NORM_TOL * ref
    assert torch.equal(got, B.grad_norm(ts))


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("out", [None, f32, bf16, f16])
def test_clip(sizes, out):
    ts = some(sizes, 3 + len(sizes))
    ref = ref_norm(ts)
    before = [t.clone() for t in ts]
    outs = None if out is None else [torch.empty_like(t, dtype=out) for t in ts]
    max_norm = 0.4 * ref
    norm = B.clip_grads(ts, max_norm, out=outs)
    assert abs(float(norm) - ref) <= NORM_TOL * ref
    coef = min(1.0, max_norm / (ref + 1e-6))
    for t, b, o in zip(ts, before, outs or ts):
        want = b.to(f64) * coef
        # the factor's roundings and the product's, then the output's
        tol = want.abs() * (NORM_TOL + 5 * 2.0 ** -24 + HALF[o.dtype]) + TINY[o.dtype]
        assert bool(((o.to(f64) - want).abs() <= tol).all())
        if outs is not None:
            assert torch.equal(t, b)


def test_within_the_norm_nothing_changes():
    ts = some([1000, 33, 70000], 1)
    before = [t.clone() for t in ts]
    B.clip_grads(ts, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    outs = [torch.empty_like(t) for t in ts]
    B.clip_grads(ts, float("inf"), out=outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, before))
    B.clip_grads(ts, 0.0)
    assert all(float(t.abs().max()) == 0 for t in ts)


@pytest.mark.parametrize("value,dtype", [(1e30, f32), (1e-30, f32), (1e-42, f32), (1e30, bf16), (1e-35, bf16), (6e4, f16),
                                         (6e-8, f16), (0.0, f32), (1e-14, f32), (1e19, f32)])
@pytest.mark.parametrize("n,off", [(1, 0), (100, 1), (16384, 0), (100003, 3), (6_000_000, 0)])
def test_values_whose_squares_leave_fp32(value, dtype, n, off):
    t = torch.full((n + off,), value, dtype=dtype, device="cuda")[off:]
    # one small value among large ones and one large among small ones
    u = t.clone()
    u[n // 2] = 1.0
    for v in (t, u):
        ref = ref_norm([v])
        assert abs(float(B.grad_norm([v])) - ref) <= NORM_TOL * ref + 2.0 ** -150


def test_not_finite():
    for bad in (float("nan"), float("inf")):
        ts = some([3000, 5000], 2)
        ts[1][77] = bad
        assert not bool(torch.isfinite(B.grad_norm(ts)))
        ref = [t.clone() for t in ts]
        norm = B.clip_grads(ts, 1.0)
        coef = torch.clamp(1.0 / (norm + 1e-6), max=1.0)
        for t, r in zip(ts, ref):
            assert torch.equal(torch.nan_to_num(t.float(), nan=7.0), torch.nan_to_num((r.float() * coef).to(t.dtype).float(), nan=7.0))
    big = torch.full((10,), 3e38, device="cuda")
    assert float(B.grad_norm([big])) == float("inf")  # past fp32


def test_layouts_and_neighbours():
    """Permuted tensors count once; views in one buffer are scaled, what lies between them is left alone."""
    buf = torch.full((10000,), 2.0, device="cuda")
    ts = [buf[1:1001].view(10, 100).t(), buf[1001:1002], buf[1010:9000].view(-1, 10)]
    keep = buf.clone()
    norm = B.clip_grads(ts, 1.0)
    ref = (4.0 * (1000 + 1 + 7990)) ** 0.5
    assert abs(float(norm) - ref) <= NORM_TOL * ref
    inside = torch.zeros(10000, dtype=torch.bool, device="cuda")
    inside[1:1002] = True
    inside[1010:9000] = True
    assert torch.equal(buf[~inside], keep[~inside]) and bool((buf[inside] < 1).all())
    m = torch.randn(4, 6, 8, device="cuda").permute(2, 0, 1)
    o = torch.empty_like(m)
    assert o.stride() == m.stride()
    B.clip_grads([m], 0.5, out=[o])
    assert bool(((o - m * (0.5 / (m.norm() + 1e-6))).abs() <= m.abs() * 2.0 ** -20).all())


def test_refusals():
    a = torch.ones(100, device="cuda")
    for bad in (lambda: B.grad_norm([a.double()]), lambda: B.grad_norm([a.cpu()]), lambda: B.grad_norm([a[::2]]),
                lambda: B.grad_norm([a[:1].expand(5)]), lambda: B.clip_grads([a], 1.0, out=[a[:50]]),
                lambda: B.clip_grads([a], 1.0, out=[]), lambda: B.clip_grads([a], 1.0, out=[a.double()])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: B.clip_grads([a, a], 1.0), lambda: B.clip_grads([a[:60], a[50:]], 1.0), lambda: B.clip_grads([a], -1.0),
                lambda: B.clip_grads([a], float("nan")), lambda: B.clip_grads([a, a.clone()], 1.0, out=[a.clone(), a])):
        with pytest.raises(B.Bfp8Error):
            bad()
    assert bool((a == 1).all())
    assert abs(float(B.grad_norm([a, a])) - 200 ** 0.5) < 1e-5  # read alone, a tensor may come twice


def test_captured_and_replayed():
    ts = some([100_000, 17, 4000], 5, dtypes=(bf16,))
    outs = [torch.empty_like(t, dtype=f32) for t in ts]
    B.clip_grads(ts, 1.0, out=outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = B.clip_grads(ts, 1.0, out=outs)
    for scale in (3.0, 1e-6):
        for t in ts:
            t.normal_().mul_(scale)
        g.replay()
        torch.cuda.synchronize()
        ref = ref_norm(ts)
        assert abs(float(norm) - ref) <= NORM_TOL * ref
        want = ts[0].to(f64) * min(1.0, 1.0 / (ref + 1e-6))
        assert bool(((outs[0].to(f64) - want).abs() <= want.abs() * 2.0 ** -18 + TINY[f32]).all())


def test_two_streams():
    a, b = some([200_000] * 5, 7), some([300_000] * 4, 8)
    ra, rb = B.grad_norm(a), B.grad_norm(b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s):
            x = B.grad_norm(a)
        with torch.cuda.stream(t):
            y = B.grad_norm(b)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) and torch.equal(y, rb) for x, y in got)
