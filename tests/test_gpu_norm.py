"""The RMS norm with the residual's addition and quantised outputs, and its
gradient, against the definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

F8 = torch.float8_e4m3fn
bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(T, K, seed, residual, wdtype=f32):
    g = gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (n(T, K) * (0.1 + 3 * torch.rand(T, 1, generator=g, device="cuda"))).to(bf16)
    return x, (n(T, K).to(bf16) if residual else None), (1 + 0.3 * n(K)).to(wdtype)


def definition(x, r, w):
    h = x if r is None else (x.float() + r.float()).to(bf16)
    h64 = h.to(f64)
    rstd = (h64.square().mean(1) + EPS).rsqrt() if x.shape[1] else torch.zeros(x.shape[0], dtype=f64, device="cuda")
    return h, rstd, h64 * rstd[:, None] * w.to(f64)


# fp32 sums of positive terms: a thread adds at most K / 32 pairs one after another, the lanes' and warps' sums 10 more; half
# of that in the root, and the mean, eps, root and reciprocal one rounding each.
def rstd_tol(K):
    return ((K / 64 + 12) / 2 + 4) * 2.0 ** -24


def check_codes(q, s, y, tol, what):
    """q [A, C] codes, s [Cb, A] scales of y [A, C] in 64 bits, formed from values within tol of them."""
    A, C = y.shape
    full = torch.nn.functional.pad(y.abs(), (0, -C % 128)).view(A, -1, 128)
    ref = full.amax(2).clamp_min(1e-12) / 448
    rel = tol + 4 * 2.0 ** -24  # the product with r or w, the maximum's, the division by 448
    assert bool(((s.t().to(f64) - ref).abs() <= rel * ref).all()), f"{what}: scales"
    v = y / s.t().to(f64).repeat_interleave(128, 1)[:, :C]
    got = q.view(F8).to(f64)
    # a rounding to e4m3 is off by half a step: 2^-4 of a normal value, 2^-10 of the smallest ones; the value before it by
    # its products' roundings
    slack = v.abs() * (tol + 6 * 2.0 ** -24)
    bad = (got - v.clamp(-448, 448)).abs() > torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + slack
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes"


CASES = [(1, 8), (1, 4096), (3, 1), (5, 129), (2, 8192), (130, 16384), (127, 256), (128, 512), (129, 520), (300, 2001),
         (257, 96), (153, 4096), (400, 640), (160, 8200), (161, 2056), (1000, 33)]


@pytest.mark.parametrize("T,K", CASES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("wdtype", [f32, bf16])
def test_forward(T, K, residual, wdtype):
    x, r, w = make(T, K, T * 7 + K, residual, wdtype)
    h, rstd, y = definition(x, r, w)
    o = B.rms_norm_quant(x, w, residual=r, eps=EPS, cols=True, out=True)
    assert torch.equal(o.h, h) and (residual or o.h is x)
    tol = rstd_tol(K)
    assert bool(((o.rstd.to(f64) - rstd).abs() <= tol * rstd).all())
    check_codes(o.q_row[:, :K], o.s_row[:, :T], y, tol, "rows")
    check_codes(o.q_col[:, :T], o.s_col[:, :K], y.t().contiguous(), tol, "columns")
    assert bool(((o.y.to(f64) - y).abs() <= y.abs() * (2.0 ** -8 + tol + 2.0 ** -22) + 1e-38).all())
    # each output by itself, the same bits
    p = B.rms_norm_quant(x, w, residual=r, eps=EPS)
    assert torch.equal(p.q_row[:, :K], o.q_row[:, :K]) and torch.equal(p.s_row, o.s_row) and p.q_col is None and p.y is None
    p = B.rms_norm_quant(x, w, residual=r, eps=EPS, rows=False, cols=True)
    assert torch.equal(p.q_col[:, :T], o.q_col[:, :T]) and torch.equal(p.s_col[:, :K], o.s_col[:, :K]) and p.q_row is None
    p = B.rms_norm_quant(x, w, residual=r, eps=EPS, rows=False, out=True)
    assert torch.equal(p.y, o.y)
    B.check_device_errors()


@pytest.mark.parametrize("T,K,off,ld", [(200, 1024, 1, 1031), (200, 1024, 8, 1032), (180, 130, 3, 140), (1, 4096, 5, 5000),
                                        (170, 5120, 2, 5122), (400, 2001, 7, 2011), (350, 4001, 1, 4003),
                                        (300, 7003, 5, 7003), (200, 16383, 3, 16384), (5000, 513, 3, 513),
                                        (1200, 1024, 4, 1024), (700, 1026, 6, 1027)])
def test_parts_of_larger_buffers(T, K, off, ld):
    """Rows inside larger buffers: what lies around them is neither read as data (NaN there) nor written."""
    g = gen(T + K)

    def part(values=None):
        buf = torch.full((T * ld + off + 64,), float("nan"), dtype=bf16, device="cuda")
        view = buf[off:off + T * ld].view(T, ld)[:, :K]
        if values is not None:
            view.copy_(values)
        return buf, view
    xv, rv = (torch.randn(T, K, generator=g, device="cuda").to(bf16) for _ in range(2))
    w = torch.randn(K, generator=g, device="cuda")
    _, x = part(xv)
    _, r = part(rv)
    hbuf, h = part()
    o = B.rms_norm_quant(x, w, residual=r, h=h, cols=True, out=True)
    # (rows of another alignment are summed in another order: not the same bits as the packed tensors', but as near)
    hv, rstd, y = definition(xv, rv, w)
    assert o.h is h and torch.equal(h, hv)
    check_codes(o.q_row[:, :K], o.s_row[:, :T], y, rstd_tol(K), "rows")
    check_codes(o.q_col[:, :T], o.s_col[:, :K], y.t().contiguous(), rstd_tol(K), "columns")
    assert bool(((o.y.to(f64) - y).abs() <= y.abs() * (2.0 ** -8 + rstd_tol(K) + 2.0 ** -22) + 1e-38).all())
    around = torch.ones(hbuf.numel(), dtype=torch.bool, device="cuda")
    around[off:off + T * ld].view(T, ld)[:, :K] = False
    assert bool(hbuf[around].isnan().all())
    dy, dh = (torch.randn(T, K, generator=g, device="cuda").to(bf16) for _ in range(2))
    _, dyp = part(dy)
    _, dhp = part(dh)
    check_backward(dyp, h, w, o.rstd, dhp)


@pytest.mark.parametrize("K", [1000, 1003, 4101, 9001])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_sum_in_place(K, which):
    x, r, w = make(400, K, 3, True)
    ref = B.rms_norm_quant(x, w, residual=r, cols=True)
    a, b = x.clone(), r.clone()
    o = B.rms_norm_quant(a, w, residual=b, cols=True, h=a if which == "x" else b)
    assert o.h.data_ptr() == (a if which == "x" else b).data_ptr() and torch.equal(o.h, ref.h)
    assert torch.equal(b if which == "x" else a, r if which == "x" else x)
    assert torch.equal(o.q_row[:, :K], ref.q_row[:, :K]) and torch.equal(o.q_col[:, :400], ref.q_col[:, :400])


def test_halves_of_one_buffer():
    """x and the sum as the left and right columns of the same rows: no element is shared."""
    x, r, w = make(300, 520, 3, True)
    ref = B.rms_norm_quant(x, w, residual=r, cols=True)
    buf = torch.empty(300, 1040, device="cuda", dtype=bf16)
    buf[:, :520] = x
    o = B.rms_norm_quant(buf[:, :520], w, residual=r, cols=True, h=buf[:, 520:])
    assert torch.equal(buf[:, :520], x) and torch.equal(buf[:, 520:], ref.h)
    assert torch.equal(o.q_row[:, :520], ref.q_row[:, :520]) and torch.equal(o.q_col[:, :300], ref.q_col[:, :300])
    with pytest.raises(B.Bfp8Error):
        B.rms_norm_quant(buf[:, :520], w, residual=r, h=buf[:, 519:1039])


@pytest.mark.parametrize("T,K,residual", [(8192, 4096, False), (8192, 4096, True), (6000, 5120, True), (4000, 2001, True),
                                          (4000, 16384, True)])
def test_many_runs_of_many_rows(T, K, residual):
    """Rows that take the places of rows before them, with another number of places than of rows at once."""
    x, r, w = make(T, K, 5, residual)
    first = B.rms_norm_quant(x, w, residual=r)
    dx, dw = B.rms_norm_bwd(x, first.h, w, first.rstd)
    for _ in range(20):
        o = B.rms_norm_quant(x, w, residual=r)
        assert torch.equal(o.h, first.h) and torch.equal(o.rstd, first.rstd)
        assert torch.equal(o.q_row[:, :K], first.q_row[:, :K]) and torch.equal(o.s_row[:, :T], first.s_row[:, :T])
        dx2, dw2 = B.rms_norm_bwd(x, first.h, w, first.rstd)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    B.check_device_errors()


def test_zeros_and_extremes():
    """Rows and columns of zeros have finite scales and zero codes; weights of 0 and below 0; rows of one large value."""
    x = torch.zeros(256, 384, device="cuda", dtype=bf16)
    x[0] = 1e15
    x[1, 5] = -3e4
    x[2] = 1e-30
    w = torch.ones(384, device="cuda")
    w[7], w[8] = 0, -2
    _, rstd, y = definition(x, None, w)
    o = B.rms_norm_quant(x, w, cols=True, out=True)
    check_codes(o.q_row, o.s_row, y, rstd_tol(384), "rows")
    check_codes(o.q_col, o.s_col[:, :384], y.t().contiguous(), rstd_tol(384), "columns")
    assert float(o.q_row[3:].view(F8).float().abs().max()) == 0 and float(o.y[3:].abs().max()) == 0


def check_backward(dy, h, w, rstd, dh):
    T, K = dy.shape
    dx, dw = B.rms_norm_bwd(dy, h, w, rstd, dh=dh)
    h64 = h.to(f64).requires_grad_()
    w64 = w.to(f64).requires_grad_()
    y = h64 * (h64.square().mean(1, keepdim=True) + EPS).rsqrt() * w64
    y.backward(dy.to(f64))
    ref = h64.grad if dh is None else h64.grad + dh.to(f64)
    n = h.to(f64) * rstd.to(f64)[:, None]
    gr = dy.to(f64) * w.to(f64)
    # one rounding to bf16; before it fp32's: of each term, and of the mean (a thread adds up to K / 32 terms in turn)
    size = rstd.to(f64)[:, None] * (gr.abs() + n.abs() * (gr * n).abs().mean(1, keepdim=True))
    tol = ref.abs() * 2.0 ** -8 + size * (K / 32 + 24) * 2.0 ** -24
    assert bool(((dx.to(f64) - ref).abs() <= tol).all())
    # sums over T of fp32 products, at most T + 32 additions one after another
    assert bool(((dw.to(f64) - w64.grad).abs() <= (T + 40) * 2.0 ** -24 * (dy.to(f64) * n).abs().sum(0) + 1e-30).all())
    return dx, dw


@pytest.mark.parametrize("T,K", [(1, 16), (7, 1), (64, 128), (300, 1000), (33, 4096), (2000, 72), (200, 8192), (150, 16384),
                                 (129, 1001), (40, 9001)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward(T, K, with_dh):
    x, r, w = make(T, K, T + K, True, bf16 if K % 3 else f32)
    g = gen(5)
    dy = torch.randn(T, K, generator=g, device="cuda").to(bf16)
    dh = torch.randn(T, K, generator=g, device="cuda").to(bf16) if with_dh else None
    o = B.rms_norm_quant(x, w, residual=r)
    dx, dw = check_backward(dy, o.h, w, o.rstd, dh)
    again = B.rms_norm_bwd(dy, o.h, w, o.rstd, dh=dh)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    B.check_device_errors()


def test_backward_by_differences():
    """The gradient of a loss against central differences of the definition in 64 bits, along random directions."""
    T, K = 6, 40
    x, _, w = make(T, K, 9, False)
    c = torch.randn(T, K, generator=gen(1), device="cuda").to(bf16)
    o = B.rms_norm_quant(x, w)
    dx, dw = B.rms_norm_bwd(c, x, w, o.rstd)

    def loss(x64, w64):
        return float((x64 * (x64.square().mean(1, keepdim=True) + EPS).rsqrt() * w64 * c.to(f64)).sum())
    g = gen(2)
    for _ in range(8):
        vx = torch.randn(T, K, generator=g, device="cuda", dtype=f64)
        vw = torch.randn(K, generator=g, device="cuda", dtype=f64)
        t = 1e-5
        for v, d, at in ((vx, dx, lambda s: loss(x.to(f64) + s * vx, w.to(f64))), (vw, dw, lambda s: loss(x.to(f64), w.to(f64) + s * vw))):
            num = (at(t) - at(-t)) / (2 * t)
            # each element of dx is off by half a bf16 step at most; differences by t^2
            bound = float((d.to(f64) * v).abs().sum()) * 2.0 ** -8 + 1e-6 * float(v.abs().sum())
            assert abs(float((d.to(f64) * v).sum()) - num) <= bound


def test_empty():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda", dtype=bf16)
    o = B.rms_norm_quant(x, w, residual=x, cols=True, out=True)
    assert o.h.shape == (0, 64) and o.q_row.shape[0] == 0 and o.y.shape == (0, 64)
    dx, dw = B.rms_norm_bwd(x, o.h, w, o.rstd)
    assert dx.shape == (0, 64) and float(dw.abs().max()) == 0


def test_captured_and_replayed_on_another_stream():
    x, r, w = make(300, 2048, 1, True)
    dy = torch.randn(300, 2048, device="cuda").to(bf16)
    eager = B.rms_norm_quant(x, w, residual=r, cols=True)
    eager_b = B.rms_norm_bwd(dy, eager.h, w, eager.rstd, dh=r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = B.rms_norm_quant(x, w, residual=r, cols=True)
        b = B.rms_norm_bwd(dy, o.h, w, o.rstd, dh=r)
    s = torch.cuda.Stream()
    for seed in (4, 5):
        x2, r2, _ = make(300, 2048, seed, True)
        x.copy_(x2)
        r.copy_(r2)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
            ref = B.rms_norm_quant(x, w, residual=r, cols=True)
            ref_b = B.rms_norm_bwd(dy, ref.h, w, ref.rstd, dh=r)
        torch.cuda.synchronize()
        assert torch.equal(o.q_row, ref.q_row) and torch.equal(o.h, ref.h) and torch.equal(b[0], ref_b[0])
        assert torch.equal(b[1], ref_b[1]) and not torch.equal(o.h, eager.h) and not torch.equal(b[0], eager_b[0])


def test_refusals():
    x = torch.zeros(4, 256, device="cuda", dtype=bf16)
    w = torch.ones(256, device="cuda")
    rstd = torch.ones(4, device="cuda")
    for bad in (lambda: B.rms_norm_quant(x.float(), w), lambda: B.rms_norm_quant(x, w[:255]), lambda: B.rms_norm_quant(x, w.half()),
                lambda: B.rms_norm_quant(x.t(), w[:4]), lambda: B.rms_norm_quant(x, w, residual=x[:3]),
                lambda: B.rms_norm_quant(x, w, h=x.clone()), lambda: B.rms_norm_quant(x[:1].expand(4, 256), w),
                lambda: B.rms_norm_quant(x, w, residual=x, h=torch.zeros(1, 256, device="cuda", dtype=bf16).expand(4, 256)),
                lambda: B.rms_norm_quant(x.cpu(), w), lambda: B.rms_norm_bwd(x, x, w, rstd[:3]),
                lambda: B.rms_norm_bwd(x, x, w, rstd.to(bf16)), lambda: B.rms_norm_bwd(x, x[:3], w, rstd),
                lambda: B.rms_norm_bwd(x, x, w, rstd, dh=x.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.Bfp8Error):
        B.rms_norm_quant(x, w, eps=0.0)
    wide = torch.zeros(2, 16392, device="cuda", dtype=bf16)
    with pytest.raises(B.Bfp8Error):
        B.rms_norm_quant(wide, torch.ones(16392, device="cuda"))


@pytest.mark.parametrize("residual", [False, True])
def test_norm_linear_module(residual):
    """Forward and gradients of the layer that reads the norm's codes, against the products of the codes' values in 64 bits
    (forward) and the gradient's formula."""
    T, K, N = 200, 384, 256
    torch.manual_seed(0)
    layer = B.Float8NormLinear(K, N, device="cuda")
    with torch.no_grad():
        layer.norm_weight.normal_(1, 0.2)
    x, r, _ = make(T, K, 2, residual)
    x.requires_grad_()
    if residual:
        r.requires_grad_()
    y, h = layer(x.view(2, 100, K), None if r is None else r.view(2, 100, K))
    o = B.rms_norm_quant(x.detach(), layer.norm_weight.detach(), residual=None if r is None else r.detach(), cols=True)
    qw, qwt, sw = B.quant_weight(layer.weight.detach(), with_t=True)
    assert torch.equal(y.reshape(T, N), B.gemm_1x128_128x128(o.q_row, o.s_row, qw, sw, K)) and torch.equal(h.reshape(T, K), o.h)
    dy = torch.randn(2, 100, N, device="cuda").to(bf16)
    dh = torch.randn(2, 100, K, device="cuda").to(bf16)
    torch.autograd.backward([y, h], [dy, dh])
    # the unquantised gradient: the FP8 products are within their quantisations' noise of it (e4m3 rounds by up to 2^-4 of a
    # value, independently: a product over hundreds of terms is within 5% of its norm)
    h64 = o.h.to(f64).requires_grad_()
    w64, nw64 = layer.weight.detach().to(f64).requires_grad_(), layer.norm_weight.detach().to(f64).requires_grad_()
    yr = (h64 * (h64.square().mean(1, keepdim=True) + EPS).rsqrt() * nw64) @ w64.t()
    torch.autograd.backward([yr, h64], [dy.reshape(T, N).to(f64), dh.reshape(T, K).to(f64)])
    near = lambda a, b: float((a.to(f64) - b).norm() / b.norm()) < 0.08  # noqa: E731
    assert near(x.grad, h64.grad) and near(layer.weight.grad, w64.grad) and near(layer.norm_weight.grad, nw64.grad)
    if residual:
        assert torch.equal(r.grad, x.grad)
    with pytest.raises(RuntimeError):
        y2, _ = layer(x, r)
        (g,) = torch.autograd.grad(y2.float().sum(), x, create_graph=True)
        g.float().sum().backward()
    assert bool(torch.isfinite(y.detach()).all())
