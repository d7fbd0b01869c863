"""The few-token layer of gated experts against its definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

F8 = torch.float8_e4m3fn
bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64


class Layer:
    def __init__(self, E, K, I, N, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.E, self.K, self.I, self.N = E, K, I, N
        gu = (n(E, 2 * I, K) * 1.3 / K ** 0.5).to(bf16)
        d = (n(E, N, I) * 1.3 / I ** 0.5).to(bf16)
        self.qgu, _, self.sgu = B.quant_weight(gu.view(E * 2 * I, K))
        self.qd, _, self.sd = B.quant_weight(d.view(E * N, I))
        self.g = g

    def inputs(self, T, dtype=f32):
        x = torch.randn(T, self.K, generator=self.g, device="cuda").to(bf16)
        return x, (1.5 * torch.randn(T, self.E, generator=self.g, device="cuda")).to(dtype)

    def __call__(self, x, logits, k, **how):
        return B.moe_mlp_decode(x, logits, k, self.qgu, self.sgu, self.qd, self.sd, I=self.I, N=self.N, **how)

    def weight(self, q, s, e, rows, cols):
        nb = -(-rows // 128)
        s = s[e * nb:(e + 1) * nb].to(f64).repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
        return q[e * rows:(e + 1) * rows].view(F8)[:, :cols].to(f64) * s


def groups(v):
    T, C = v.shape
    return torch.nn.functional.pad(v, (0, -C % 128)).view(T, -1, 128)


def held(v, s):
    """The values of the codes of v [T, C] by scales s [T, Cb]."""
    wide = s.repeat_interleave(128, 1)[:, :v.shape[1]]
    return (v / wide).clamp(-448, 448).to(f32).to(F8).to(f64) * wide


def definition(layer, x, idx, w):
    """y in 64 bits from the router's choices, and how far a right kernel may be off."""
    T = x.shape[0]
    y = torch.zeros(T, layer.N, dtype=f64, device="cuda")
    tol = torch.zeros_like(y)
    xs = (groups(x.float()).abs().amax(2).clamp_min(1e-12) * torch.tensor(1 / 448, dtype=f32)).to(f32)
    wide = xs.repeat_interleave(128, 1)[:, :layer.K]
    xq = (x.float() / wide).to(F8).to(f64) * wide.to(f64)  # fp32 quotients, as the kernel's
    for t in range(T):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if e < 0:
                continue
            gu = layer.weight(layer.qgu, layer.sgu, e, 2 * layer.I, layer.K)
            d = layer.weight(layer.qd, layer.sd, e, layer.N, layer.I)
            p, size = gu @ xq[t], gu.abs() @ xq[t].abs()
            gate, up = p[:layer.I], p[layer.I:]
            a = torch.nn.functional.silu(gate) * up
            # fp32 sums of the products, at most Kb + 160 roundings of terms that add up to `size`; silu's slope is below 1.1
            eps = (layer.K / 128 + 160) * 2.0 ** -24
            err = eps * (1.1 * size[:layer.I] * up.abs() + torch.nn.functional.silu(gate).abs() * size[layer.I:]) + a.abs() * 2.0 ** -20
            s = groups(a[None]).abs().amax(2).clamp_min(1e-12) / 448
            lo, mid, hi = (held((a + c * err)[None], s)[0] for c in (-1, 0, 1))
            wt = float(w[t, j])
            y[t] += wt * (d @ mid)
            # codes that the error may carry over a tie, the scale's own rounding and error, and the sums'
            flip = (hi - lo).abs()
            s_rel = float((groups(err[None]).amax(2) / groups(a[None]).abs().amax(2).clamp_min(1e-12)).max()) + 2.0 ** -22
            tol[t] += abs(wt) * (d.abs() @ flip + (d.abs() @ mid.abs()) * (s_rel + (layer.I / 128 + 160) * 2.0 ** -24))
    return y, tol + y.abs() * 2.0 ** -8


def check(layer, x, logits, k, **how):
    y = layer(x, logits, k, **how)
    B.check_device_errors()
    idx, w = B.moe_route(logits, k, **how)
    ref, tol = definition(layer, x, idx, w)
    bad = (y.to(f64) - ref).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}; off by up to {float(((y.to(f64) - ref).abs() / tol).max()):.2f} tolerances"
    # the tolerance is one that wrong values miss: their typical size is far above it
    assert float(tol.square().mean().sqrt()) < 0.2 * float(ref.square().mean().sqrt()) + 1e-30
    return y


@pytest.mark.parametrize("T,E,k,K,I,N", [(1, 4, 1, 128, 64, 128), (1, 8, 8, 256, 128, 256), (2, 5, 2, 40, 64, 128),
                                         (3, 16, 4, 1000, 192, 384), (8, 7, 3, 640, 320, 128), (9, 12, 2, 129, 128, 2560),
                                         (16, 64, 8, 512, 64, 128), (16, 3, 3, 1536, 448, 5120), (5, 2, 1, 16, 64, 9856),
                                         (7, 200, 6, 384, 256, 256), (16, 1024, 32, 128, 64, 128), (4, 40, 5, 4096, 64, 128)])
def test_against_the_definition(T, E, k, K, I, N):
    layer = Layer(E, K, I, N, seed=T + K)
    x, logits = layer.inputs(T, bf16 if T % 2 else f32)
    y = check(layer, x, logits, k, score="sigmoid" if E % 2 else "softmax", renormalize=T % 3 != 0, scale=1.5)
    assert torch.equal(y, layer(x, logits, k, score="sigmoid" if E % 2 else "softmax", renormalize=T % 3 != 0, scale=1.5))


def test_one_expert_of_any_width():
    layer = Layer(1, 200, 64, 77)
    x, logits = layer.inputs(3)
    check(layer, x, logits, 1)


def test_groups_bias_and_masks():
    layer = Layer(32, 256, 128, 256)
    x, logits = layer.inputs(12)
    logits[3] = float("-inf")               # a token without experts
    logits[5, 4:] = float("-inf")           # fewer experts than choices
    logits[6, 7] = float("nan")
    bias = torch.randn(32, device="cuda") * 0.1
    y = check(layer, x, logits, 6, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2)
    assert float(y[3].abs().max()) == 0
    logits[:] = float("-inf")               # no token has any
    assert float(layer(x, logits, 6).abs().max()) == 0
    B.check_device_errors()


def test_every_token_at_one_expert():
    layer = Layer(8, 384, 256, 384)
    x, logits = layer.inputs(16)
    logits[:] = 0
    logits[:, 5] = 9
    check(layer, x, logits, 1, score="softmax")


def test_zero_tokens_and_rows_of_zeros():
    layer = Layer(4, 256, 64, 128)
    x, logits = layer.inputs(4)
    assert layer(x[:0], logits[:0], 2).shape == (0, 128)
    x[1] = 0
    y = check(layer, x, logits, 2)
    assert float(y[1].abs().max()) == 0


def test_weights_of_experts_that_no_token_reaches_are_not_used():
    layer = Layer(16, 256, 128, 256)
    x, logits = layer.inputs(2)
    logits[:, 3] += 50
    logits[:, 11] += 50
    ref = layer(x, logits, 2)
    for e in range(16):
        if e not in (3, 11):
            layer.qgu[e * 256:(e + 1) * 256] = 0x7F  # NaN
            layer.qd[e * 256:(e + 1) * 256] = 0x7F
            layer.sd[e * 2:(e + 1) * 2] = float("nan")
    assert torch.equal(layer(x, logits, 2), ref)


def test_padding_of_codes_is_not_data():
    """Codes with bytes between the features and the row stride, NaN there; tokens and outputs in larger buffers."""
    layer = Layer(6, 200, 64, 128)
    x, logits = layer.inputs(5)
    ref = layer(x, logits, 3)
    for name, cols in (("qgu", 200), ("qd", 64)):
        q = getattr(layer, name)
        wide = torch.full((q.shape[0], 272), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, :cols] = q[:, :cols]
        setattr(layer, name, wide)
    for name in ("sgu", "sd"):
        s = getattr(layer, name)
        wide = torch.full((s.shape[0], 7), float("nan"), device="cuda")
        wide[:, :s.shape[1]] = s
        setattr(layer, name, wide)
    big = torch.full((5, 333), float("nan"), dtype=bf16, device="cuda")
    big[:, 1:201] = x
    lg = torch.full((5, 11), 1e9, device="cuda")
    lg[:, 2:8] = logits
    assert torch.equal(layer(big[:, 1:201], lg[:, 2:8], 3), ref)


def test_near_the_five_launches():
    """The same layer from its parts: quantised tokens, two routed products, the activation in torch, the combine.  They
    round the products and the experts' outputs to bf16, which this layer does not: a few halves of bf16's steps a term."""
    layer = Layer(16, 512, 256, 384)
    x, logits = layer.inputs(6)
    idx, w = B.moe_route(logits, 4)
    plan = B.moe_plan(idx, 16, align=1)
    q, s = B.quant_lhs(x)
    gu = B.gemm_routed_1x128_128x128(q, s, layer.qgu, layer.sgu, plan, 512, 512).float()
    a = (torch.nn.functional.silu(gu[:, :256]) * gu[:, 256:]).to(bf16)
    q, s = B.quant_lhs(a)
    y = B.moe_combine(B.gemm_routed_1x128_128x128(q, s, layer.qd, layer.sd, plan, 384, 256, gathered=False), plan, w)
    z = layer(x, logits, 4)
    # e4m3 noise of the few codes that the roundings to bf16 carry over a tie (2^-3 of a value each)
    assert float((y.float() - z.float()).norm() / z.float().norm()) < 0.03


@pytest.mark.parametrize("T,E,k,K,I,N", [(1, 16, 8, 1024, 512, 1024), (16, 64, 8, 1024, 512, 1024), (16, 8, 2, 2048, 2048, 2048),
                                         (5, 64, 6, 1920, 704, 1920), (12, 8, 2, 512, 4096, 512), (7, 32, 4, 384, 192, 4096)])
def test_many_runs_in_a_row(T, E, k, K, I, N):
    """The same bits of calls that follow one another without a pause, on inputs in turn."""
    layer = Layer(E, K, I, N)
    sets = [layer.inputs(T) for _ in range(3)]
    first = [layer(x, logits, k) for x, logits in sets]
    got = [layer(*sets[i % 3], k) for i in range(90)]
    B.check_device_errors()
    assert all(torch.equal(y, first[i % 3]) for i, y in enumerate(got))
    assert all(bool(torch.isfinite(y.float()).all()) and float(y.float().abs().max()) > 0 for y in first)


def test_captured_replayed_and_concurrent():
    layer, other = Layer(16, 512, 256, 512), Layer(8, 256, 128, 256, seed=3)
    x, logits = layer.inputs(4)
    x2, logits2 = other.inputs(9)
    layer(x, logits, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(x, logits, 4)
    for _ in range(3):
        nx, nl = layer.inputs(4)
        x.copy_(nx)
        logits.copy_(nl)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer(x, logits, 4))
    # two layers at once on two streams: each launch waits for all of its own CTAs
    r1, r2 = layer(x, logits, 4), other(x2, logits2, 3)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(30):
        with torch.cuda.stream(s):
            a = layer(x, logits, 4)
        with torch.cuda.stream(t):
            b = other(x2, logits2, 3)
        got.append((a, b))
    torch.cuda.synchronize()
    B.check_device_errors()
    assert all(torch.equal(a, r1) and torch.equal(b, r2) for a, b in got)


def test_refusals():
    layer = Layer(4, 256, 64, 128)
    x, logits = layer.inputs(4)
    call = lambda **kw: B.moe_mlp_decode(**{**dict(x=x, logits=logits, k=2, qgu=layer.qgu, sgu=layer.sgu, qd=layer.qd,  # noqa: E731
                                                   sd=layer.sd, I=64, N=128), **kw})
    for kw in (dict(x=x[:3]), dict(x=x.float()), dict(logits=logits[:, :3]), dict(I=128), dict(N=256), dict(qgu=layer.qgu[:, :240]),
               dict(sgu=layer.sgu[:, :1]), dict(sd=layer.sd[:2]), dict(qd=layer.qd.float()), dict(sd=layer.sd.double()),
               dict(qgu=layer.qgu.cpu()), dict(bias=torch.zeros(3, device="cuda")), dict(score="other")):
        with pytest.raises(ValueError):
            call(**kw)
    many, ml = layer.inputs(17)
    with pytest.raises(B.Bfp8Error, match="17"):
        call(x=many, logits=ml)
    with pytest.raises(B.Bfp8Error):
        call(k=5)


def test_a_served_layer():
    """Norm, router, experts, the next norm, as a served model runs them: a step captured once and replayed for new tokens."""
    K, E = 512, 16
    layer = Layer(E, K, 256, K)
    g = torch.Generator(device="cuda").manual_seed(1)
    gate = (torch.randn(E, K, generator=g, device="cuda") / K ** 0.5).to(bf16)
    w1, w2 = (1 + 0.1 * torch.randn(K, generator=g, device="cuda") for _ in range(2))
    x = torch.randn(3, K, generator=g, device="cuda").to(bf16)
    r = torch.randn(3, K, generator=g, device="cuda").to(bf16)

    def step():
        o = B.rms_norm_quant(x, w1, residual=r, rows=False, out=True)
        y = layer(o.y, (o.y.float() @ gate.float().t()), 4, score="sigmoid")
        return B.rms_norm_quant(y, w2, residual=o.h), o, y

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n, o, y = step()
    x.normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    B.check_device_errors()
    check(layer, o.y, o.y.float() @ gate.float().t(), 4, score="sigmoid")
    assert torch.equal(o.h, (x.float() + r.float()).to(bf16)) and torch.equal(n.h, (y.float() + o.h.float()).to(bf16))


def test_a_training_step_to_its_clipping():
    """A norm and the linear layer that reads it, their gradients, and the clipping of all of them by their norm."""
    torch.manual_seed(0)
    a, b = B.Float8NormLinear(256, 384, device="cuda"), B.Float8NormLinear(384, 256, device="cuda")
    x = torch.randn(200, 256, device="cuda").to(bf16)
    u, h = a(x)
    y, _ = b(u)
    (y.float() + h.float()).square().mean().backward()
    grads = [p.grad for m in (a, b) for p in m.parameters()]
    assert all(bool(torch.isfinite(t).all()) and float(t.float().abs().max()) > 0 for t in grads)
    ref = float(torch.stack([t.to(f64).square().sum() for t in grads]).sum().sqrt())
    out = [torch.empty_like(t, dtype=f32) for t in grads]
    norm = B.clip_grads(grads, 0.5 * ref, out=out)
    assert abs(float(norm) - ref) <= 2.0 ** -20 * ref
    assert abs(float(B.grad_norm(out)) - 0.5 * ref) <= 2.0 ** -18 * ref + 1e-6
