"""The few-token layer at the sizes that decide how its parts share their work: each number of buffers of activations
(one, two, three to five, more) and of rows a CTA, and the largest K, I and N.  Tokens and weights are small integers with one
448 a group and a tile, so scales are 1 and the sums of the first product exact; what a right kernel may be off by is small."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

F8 = torch.float8_e4m3fn
bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64


def integers(g, rows, cols, tile):
    """Integers up to 8, with a 448 in every tile x 128 block."""
    v = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda", dtype=torch.int8).to(bf16)
    at = torch.arange(0, cols, 128, device="cuda")
    for r in range(0, rows, tile):
        v[r + (5 * at // 128) % min(tile, rows - r), torch.clamp(at + 3, max=cols - 1)] = 448
    return v


class Layer:
    def __init__(self, E, K, I, N, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.K, self.I, self.N = E, K, I, N
        self.gu, self.d = integers(self.g, E * 2 * I, K, 128), integers(self.g, E * N, I, 128)
        self.qgu, _, self.sgu = B.quant_weight(self.gu)
        self.qd, _, self.sd = B.quant_weight(self.d)
        assert bool((self.sgu == 1).all()) and bool((self.sd == 1).all())

    def inputs(self, T):
        return integers(self.g, T, self.K, 1), 1.5 * torch.randn(T, self.E, generator=self.g, device="cuda")

    def __call__(self, x, logits, k):
        return B.moe_mlp_decode(x, logits, k, self.qgu, self.sgu, self.qd, self.sd, I=self.I, N=self.N)


def groups(v):
    return torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).view(v.shape[0], -1, 128)


def definition(layer, x, idx, w):
    T, K, I, N = x.shape[0], layer.K, layer.I, layer.N
    y = torch.zeros(T, N, dtype=f64, device="cuda")
    tol = torch.zeros_like(y)
    for e in idx.unique().tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        # (integers below 2^24 all the way: exact in fp32 in any order; 64 bits here)
        p = x[t].to(f64) @ layer.gu[e * 2 * I:(e + 1) * 2 * I].to(f64).t()
        a = torch.nn.functional.silu(p[:, :I]) * p[:, I:]
        # the scales' product with 1/448, exp, the quotient and two products: a few roundings of 2^-24
        s = groups(a).abs().amax(2).clamp_min(1e-12) / 448
        wide = s.repeat_interleave(128, 1)[:, :I]
        lo, mid, hi = ((a * (1 + c * 2.0 ** -20) / wide).clamp(-448, 448).to(f32).to(F8).to(f64) * wide for c in (-1, 0, 1))
        d = layer.d[e * N:(e + 1) * N].to(f64)
        wt = w[t, j].to(f64)[:, None]
        y[t] += wt * (mid @ d.t())
        # codes that those roundings may carry over a tie; the scale's; the sums of the second product, at most
        # I / 128 + 160 roundings of terms that add up to |mid| |d|
        tol[t] += wt * ((hi - lo).abs() @ d.abs().t() + (mid.abs() @ d.abs().t()) * (2.0 ** -20 + (I / 128 + 160) * 2.0 ** -24))
    return y, tol + y.abs() * 2.0 ** -8


# T, E, k, K, I, N: buffers of activations (teams of coders), what else is special
SHAPES = [(1, 8, 8, 512, 2048, 512),         # 3 (three teams of two warps)
          (16, 24, 8, 512, 832, 2048),       # 3, two sets of tokens, an expert is one stage
          (8, 12, 5, 256, 1216, 256),        # 4
          (3, 20, 7, 384, 1152, 384),        # 5
          (5, 20, 6, 1000, 1024, 640),       # 6 (a warp an expert), an expert is one stage, K is no multiple of 128
          (3, 9, 4, 640, 2560, 640),         # 2 (all six warps an expert)
          (16, 4, 3, 256, 4160, 256),        # 1
          (8, 3, 2, 128, 16384, 2560),       # 1, a ring of four stages
          (2, 2, 1, 16384, 16384, 128),      # 1, the largest K and I
          (16, 2, 2, 8192, 8192, 128),       # 1, the largest for more than eight tokens
          (1, 4, 2, 16384, 64, 256),         # 8, a ring of four stages
          (16, 16, 4, 7168, 512, 7168)]      # 6, a ring of four stages, 48 rows a CTA


@pytest.mark.parametrize("T,E,k,K,I,N", SHAPES)
def test_every_schedule(T, E, k, K, I, N):
    layer = Layer(E, K, I, N, seed=K + I)
    x, logits = layer.inputs(T)
    y = layer(x, logits, k)
    B.check_device_errors()
    idx, w = B.moe_route(logits, k)
    ref, tol = definition(layer, x, idx.long(), w)
    bad = (y.to(f64) - ref).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}"
    # a value that misses a K-block, or takes a neighbour's, is off by far more
    assert float(tol.square().mean().sqrt()) < 0.05 * float(ref.square().mean().sqrt())
    got = [layer(x, logits, k) for _ in range(20)]
    B.check_device_errors()
    assert all(torch.equal(z, y) for z in got)


def test_the_most_rows():
    """128 rows of the way down a CTA."""
    N = 128 * torch.cuda.get_device_properties(0).multi_processor_count
    test_every_schedule(8, 2, 2, 256, 128, N)


def test_one_size_past_each_limit_is_refused():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    buf = torch.zeros(1 << 16, device="cuda")
    at = ctypes.c_void_p(buf.data_ptr())

    def call(T, K, I, N):
        return B.lib().bfp8_moe_mlp_decode(at, T, K, K, at, 1, 2, 2, None, 1, 0, 1, 1, 1, 1, 1.0, at, -(-K // 16) * 16, at,
                                           -(-K // 128), at, I, at, -(-I // 128), I, N, at, N, at, 1 << 40, B._stream())

    for size in ((1, 16385, 64, 128), (8, 128, 16448, 128), (9, 8193, 64, 128), (16, 128, 8256, 128), (1, 128, 64, 128 * sms + 128)):
        assert call(*size) == 1 and b"16384" in B.lib().bfp8_last_error(), size  # BFP8_ERR_INVALID_ARG, nothing launched
    B.check_device_errors()
