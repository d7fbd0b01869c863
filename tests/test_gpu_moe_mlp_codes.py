"""The few-token layer's codes of its activations, bit for bit, where quotients lie at ties of two codes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

F8 = torch.float8_e4m3fn
bf16, f32 = torch.bfloat16, torch.float32


def parts(n):
    """n as a sum of at most 128 e4m3 values that are powers of two or 448."""
    out = [448] * (n // 448)
    n -= 448 * len(out)
    return out + [1 << b for b in range(9) if n >> b & 1]


@pytest.mark.parametrize("T", [3, 16])
def test_activations_at_ties(T):
    """One expert a token whose way down is the identity, so y is the activations' codes times their scale.  Up rows give
    n c for integers n, with 448 * 16 the largest of the group and the others ties between two codes of n / 16; c, a product of
    random scales, decides on which side of the tie the fp32 quotient by the scale falls.  Gates are the same large value,
    whose exp does not reach fp32's 1, so that every fp32 operation before the codes is one of torch's."""
    E, K, I = 64, 128, 128
    g = torch.Generator(device="cuda").manual_seed(T)
    ns = [448 * 16] + [m << p for m in range(17, 32, 2) for p in range(8)]
    assert max(ns) == ns[0] and len(ns) <= I
    w = torch.zeros(2 * I, K)
    w[:I, 0] = 448  # gates: 448 * 448 x scales
    for i, n in enumerate(ns):
        v = torch.tensor(parts(n), dtype=f32)
        w[I + i, :len(v)] = v
    qgu = w.to(F8).view(torch.uint8).cuda().repeat(E, 1)
    sgu = 0.01 * (1 + torch.rand(2 * E, 1, generator=g, device="cuda"))  # (I = 128: a tile of gates, one of ups)
    sgu[::2] += 0.2
    qd = torch.eye(I).to(F8).view(torch.uint8).cuda().repeat(E, 1)
    sd = torch.ones(E, 1, device="cuda")
    flips = near = 0
    for _ in range(8):
        x = (0.5 + torch.rand(T, 1, generator=g, device="cuda")).to(bf16).repeat(1, K)
        logits = torch.randn(T, E, generator=g, device="cuda")
        y = B.moe_mlp_decode(x, logits, 1, qgu, sgu, qd, sd, I=I, N=I)
        B.check_device_errors()
        e = logits.argmax(1)
        inv = torch.tensor(1 / 448, dtype=f32, device="cuda")
        xs = x[:, :1].float() * inv
        assert bool(((x.float() / xs).to(F8).float() == 448).all())
        # exact integers times a scale: one rounding of the scales' product, one of the product with it
        dot = 448 * torch.tensor(ns, dtype=f32, device="cuda")
        gate = (xs * sgu[2 * e]) * (448.0 * 448.0)
        assert float(gate.min()) > 17
        a = gate * ((xs * sgu[2 * e + 1]) * dot)
        s = a.amax(1, keepdim=True) * inv
        codes = (a / s).to(F8).float()
        # the weight is 1: its scale times the scale, once, times codes that 1 multiplies
        want = torch.zeros(T, I, dtype=bf16, device="cuda")
        want[:, :len(ns)] = (s * codes).to(bf16)
        assert torch.equal(y, want), f"{int((y != want).sum())} of {T * len(ns)} codes"
        flips += int(((a * (1 / s.double()).float()).to(F8).float() != codes).sum())
        near += T * (len(ns) - 1)
    assert flips > 0.01 * near  # (a product with 1/s instead of the quotient would be seen)
