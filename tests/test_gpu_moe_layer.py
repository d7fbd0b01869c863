"""The routed experts end to end: the composed path against 64-bit dense sums,
its gradients against the formulas, decoding against the training forward, and
the example."""
import importlib.util
import os

import numpy as np
import pytest

import moe_reference as ref
from gpu_util import sqnr_db, torch

import blockwise_scaled_fp8_gb300 as B

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# Blockwise e4m3 products of normal data keep about 28 dB (an e4m3 code is off by up to 1/16, 1/16/sqrt(3) rms, per
# operand); a gradient through two of them adds their errors: 3 dB less, and 1 dB of margin.
SQNR_ONE, SQNR_TWO = 27.0, 24.0


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    yield
    B.check_device_errors()


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T,K,N,E,k,score", [(300, 256, 128, 8, 2, "softmax"), (97, 384, 256, 24, 6, "sigmoid"),
                                             (1, 128, 128, 4, 4, "softmax")])
def test_routed_experts_forward_and_gradients(T, K, N, E, k, score):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = rn(T, K).bfloat16().requires_grad_()
    w = (0.05 * rn(E, N, K)).bfloat16().requires_grad_()
    logits = rn(T, E).requires_grad_()
    if T > 10:
        with torch.no_grad():
            logits[3] = -float("inf")             # a padding token
    y, counts = B.blockwise_fp8_experts(x, w, logits, k, score=score, scale=1.5)
    dy = 1e-2 * rn(T, N).bfloat16()
    y.backward(dy)
    ln = logits.detach().cpu().numpy()
    p, ok = ref.scores(ln, score, float(np.finfo(np.float32).min))
    idx, _ = ref.choose(p, ok, ln, score, None, k, 1, 1, 1)
    wt = ref.weights(p, idx, True, 1.5)
    assert np.array_equal(counts.cpu().numpy(), np.bincount(idx[idx >= 0], minlength=E))
    xn, wn, dn = _f64(x), _f64(w), _f64(dy)
    yr, dxr, dwr, dwt = np.zeros((T, N)), np.zeros((T, K)), np.zeros((E, N, K)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if e >= 0:
                out = wn[e] @ xn[t]
                yr[t] += wt[t, j] * out
                dwt[t, j] = out @ dn[t]
                dxr[t] += wt[t, j] * (dn[t] @ wn[e])
                dwr[e] += wt[t, j] * np.outer(dn[t], xn[t])
    dlr = ref.route_grad(p, idx, dwt, score, True, 1.5)
    assert sqnr_db(yr, _f64(y)) >= SQNR_ONE
    assert sqnr_db(dxr, _f64(x.grad)) >= SQNR_ONE
    assert sqnr_db(dwr, _f64(w.grad)) >= SQNR_ONE
    if np.abs(dlr).max() > 0:                     # (all experts chosen, renormalised softmax: still not zero)
        assert sqnr_db(dlr, _f64(logits.grad)) >= SQNR_TWO - 4.0   # a difference of dot products
    if T > 10:
        assert not y[3].any() and not x.grad[3].any() and not logits.grad[3].any()


def test_decode_matches_the_training_forward():
    g = torch.Generator(device="cuda").manual_seed(9)
    layer = B.Float8RoutedExperts(512, 256, 16, 4, score="sigmoid", groups=4, top_groups=2, choice_bias=True, device="cuda")
    layer.choice_bias.normal_(generator=g).mul_(0.1)
    with pytest.raises(RuntimeError, match="quantize"):
        layer.decode(torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 16, device="cuda"))
    layer.quantize()
    for lead in ((1,), (3,), (2, 20)):
        x = torch.randn(*lead, 512, generator=g, device="cuda").bfloat16()
        logits = torch.randn(*lead, 16, generator=g, device="cuda")
        with torch.no_grad():
            y, _ = layer(x, logits)
        z = layer.decode(x, logits)
        assert z.shape == (*lead, 256)
        # the same codes and scales: fp32 sums in another order, each expert's output rounded to bf16 once in both
        # (2^-8 relative apart at most), as the sum is
        size = float(y.float().abs().max())
        assert float((y.float() - z.float()).abs().max()) <= 3 * 2.0 ** -8 * size


def test_layer_refuses_wrong_types_and_shapes():
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 128, 128, dtype=torch.bfloat16, device="cuda")
    l = torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError, match="bfloat16"):
        B.blockwise_fp8_experts(x.float(), w, l, 2)
    with pytest.raises(ValueError, match="logits"):
        B.blockwise_fp8_experts(x, w, l[:, :7], 2)
    with pytest.raises(B.Bfp8Error, match="k=9"):
        B.blockwise_fp8_experts(x, w, l, 9)
    with pytest.raises(ValueError, match="score"):
        B.blockwise_fp8_experts(x, w, l, 2, score="relu")
    with pytest.raises(ValueError, match="128"):
        B.Float8RoutedExperts(128, 100, 8, 2)


def test_training_forward_refuses_a_plan_of_unaligned_rows():
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 128, 128, dtype=torch.bfloat16, device="cuda")
    idx, weight = B.moe_route(torch.zeros(4, 8, device="cuda"), 2)
    with pytest.raises(ValueError, match="multiples of 128"):
        B.moe_experts_fwd(x, w, B.moe_plan(idx, 8, align=1), weight)


def test_layer_takes_broadcast_and_strided_inputs():
    """One row of logits for every token, and a token broadcast: the same as their copies, gradients summed."""
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(4, 128, 256, generator=g, device="cuda").bfloat16()
    row, x = torch.randn(1, 4, generator=g, device="cuda"), torch.randn(6, 256, generator=g, device="cuda").bfloat16()
    def grads(l, x1):
        l, x1 = l.clone().requires_grad_(), x1.clone().requires_grad_()
        y, _ = B.blockwise_fp8_experts(x1.expand(6, 256), w, l.expand(6, 4), 2)
        y.float().sum().backward()
        return y, l.grad, x1.grad
    y0, l0, x0 = grads(row.expand(6, 4).contiguous(), x)
    y1, l1, _ = grads(row, x)
    assert torch.equal(y0, y1) and float((l1 - l0.sum(0, keepdim=True)).abs().max()) <= 8 * 2.0 ** -24 * float(l0.abs().sum())
    y2, _, x2 = grads(row, x[:1])
    assert torch.equal(y2, y1[:1].expand(6, 128)) and x2.shape == (1, 256)
    layer = B.Float8RoutedExperts(256, 128, 4, 2, device="cuda")
    with torch.no_grad():
        layer.weight.copy_(w)
    layer.quantize()
    assert torch.equal(layer.decode(x[:1].expand(6, 256), row.expand(6, 4)), layer.decode(x[:1].repeat(6, 1), row.repeat(6, 1)))


def test_layer_in_a_cuda_graph_and_on_a_side_stream():
    g = torch.Generator(device="cuda").manual_seed(2)
    layer = B.Float8RoutedExperts(256, 128, 8, 2, device="cuda")
    layer.quantize()
    x = torch.randn(5, 256, generator=g, device="cuda").bfloat16()
    logits = torch.randn(5, 8, generator=g, device="cuda")
    want = layer.decode(x, logits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(layer.decode(x, logits), want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = layer.decode(x, logits)
    logits.copy_(torch.randn(5, 8, generator=g, device="cuda"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, layer.decode(x, logits))


def test_example_learns():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    _, _, losses = m.train(steps=12)
    assert losses[-1] < 0.7 * losses[0]


def test_layer_of_no_tokens():
    layer = B.Float8RoutedExperts(128, 256, 8, 2, device="cuda")
    x = torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    logits = torch.zeros(0, 8, device="cuda", requires_grad=True)
    y, counts = layer(x, logits)
    assert y.shape == (0, 256) and not counts.any()
    y.float().sum().backward()
    assert x.grad.shape == (0, 128) and logits.grad.shape == (0, 8) and not layer.weight.grad.any()
    layer.quantize()
    assert layer.decode(x.detach(), logits.detach()).shape == (0, 256)
