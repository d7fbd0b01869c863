"""Host logic of the routed layer (no GPU: the kernels' entries are stood in for)."""
import copy

import pytest
import torch

from blockwise_scaled_fp8_gb300 import module as M


@pytest.fixture
def layer(monkeypatch):
    """A layer on the CPU whose decode() gives the sum of the weights that were quantised."""
    monkeypatch.setattr(M, "quant_weight", lambda w: (w.detach().float().sum(), None, None))
    monkeypatch.setattr(M, "moe_route", lambda logits, k, **_: (None, None))
    monkeypatch.setattr(M, "moe_plan", lambda *_, **__: None)
    monkeypatch.setattr(M, "moe_experts_decode", lambda x, qw, sw, plan, w, N: qw.expand(x.shape[0], N))
    return M.Float8RoutedExperts(16, 128, 4, 2)


def _decode(layer):
    return float(layer.decode(torch.zeros(1, 16, dtype=torch.bfloat16), torch.zeros(1, 4))[0, 0])


def test_decode_refuses_codes_of_other_weights(layer):
    with pytest.raises(RuntimeError, match="quantize"):
        _decode(layer)

    def step():
        opt = torch.optim.SGD(layer.parameters(), lr=1.0)
        layer.weight.grad = torch.ones_like(layer.weight)
        opt.step()

    def swap():
        layer.weight = torch.nn.Parameter(layer.weight.detach() + 1)

    def data():
        layer.weight.data = layer.weight.data.clone()

    state = copy.deepcopy(layer.state_dict())
    for change in (step, lambda: layer.load_state_dict(state), lambda: layer.to(torch.float32).to(torch.bfloat16), swap, data,
                   lambda: torch.nn.init.ones_(layer.weight)):
        layer.quantize()
        assert _decode(layer) == float(layer.weight.detach().float().sum())
        change()
        with pytest.raises(RuntimeError, match="changed since quantize"):
            _decode(layer)


def test_decode_keeps_codes_of_unchanged_weights(layer):
    layer.quantize()
    want = _decode(layer)
    layer.eval().train().requires_grad_(False)
    layer.to(torch.device("cpu"))
    layer.weight.grad = None
    assert _decode(layer) == want


@pytest.fixture
def experts(monkeypatch):
    """blockwise_fp8_experts on the CPU whose entries compute y = 2 x and dx = 2 dy."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    monkeypatch.setattr(M, "moe_route", lambda logits, k, **_: (i(logits.shape[0], k), torch.zeros(logits.shape[0], k)))
    monkeypatch.setattr(M, "moe_plan", lambda idx, E: M.MoePlan(i(E + 1), idx, i(128), i(E)))
    monkeypatch.setattr(M, "moe_experts_fwd", lambda x, w, plan, wt: (2 * x, (x, x, x, x, x, plan, wt)))
    monkeypatch.setattr(M, "moe_experts_bwd", lambda dy, saved: (2 * dy.detach(), torch.zeros(4, 128, 128), saved[-1]))
    monkeypatch.setattr(M, "moe_route_bwd", lambda logits, *_, **__: torch.zeros_like(logits))
    return M.blockwise_fp8_experts


def test_a_second_derivative_is_refused(experts):
    """The kernels' gradients have none: without a refusal its terms would be left out of the sum."""
    x = torch.randn(3, 128).bfloat16().requires_grad_()
    w = torch.zeros(4, 128, 128, dtype=torch.bfloat16, requires_grad=True)
    y, _ = experts(x, w, torch.zeros(3, 4, requires_grad=True), 2)
    (g,) = torch.autograd.grad(y.float().square().sum() + x.float().pow(3).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        g.float().sum().backward()


def test_a_first_derivative_with_its_graph_is_served(experts):
    x = torch.ones(3, 128).bfloat16().requires_grad_()
    w = torch.zeros(4, 128, 128, dtype=torch.bfloat16, requires_grad=True)
    y, _ = experts(x, w, torch.zeros(3, 4, requires_grad=True), 2)
    (g,) = torch.autograd.grad(y.float().sum(), x, create_graph=True)
    assert bool((g == 2).all())


def test_the_returned_counts_may_be_written(experts):
    """Summed over processes in place, say, before the backward pass."""
    x = torch.ones(3, 128).bfloat16().requires_grad_()
    w = torch.zeros(4, 128, 128, dtype=torch.bfloat16, requires_grad=True)
    y, counts = experts(x, w, torch.zeros(3, 4, requires_grad=True), 2)
    counts.add_(1)
    y.float().sum().backward()
    assert bool((x.grad == 2).all())


def test_choice_bias_joins_in_fp32_after_the_layer_is_cast(monkeypatch):
    """Casting a whole model to bf16 casts the buffer too."""
    seen = []
    monkeypatch.setattr(M, "moe_route", lambda logits, k, bias=None, **_: seen.append(bias) or (None, None))
    monkeypatch.setattr(M, "moe_plan", lambda *_, **__: None)
    monkeypatch.setattr(M, "quant_weight", lambda w: (w, None, w))
    monkeypatch.setattr(M, "moe_experts_decode", lambda x, qw, sw, plan, w, N: x.new_zeros(x.shape[0], N))
    layer = M.Float8RoutedExperts(16, 128, 4, 2, choice_bias=True)
    layer.choice_bias += 0.5
    for cast in (False, True):
        if cast:
            layer.to(torch.bfloat16)
        layer.quantize()
        layer.decode(torch.zeros(1, 16, dtype=torch.bfloat16), torch.zeros(1, 4))
        with pytest.raises(AttributeError):  # the forward stops at what stands in for the plan
            layer(torch.zeros(1, 16, dtype=torch.bfloat16), torch.zeros(1, 4))
    assert len(seen) == 4 and all(b.dtype == torch.float32 and bool((b == 0.5).all()) for b in seen)
