"""Float8NormLinear where torch leaves the strides of gradients and inputs open: no rows, one row, one feature."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

bf16 = torch.bfloat16


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("lead", [(0,), (2, 0), (1,), (1, 1)])
@pytest.mark.parametrize("N", [1, 384])
def test_few_rows(lead, N, residual):
    torch.manual_seed(0)
    K = 256
    layer = B.Float8NormLinear(K, N, device="cuda")
    x = torch.randn(*lead, K, device="cuda").to(bf16).requires_grad_()
    r = torch.randn(*lead, K, device="cuda").to(bf16) if residual else None
    y, h = layer(x, r)
    assert y.shape == (*lead, N) and h.shape == (*lead, K)
    y.float().sum().backward()  # (the gradient of a sum is one element, expanded)
    first = [x.grad] + [p.grad for p in layer.parameters()]
    assert x.grad.shape == x.shape and all(bool(torch.isfinite(g).all()) for g in first)
    if 0 in lead:
        assert all(float(p.grad.float().abs().max()) == 0 for p in layer.parameters())
    # the same gradient, written out
    x.grad = None
    layer.zero_grad()
    y, _ = layer(x, r)
    y.backward(torch.ones(*lead, N, device="cuda").to(bf16).clone())
    assert all(torch.equal(a, b) for a, b in zip(first, [x.grad] + [p.grad for p in layer.parameters()]))
    B.check_device_errors()


def test_inputs_without_rows_of_any_strides():
    layer = B.Float8NormLinear(256, 128, device="cuda")
    x = torch.empty(1, 1, device="cuda", dtype=bf16).expand(1, 256)[:0].expand(0, 256)
    wide = torch.empty(256, 0, device="cuda", dtype=bf16).t()
    for a, b in ((x, None), (wide, None), (wide, x)):
        y, h = layer(a, b)
        assert y.shape == (0, 128) and h.shape == (0, 256)


def test_gradients_that_are_not_packed():
    """Those of a transposed and of a sliced output are the packed ones."""
    layer = B.Float8NormLinear(256, 384, device="cuda")
    x = torch.randn(40, 256, device="cuda").to(bf16).requires_grad_()
    dy = torch.randn(40, 384, device="cuda").to(bf16)
    dh = torch.randn(40, 256, device="cuda").to(bf16)
    want = None
    for a, b in ((dy, dh), (dy.t().contiguous().t(), dh.t().contiguous().t()), (torch.cat([dy, dy], 1)[:, :384], torch.cat([dh, dh], 1)[:, :256])):
        x.grad = None
        layer.zero_grad()
        y, h = layer(x, torch.ones_like(x))
        torch.autograd.backward([y, h], [a, b])
        got = [x.grad] + [p.grad for p in layer.parameters()]
        want = want or got
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_residual_of_another_type_is_refused():
    layer = B.Float8NormLinear(256, 128, device="cuda")
    x = torch.zeros(4, 256, device="cuda", dtype=bf16)
    with pytest.raises(ValueError, match="residual"):
        layer(x, x.float())
