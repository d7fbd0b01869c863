"""Tensors that an entry point writes by the caller's wish count as written for autograd: a graph that saved their old
values refuses to go backward instead of using the new ones."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

bf16, f32 = torch.bfloat16, torch.float32


def saved(t):
    """A graph whose backward pass wants t as it is now."""
    leaf = torch.ones_like(t, requires_grad=True)
    return (leaf * t).sum()


@pytest.mark.parametrize("into", ["x", "residual", "view"])
def test_the_norms_sum(into):
    x, r = torch.randn(8, 256, device="cuda").to(bf16), torch.randn(8, 256, device="cuda").to(bf16)
    buf = torch.randn(16, 256, device="cuda").to(bf16)
    h, graph = dict(x=(x, x), residual=(r, r), view=(buf[4:12], buf))[into]
    loss = saved(graph)
    B.rms_norm_quant(x, torch.ones(256, device="cuda"), residual=r, h=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_its_inputs_and_its_own_outputs_do_not():
    x, r, w = torch.randn(8, 256, device="cuda").to(bf16), torch.randn(8, 256, device="cuda").to(bf16), torch.ones(256, device="cuda")
    losses = [saved(t) for t in (x, r, w)]
    o = B.rms_norm_quant(x, w, residual=r)
    B.rms_norm_bwd(x, o.h, w, o.rstd)
    for loss in losses:
        loss.backward()


def test_clipping():
    a, b = torch.randn(1000, device="cuda"), torch.randn(33, device="cuda").to(bf16)
    losses = [saved(a), saved(b)]
    B.grad_norm([a, b])
    out = [torch.zeros_like(a), torch.zeros_like(b)]
    written = [saved(t) for t in out]
    B.clip_grads([a, b], 1.0, out=out)
    for loss in losses:
        loss.backward()
    for loss in written:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    losses = [saved(a), saved(b)]
    B.clip_grads([a, b], 1.0)
    for loss in losses:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_codes_of_weights_that_clipping_wrote_are_refused():
    layer = B.Float8RoutedExperts(128, 128, 4, 2, device="cuda")
    x, logits = torch.randn(3, 128, device="cuda").to(bf16), torch.randn(3, 4, device="cuda")
    layer.quantize()
    layer.decode(x, logits)
    B.clip_grads([layer.weight], 1e-3)
    with pytest.raises(RuntimeError, match="changed since"):
        layer.decode(x, logits)


def test_tensors_of_inference_mode():
    with torch.inference_mode():
        x, r = torch.randn(8, 256, device="cuda").to(bf16), torch.randn(8, 256, device="cuda").to(bf16)
        B.rms_norm_quant(x, torch.ones(256, device="cuda"), residual=r, h=x)
        B.clip_grads([torch.ones(100, device="cuda")], 1.0)
