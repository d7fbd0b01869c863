"""Autograd wrapper: a bf16 linear layer whose forward and backward run the
blockwise-FP8 training path of this library (the Float8BlockwiseLinear
computation that "Enable blockwise FP8 dense training kernels on ROCm" tests).

Forward: one launch quantises x (1x128 groups along K and 128x1 groups along
the token dim) and W (128x128 tiles, as is and transposed), then the forward
GEMM; the quantised operands stay in a per-call workspace.  Backward: dY is
quantised once (both forms), then the input-gradient and weight-gradient
GEMMs.  Every step runs in the library's kernels through the C ABI; this
module only reshapes, allocates outputs with torch and keeps the workspace
for the backward.  No bias: the method has none.

Float8RoutedExperts puts a mixture of such layers behind a router: the router's
logits choose each token's experts, and the layer is the weighted sum of their
outputs, differentiable in the tokens, the experts' weights and the logits.
"""
from __future__ import annotations

import torch

from . import (MoePlan, linear_bwd_saved, linear_fwd_train, linear_train_workspace, moe_experts_bwd, moe_experts_decode,
               moe_experts_fwd, moe_plan, moe_route, moe_route_bwd, quant_weight)


class _BlockwiseFp8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
            raise TypeError("blockwise_fp8_linear: x and weight must be bfloat16")
        lead = x.shape[:-1]
        K = x.shape[-1]
        N = weight.shape[0]
        if weight.shape[1] != K:
            raise ValueError(f"blockwise_fp8_linear: weight is {tuple(weight.shape)}, x has {K} features")
        x2 = x.reshape(-1, K).contiguous()
        M = x2.shape[0]
        ws = linear_train_workspace(M, N, K, device=x.device)
        y = linear_fwd_train(x2, weight.contiguous(), ws)
        ctx.save_for_backward(ws)
        ctx.dims = (M, N, K)
        ctx.lead = lead
        return y.reshape(*lead, N)

    @staticmethod
    def backward(ctx, dy):
        (ws,) = ctx.saved_tensors
        M, N, K = ctx.dims
        dy2 = dy.reshape(M, N).to(torch.bfloat16).contiguous()
        dx, dw = linear_bwd_saved(dy2, ws, M, N, K)
        return dx.reshape(*ctx.lead, K), dw


def blockwise_fp8_linear(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """y = x W^T with blockwise-FP8 forward and backward (x [..., K], weight [N, K], bf16)."""
    return _BlockwiseFp8Linear.apply(x, weight)


class Float8BlockwiseLinear(torch.nn.Module):
    """nn.Linear (no bias) in bf16 whose matmuls run as blockwise-scaled FP8 on the
    5th-generation tensor cores: 1x128 activation / gradient groups, 128x128 weight
    tiles, 128x1 groups for the weight gradient's right operand."""

    def __init__(self, in_features: int, out_features: int, device=None, dtype=torch.bfloat16):
        super().__init__()
        if dtype != torch.bfloat16:
            raise TypeError("Float8BlockwiseLinear keeps its weight in bfloat16")
        self.in_features, self.out_features = in_features, out_features
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, device=device, dtype=dtype))
        torch.nn.init.kaiming_uniform_(self.weight, a=5 ** 0.5)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear) -> "Float8BlockwiseLinear":
        if linear.bias is not None:
            raise ValueError("Float8BlockwiseLinear has no bias")
        m = cls(linear.in_features, linear.out_features, device=linear.weight.device)
        with torch.no_grad():
            m.weight.copy_(linear.weight.to(torch.bfloat16))
        return m

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return blockwise_fp8_linear(x, self.weight)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, bias=False"


class _BlockwiseFp8Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, logits, k, bias, route):
        how = {name: route[name] for name in ("score", "renormalize", "scale")}
        idx, w = moe_route(logits, k, bias=bias, **route)
        plan = moe_plan(idx, weight.shape[0])
        y, saved = moe_experts_fwd(x, weight, plan, w)
        qxt, sxt, qwt, sw, ye, plan, w = saved
        # (not the counts: they are the caller's to write, and the gradients do without)
        ctx.save_for_backward(qxt, sxt, qwt, sw, ye, plan.offs, plan.row, plan.src, w, logits, idx)
        ctx.how = how
        ctx.mark_non_differentiable(plan.counts)
        return y, plan.counts

    @staticmethod
    @torch.autograd.function.once_differentiable  # the kernels' gradients carry no graph
    def backward(ctx, dy, _):
        qxt, sxt, qwt, sw, ye, offs, row, src, w, logits, idx = ctx.saved_tensors
        plan = MoePlan(offs, row, src, None)
        dx, dw, dweight = moe_experts_bwd(dy.to(torch.bfloat16).contiguous(), (qxt, sxt, qwt, sw, ye, plan, w))
        dlogits = moe_route_bwd(logits, idx, w, dweight, **ctx.how) if ctx.needs_input_grad[2] else None
        return dx, dw, dlogits, None, None, None


def blockwise_fp8_experts(x: torch.Tensor, weight: torch.Tensor, logits: torch.Tensor, k: int, bias=None, **route):
    """y[t] = sum over the token's k experts e of their routing weight times W_e x[t],
    with blockwise-FP8 products forward and backward (x [T, K], weight [E, N, K] bf16,
    N % 128 == 0; logits [T, E] bf16 or fp32; route: moe_route's score, groups, top_groups,
    group_top, renormalize, scale).  Returns (y [T, N], the experts' token counts [E])."""
    if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError("blockwise_fp8_experts: x and weight must be bfloat16")
    if x.dim() != 2 or weight.dim() != 3 or weight.shape[2] != x.shape[1] or \
            tuple(logits.shape) != (x.shape[0], weight.shape[0]):
        raise ValueError(f"blockwise_fp8_experts: x is {tuple(x.shape)}, weight {tuple(weight.shape)}, logits "
                         f"{tuple(logits.shape)}")
    route = {"score": "softmax", "renormalize": True, "scale": 1.0, **route}
    return _BlockwiseFp8Experts.apply(x.contiguous(), weight.contiguous(), logits.contiguous(), k, bias, route)


class Float8RoutedExperts(torch.nn.Module):
    """A mixture of ``experts`` linear layers (no bias) behind a router: forward(x [..., K],
    logits [..., E]) -> (y [..., N], token counts [E]).  ``choice_bias`` (fp32, not trained)
    joins the choice of experts alone; a training loop that balances their load moves it by the
    counts.  decode() is the serving form for a few tokens: the experts' weights are quantised
    once, by quantize(), and each reached expert's are read once a call."""

    def __init__(self, in_features: int, out_features: int, experts: int, k: int, score: str = "softmax",
                 groups: int = 1, top_groups=None, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
                 choice_bias: bool = False, device=None):
        super().__init__()
        if out_features % 128:
            raise ValueError("Float8RoutedExperts: out_features must be a multiple of 128")
        self.in_features, self.out_features, self.experts, self.k = in_features, out_features, experts, k
        self.route = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top,
                          renormalize=renormalize, scale=scale)
        self.weight = torch.nn.Parameter(
            torch.empty(experts, out_features, in_features, device=device, dtype=torch.bfloat16))
        for w in self.weight:
            torch.nn.init.kaiming_uniform_(w, a=5 ** 0.5)
        self.register_buffer("choice_bias", torch.zeros(experts, device=device) if choice_bias else None)
        self._codes = self._codes_of = None

    def forward(self, x: torch.Tensor, logits: torch.Tensor):
        lead = x.shape[:-1]
        y, counts = blockwise_fp8_experts(x.reshape(-1, self.in_features), self.weight,
                                          logits.reshape(-1, self.experts), self.k, bias=self._bias(), **self.route)
        return y.reshape(*lead, self.out_features), counts

    def _bias(self):
        """The choice bias in the router's fp32 (a cast of the whole model casts the buffer)."""
        return None if self.choice_bias is None else self.choice_bias.float()

    def _weight_state(self):
        """What changes with the weights: their storage, and torch's count of writes in place."""
        w = self.weight
        return w.data_ptr(), w.device, None if w.is_inference() else w._version

    @torch.no_grad()
    def quantize(self) -> None:
        """Quantises the experts' weights for decode(); call it again after they change (decode() refuses codes of
        weights that were replaced, moved or written since; writes through weight.data or in inference mode leave no
        trace that it could see).  The codes are not part of the layer's state."""
        qw, _, sw = quant_weight(self.weight.reshape(self.experts * self.out_features, self.in_features))
        self._codes, self._codes_of = (qw, sw), self._weight_state()

    @torch.no_grad()
    def decode(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        if self._codes is None:
            raise RuntimeError("Float8RoutedExperts.decode: call quantize() first")
        if self._codes_of != self._weight_state():
            raise RuntimeError("Float8RoutedExperts.decode: the weights have changed since quantize(); call it again")
        lead = x.shape[:-1]
        logits, x = logits.reshape(-1, self.experts).contiguous(), x.reshape(-1, self.in_features).contiguous()
        idx, w = moe_route(logits, self.k, bias=self._bias(), **self.route)
        y = moe_experts_decode(x, *self._codes, moe_plan(idx, self.experts, align=1), w,
                               self.out_features)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, experts={self.experts}, k={self.k}, "
                f"bias=False")
