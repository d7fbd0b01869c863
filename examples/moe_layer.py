"""A routed mixture-of-experts layer trained for a few steps and then used to
decode: the router's logits choose each token's experts, every product runs in
blockwise FP8, the choice bias follows the experts' load.

    python examples/moe_layer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blockwise_scaled_fp8_gb300 as bfp8  # noqa: E402


def train(steps: int = 20, tokens: int = 1024, features: int = 256, experts: int = 16, k: int = 4, seed: int = 0):
    """Fits y = x A (a fixed linear map) with a routed layer.  Returns (the layer, the router, the losses)."""
    torch.manual_seed(seed)
    layer = bfp8.Float8RoutedExperts(features, features, experts, k, score="sigmoid", groups=4, top_groups=2, group_top=2,
                                     choice_bias=True, device="cuda")
    gate = torch.nn.Linear(features, experts, bias=False, device="cuda", dtype=torch.bfloat16)
    target = torch.randn(features, features, device="cuda") / features ** 0.5
    opt = torch.optim.AdamW([*layer.parameters(), *gate.parameters()], lr=1e-2)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, features, device="cuda", dtype=torch.bfloat16)
        y, counts = layer(x, gate(x))
        loss = (y.float() - x.float() @ target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        # an expert above its share becomes a little less likely to be chosen, one below it a little more
        layer.choice_bias += 1e-2 * torch.sign(tokens * k / experts - counts)
        losses.append(loss.detach())
    return layer, gate, [float(v) for v in losses]


def main() -> None:
    bfp8.build()
    layer, gate, losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    layer.quantize()
    x = torch.randn(3, layer.in_features, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        y, counts = layer(x, gate(x))
        z = layer.decode(x, gate(x))
    bfp8.check_device_errors()
    print(f"{int((counts > 0).sum())} experts reached by 3 tokens; decode differs from the training forward by at most "
          f"{float((y.float() - z.float()).abs().max()):.2e}")


if __name__ == "__main__":
    main()
