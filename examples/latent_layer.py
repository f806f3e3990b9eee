"""One latent MoE layer's operators together, as a program would run them.

decode_round   a decode round of 1..20 rows: layer norm of the hidden rows, the
               route (latent, router logits, top-16) on the normalised rows, a
               gated feed-forward product on the latent and the linear product
               back to the hidden width onto the residual stream.
TrainStep      a training step of the layer's dense branch (a shared expert on
               the hidden rows): norm, gated, linear with residual, and the
               whole backward pass, every gradient from the library's kernels;
               dx gets the residual branch's share, dy itself, by one addition
               of torch's after them.

Weights and inputs are random; run it on an MI355X with
    python examples/latent_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from latent_projection_top_amd import block, route  # noqa: E402

BF = torch.bfloat16


def weights(inputs: int, inner: int, outputs: int, device="cuda", seed: int = 0) -> dict:
    """Norm parameters (FP32) and the three matrices, [K][N] BF16."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def matrix(k, n):
        return (torch.randn(k, n, generator=gen, device=device) * k ** -0.5).to(BF)

    return {"norm_w": 1 + 0.1 * torch.randn(route.HIDDEN, generator=gen, device=device),
            "norm_b": 0.1 * torch.randn(route.HIDDEN, generator=gen, device=device),
            "w_gate": matrix(inputs, inner), "w_up": matrix(inputs, inner), "w_down": matrix(inner, outputs)}


class DecodeRound:
    """Plans, workspaces and buffers of a decode round, made once."""

    def __init__(self, rows: int, inner: int, device: int | None = None):
        dev = f"cuda:{torch.cuda.current_device() if device is None else device}"
        self.norm = block.NormPlan(rows, route.HIDDEN)
        self.route = route.Plan(route.MODE_DECODE, rows)
        self.gated = block.GatedPlan(rows, route.LATENT, inner)
        self.down = block.LinearPlan(rows, inner, route.HIDDEN)
        self.ws = {"route": self.route.new_workspace(), "gated": self.gated.new_workspace(),
                   "down": self.down.new_workspace()}

        def empty(n, dtype=BF):
            return torch.empty(rows, n, dtype=dtype, device=dev)

        self.xn, self.latent, self.h = empty(route.HIDDEN), empty(route.LATENT), empty(inner)
        self.logits, self.weights = empty(route.EXPERTS, torch.float32), empty(route.TOPK, torch.float32)
        self.ids = empty(route.TOPK, torch.int32)

    def __call__(self, x, w_latent, w_router, p: dict) -> None:
        """x [rows][7168] becomes x + layer(x), in place; ids and weights hold
        the round's experts. Five launches or so, nothing allocated: the call
        can be captured into a HIP graph."""
        block.layer_norm(self.norm, x, p["norm_w"], p["norm_b"], self.xn)
        route.fused(self.route, self.xn, w_latent, w_router, self.latent, self.logits, self.ids, self.weights,
                    self.ws["route"])
        block.gated(self.gated, self.latent, p["w_gate"], p["w_up"], self.h, self.ws["gated"])
        block.linear(self.down, self.h, p["w_down"], x, self.ws["down"], residual=x)


class TrainStep:
    """Forward and backward pass of y = x + gated(norm(x)) w_down."""

    def __init__(self, rows: int, inner: int):
        k = route.HIDDEN
        self.norm = block.NormPlan(rows, k)
        self.gated = block.GatedPlan(rows, k, inner, training=True)
        self.down = block.LinearPlan(rows, inner, k, training=True)
        self.ws = [p.new_workspace() for p in (self.norm, self.gated, self.down)]

        def empty(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        self.xn, self.y, self.dxn, self.dx = (empty(rows, k) for _ in range(4))
        self.h, self.d_gate, self.d_up, self.dh = (empty(rows, inner) for _ in range(4))
        self.mean, self.rstd = (empty(rows, dtype=torch.float32) for _ in range(2))
        self.grads = {"norm_w": empty(k, dtype=torch.float32), "norm_b": empty(k, dtype=torch.float32),
                      "w_gate": empty(k, inner), "w_up": empty(k, inner), "w_down": empty(inner, k)}

    def forward(self, x, p: dict) -> torch.Tensor:
        block.layer_norm(self.norm, x, p["norm_w"], p["norm_b"], self.xn, self.mean, self.rstd)
        block.gated(self.gated, self.xn, p["w_gate"], p["w_up"], self.h, self.ws[1], self.d_gate, self.d_up)
        block.linear(self.down, self.h, p["w_down"], self.y, self.ws[2], residual=x)
        return self.y

    def backward(self, x, dy, p: dict) -> tuple[torch.Tensor, dict]:
        """dx (the residual branch included) and the weights' gradients."""
        g = self.grads
        block.linear_backward(self.down, dy, self.h, p["w_down"], None, self.dh, g["w_down"], None, self.ws[2])
        block.gated_backward(self.gated, self.dh, self.xn, p["w_gate"], p["w_up"], self.d_gate, self.d_up,
                             self.dxn, g["w_gate"], g["w_up"], self.ws[1])
        block.layer_norm_backward(self.norm, self.dxn, x, p["norm_w"], self.mean, self.rstd, self.dx,
                                  g["norm_w"], g["norm_b"], self.ws[0])
        self.dx.add_(dy)
        return self.dx, g

    def descend(self, x, target, p: dict, part: float = 0.05) -> float:
        """One step down the gradient of the mean squared error, as far as the
        gradient itself says takes off `part` of the error; returns the error
        before the step."""
        diff = self.forward(x, p).float() - target.float()
        loss = diff.square().mean()
        # gradients of loss * (values / 2), scaled back in the step
        _, grads = self.backward(x, diff.to(BF), p)
        scale = 2.0 / diff.numel()
        slope = sum(g.float().square().sum() for g in grads.values()) * scale ** 2
        for k, g in grads.items():
            p[k].copy_(p[k].float() - part * loss / slope * scale * g.float())
        return float(loss)


def main() -> None:
    inner = 2048
    x = torch.randn(8, route.HIDDEN, device="cuda").to(BF)
    w_latent = (torch.randn(route.HIDDEN, route.LATENT, device="cuda") * route.HIDDEN ** -0.5).to(BF)
    w_router = torch.randn(route.HIDDEN, route.EXPERTS, device="cuda") * route.HIDDEN ** -0.5
    decode = DecodeRound(8, inner)
    p = weights(route.LATENT, inner, route.HIDDEN)
    before = x.clone()
    decode(x, w_latent, w_router, p)
    torch.cuda.synchronize()
    print(f"decode round: 8 rows, |layer(x)| / |x| = {float((x - before).float().norm() / before.float().norm()):.3f}, "
          f"first row's experts {decode.ids[0].tolist()}")

    rows = 512
    step = TrainStep(rows, inner)
    p = weights(route.HIDDEN, inner, route.HIDDEN, seed=1)
    x = torch.randn(rows, route.HIDDEN, device="cuda").to(BF)
    target = torch.randn(rows, route.HIDDEN, device="cuda").to(BF)
    for i in range(5):
        print(f"training step {i}: loss {step.descend(x, target, p):.4f}")


if __name__ == "__main__":
    main()
