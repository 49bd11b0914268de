"""One layer of NVFP4 experts from compressed scales, end to end on the GPU.

    python examples/expert_layer.py

The layer keeps its weights as E2M1 codes and their scales as CSF stacks.  A
call adds the residual stream and norms and quantises it in one launch, chooses
each token's experts, decodes the scales of the chosen experts only, runs the
experts' gate/up and down products with the activation and the requantisation
in their epilogues, and adds up each token's experts with the router's weights.
Nothing is read back by the host.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lossless_nvfp4_scale_gb300 import csf, ops  # noqa: E402


@dataclass
class ExpertLayer:
    norm_weight: torch.Tensor    # [hidden]
    router: torch.Tensor         # [experts, hidden]
    gate_up: torch.Tensor        # uint8 [experts, 2 * inner, hidden / 2]: the gate rows, then the up rows
    gate_up_scales: csf.Stack    # [experts, 2 * inner, hidden / 16]
    down: torch.Tensor           # uint8 [experts, hidden, inner / 2]
    down_scales: csf.Stack       # [experts, hidden, inner / 16]
    alpha: torch.Tensor          # float32 [2, experts]: the two products' tensor scales
    x_scale: torch.Tensor        # float32 [1]: the quantised input's tensor scale
    act_scale: torch.Tensor      # float32 [1]: the quantised activation's
    workspace: tuple[torch.Tensor, torch.Tensor]   # decoded scales, shared by layers of this shape

    def __call__(self, x: torch.Tensor, residual: torch.Tensor, k: int, off: torch.Tensor | None = None):
        """The experts' output for x [tokens, hidden], and the residual stream with x added.  `off` (bool, of the
        logits' shape or one that broadcasts to it) switches experts off; a token may have fewer than k left, or none."""
        q, residual = ops.rms_norm(x, self.norm_weight, ops.NVFP4, residual=residual, tensor_scale=self.x_scale)
        logits = residual @ self.router.T
        r = ops.route(logits if off is None else logits.masked_fill(off, -float("inf")), k)
        csf.decode_pair(self.gate_up_scales, self.down_scales, *self.workspace, expert_start=r.expert_start,
                        layout=csf.LAYOUT_BLOCKED)
        act = ops.expert_matmul(q, self.gate_up, self.workspace[0], expert_start=r.expert_start, rows=r.rows,
                                alpha=self.alpha[0], activation="silu", gated=True, out=ops.NVFP4,
                                out_tensor_scale=self.act_scale)
        y = ops.expert_matmul(act, self.down, self.workspace[1], expert_start=r.expert_start, alpha=self.alpha[1],
                              out=torch.float32)
        # choices that fell away have slot -1 and add nothing
        return ops.combine(y, r.slots, r.weights, out=x.dtype), residual


def random_layer(experts: int, hidden: int, inner: int, seed: int = 0) -> ExpertLayer:
    """A layer of random weights whose products keep the size of their input."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=g)

    def weights(rows, cols):
        codes = torch.randint(0, 256, (experts, rows, cols // 2), dtype=torch.uint8, **dev)
        base = torch.randint(0x28, 0x34, (experts, rows, 1), dtype=torch.uint8, **dev)
        scales = base + torch.randint(0, 12, (experts, rows, cols // 16), dtype=torch.uint8, **dev)
        return codes, csf.prepare(scales.contiguous(), csf.NVFP4)

    gate_up, gate_up_scales = weights(2 * inner, hidden)
    down, down_scales = weights(hidden, inner)
    x_scale, act_scale = torch.full((1,), 0.01, device="cuda"), torch.full((1,), 0.005, device="cuda")
    alpha = torch.stack([(0.5 + torch.rand(experts, **dev)) * s * 0.6 / n ** 0.5
                         for s, n in ((x_scale, hidden), (act_scale, inner))])
    return ExpertLayer(
        (1 + 0.1 * torch.randn(hidden, **dev)).to(torch.bfloat16),
        (torch.randn(experts, hidden, **dev) / hidden ** 0.5).to(torch.bfloat16),
        gate_up, gate_up_scales, down, down_scales, alpha, x_scale, act_scale,
        tuple(torch.empty(csf.blocked_bytes(s), dtype=torch.uint8, device="cuda") for s in (gate_up_scales, down_scales)))


def main():
    layer = random_layer(experts=128, hidden=1600, inner=512)
    for tokens in (1, 64, 2048):
        x = torch.randn(tokens, 1600, device="cuda").to(torch.bfloat16)
        residual = torch.randn(tokens, 1600, device="cuda").to(torch.bfloat16)
        layer(x, residual, 8)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            y, _ = layer(x, residual, 8)
        end.record()
        torch.cuda.synchronize()
        print(f"{tokens:5d} tokens, 8 of 128 experts: {start.elapsed_time(end) * 50:8.1f} us, "
              f"output rms {y.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
