"""A transformer block's expert layer on this library's operators.

    python examples/expert_layer.py [--rows 4096] [--choices 2] [--steps 20]

Serving, in 8 bits: the residual sum and its norm leave as e4m3 rows with
scales (rmsnorm_fp8); every row goes through a shared dense projection
(gemm_fp8); a router sends each row to one of the experts, or to several with
a weight each (choices), the rows are sorted by expert and laid out in that
order (expert_sort, expert_dispatch), meet the experts' weights
(grouped_gemm_fp8) and are added up by token (expert_combine).

Training, in 16 bits: the norm (rmsnorm), the rows' way to the experts and
back, the experts' products (grouped_gemm), and the gradients of all of them:
expert_combine_grad for the weighted sum, grouped_gemm with trans_b for the
rows, grouped_wgrad for the weights, expert_combine for the dispatch,
rmsnorm_grad for the norm.  clip_grads scales the parameters' gradients.

PyTorch supplies memory, and the router's products and softmax.
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tile_size_decision_gb300 as tiles  # noqa: E402


class ExpertLayer:
    def __init__(self, hidden, width, experts, device="cuda", seed=0, choices=1):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g, device=device) * scale).bfloat16()

        self.experts, self.choices = experts, choices
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.router = normal(hidden, experts, scale=hidden ** -0.5)
        self.weights = normal(experts, hidden, width, scale=hidden ** -0.5)   # k x n
        shared = normal(width, hidden, scale=hidden ** -0.5)                  # n x k
        # The 8-bit weights are laid out once: n x k, one scale per 128 x 128.
        self.shared8 = tiles.quantize_fp8(shared, block_rows=128)
        self.weights8 = tiles.quantize_fp8(self.weights.transpose(1, 2).contiguous(),
                                           block_rows=128)
        self.workspace = tiles.workspace(device)

    def choose(self, rows):
        """Each row's experts (rows x choices) and their weights, which are the
        softmax of the chosen experts' logits (None of a single choice)."""
        logits, experts = (rows.float() @ self.router.float()).topk(self.choices, 1)
        return experts, None if self.choices == 1 else logits.softmax(1)

    def route(self, rows):
        """Pairs (row * choices + choice) in expert order and the experts' offsets, all
        on the device."""
        _, offsets, order = tiles.expert_sort(self.choose(rows)[0], self.experts)
        return order.long(), offsets

    def serve(self, x, residual):
        """(output rows, the new residual)."""
        q, scales, h = tiles.rmsnorm_fp8(x, self.norm, residual=residual)
        y = tiles.gemm_fp8(q, scales, *self.shared8, workspace=self.workspace)
        experts, weights = self.choose(h)
        slots, offsets, _ = tiles.expert_sort(experts, self.experts)
        rows, row_scales = tiles.expert_dispatch(q, slots, scales=scales)
        e = tiles.grouped_gemm_fp8(rows, row_scales, *self.weights8, offsets,
                                   workspace=self.workspace)
        return y.add_(tiles.expert_combine(e, slots, weights)), h

    def train_step(self, x, residual, dout, dh):
        """Output rows of the experts and every gradient (of the rows, the norm, the
        experts' weights and, with several choices, the router), given that of the
        output (dout) and of the residual stream past the layer (dh)."""
        y, h = tiles.rmsnorm(x, self.norm, residual=residual)
        experts, weights = self.choose(h)
        slots, offsets, _ = tiles.expert_sort(experts, self.experts)
        rows = tiles.expert_dispatch(y, slots)
        e = tiles.grouped_gemm(rows, self.weights, offsets, workspace=self.workspace)
        out = tiles.expert_combine(e, slots, weights)
        if weights is None:
            de = tiles.expert_dispatch(dout, slots)
        else:
            de, dweight = tiles.expert_combine_grad(dout, e, slots, weights)
        dweights = tiles.grouped_wgrad(rows, de, offsets, workspace=self.workspace)
        drows = tiles.grouped_gemm(de, self.weights, offsets, trans_b=True,
                                   workspace=self.workspace)
        dy = tiles.expert_combine(drows, slots)
        grads = [dweights]
        if weights is not None:
            # Through the softmax of the chosen logits to the router and to h.
            chosen = weights * (dweight - (weights * dweight).sum(1, keepdim=True))
            dlogits = torch.zeros((x.shape[0], self.experts), device=x.device).scatter_(
                1, experts, chosen)
            grads.append(h.float().t() @ dlogits)
            dh = (dh.float() + dlogits @ self.router.float().t()).to(dh.dtype)
        dx, dnorm = tiles.rmsnorm_grad(dy, h, self.norm, dh=dh,
                                       workspace=tiles.rmsnorm_grad_workspace(h))
        return out, dx, dnorm, *grads


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--choices", type=int, default=1, help="experts of a row")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    layer = ExpertLayer(a.hidden, a.width, a.experts, choices=a.choices)
    x, residual, dh = (torch.randn(a.rows, a.hidden, device="cuda").bfloat16() for _ in range(3))
    dout = torch.randn(a.rows, a.width, device="cuda").bfloat16()

    def train():
        _, _, *grads = layer.train_step(x, residual, dout, dh)
        return tiles.clip_grads(grads, 1.0), grads

    for name, step in (("serve (8 bits)", lambda: layer.serve(x, residual)),
                       ("train step (16 bits)", train)):
        for _ in range(3):
            step()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            step()
        end.record()
        tiles.check(layer.workspace)
        print(f"{name}: {start.elapsed_time(end) / a.steps * 1e3:.0f} us for {a.rows} rows, "
              f"{a.hidden} -> {a.width}, {a.experts} experts")
    return 0


if __name__ == "__main__":
    sys.exit(main())
