"""A transformer block's expert layer on this library's operators.

    python examples/expert_layer.py [--rows 4096] [--steps 20]

Serving, in 8 bits: the residual sum and its norm leave as e4m3 rows with
scales (rmsnorm_fp8); every row goes through a shared dense projection
(gemm_fp8); a router sends each row to one of the experts, and the rows, in
expert order, meet the experts' weights (grouped_gemm_fp8).

Training, in 16 bits: the norm (rmsnorm), the experts' products
(grouped_gemm), their gradients (grouped_gemm with trans_b for the rows,
grouped_wgrad for the weights) and the norm's (rmsnorm_grad).

PyTorch supplies memory, the router and the gathering of rows.
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tile_size_decision_gb300 as tiles  # noqa: E402


class ExpertLayer:
    def __init__(self, hidden, width, experts, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g, device=device) * scale).bfloat16()

        self.experts = experts
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.router = normal(hidden, experts, scale=hidden ** -0.5)
        self.weights = normal(experts, hidden, width, scale=hidden ** -0.5)   # k x n
        shared = normal(width, hidden, scale=hidden ** -0.5)                  # n x k
        # The 8-bit weights are laid out once: n x k, one scale per 128 x 128.
        self.shared8 = tiles.quantize_fp8(shared, block_rows=128)
        self.weights8 = tiles.quantize_fp8(self.weights.transpose(1, 2).contiguous(),
                                           block_rows=128)
        self.workspace = tiles.workspace(device)

    def route(self, rows):
        """Rows in expert order and the experts' offsets, all on the device."""
        expert = (rows.float() @ self.router.float()).argmax(1)
        order = expert.argsort(stable=True)
        counts = torch.bincount(expert, minlength=self.experts)
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=rows.device)
        offsets[1:] = counts.cumsum(0)
        return order, offsets

    def serve(self, x, residual):
        """(output rows, the new residual)."""
        q, scales, h = tiles.rmsnorm_fp8(x, self.norm, residual=residual)
        y = tiles.gemm_fp8(q, scales, *self.shared8, workspace=self.workspace)
        order, offsets = self.route(h)
        rows = q.view(torch.uint8)[order].view(torch.float8_e4m3fn)
        e = tiles.grouped_gemm_fp8(rows, scales[order], *self.weights8, offsets,
                                   workspace=self.workspace)
        return y.index_add_(0, order, e), h

    def train_step(self, x, residual, dout, dh):
        """Output rows of the experts and every gradient, given that of the
        output (dout) and of the residual stream past the layer (dh)."""
        y, h = tiles.rmsnorm(x, self.norm, residual=residual)
        order, offsets = self.route(h)
        rows = y[order]
        out = torch.empty((x.shape[0], self.weights.shape[2]), dtype=x.dtype, device=x.device)
        out[order] = tiles.grouped_gemm(rows, self.weights, offsets, workspace=self.workspace)
        dsorted = dout[order]
        dweights = tiles.grouped_wgrad(rows, dsorted, offsets, workspace=self.workspace)
        dy = torch.empty_like(y)
        dy[order] = tiles.grouped_gemm(dsorted, self.weights, offsets, trans_b=True,
                                       workspace=self.workspace)
        dx, dnorm = tiles.rmsnorm_grad(dy, h, self.norm, dh=dh,
                                       workspace=tiles.rmsnorm_grad_workspace(h))
        return out, dx, dnorm, dweights


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    layer = ExpertLayer(a.hidden, a.width, a.experts)
    x, residual, dh = (torch.randn(a.rows, a.hidden, device="cuda").bfloat16() for _ in range(3))
    dout = torch.randn(a.rows, a.width, device="cuda").bfloat16()
    for name, step in (("serve (8 bits)", lambda: layer.serve(x, residual)),
                       ("train step (16 bits)", lambda: layer.train_step(x, residual, dout, dh))):
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
