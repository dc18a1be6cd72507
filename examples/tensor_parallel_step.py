"""A tensor-parallel training step and a decoding step over virtual ranks.

A stack of feed-forward layers is split over N ranks the usual way: rank r holds F / N columns
of each layer's first matrix and the same rows of its second one, so every rank ends a layer
with a partial sum of its output.  What happens between the ranks' products runs here:

  forward    vAllReduceRmsNorm          partial sums -> residual stream, normed input of the
                                        next layer on every rank
  backward   vAllReduceRmsNormBackward  partial input gradients -> gradient of the stream and of
                                        every rank's partial sum, and of the norm's weight
  step       vClipGradNorm              one norm over all ranks' gradients, then clipping
  decoding   vAllReduceRmsNormQuant     as forward for one token, normed input in 8 bits

    python examples/tensor_parallel_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from collective_communication_virtual_gb300 import vcomm as V  # noqa: E402

EPS = 1e-6


class Block:
    """Feed-forward layers split over the communicator's ranks, with an RMS norm behind each."""

    def __init__(self, comm, layers: int, hidden: int, ffn: int, dtype=torch.bfloat16, seed: int = 0):
        self.comm, self.n = comm, V.vcommCount(comm)
        self.layers, self.hidden, self.dtype = layers, hidden, dtype
        gen = torch.Generator().manual_seed(seed)
        part = ffn // self.n

        def matrix(rows, cols):
            return (torch.randn(rows, cols, generator=gen) * rows ** -0.5).to(dtype).cuda()

        # [layer][rank]
        self.up = [[matrix(hidden, part) for _ in range(self.n)] for _ in range(layers)]
        self.down = [[matrix(part, hidden) for _ in range(self.n)] for _ in range(layers)]
        # every rank holds every norm's weight (the one before the first layer too)
        self.norm = [[torch.ones(hidden, device="cuda") for _ in range(self.n)] for _ in range(layers + 1)]

    # ---- parameters, their gradients and the list that the norm is taken over -----------------

    def parameters(self):
        """[rank][tensor]: the matrices' pieces, then the norms' weights, the same on every rank."""
        return [[m[r] for m in self.up] + [m[r] for m in self.down] + [w[r] for w in self.norm] for r in range(self.n)]

    def prepare_training(self, rows: int):
        self.rows = rows
        self.desc = V.vRmsNormDesc(rows, self.hidden, self.dtype, torch.float32, EPS)
        self.grads = [[torch.zeros_like(p) for p in ps] for ps in self.parameters()]
        split = 2 * self.layers
        self.list = V.vTensorList(self.grads, replicated=[False] * split + [True] * (self.layers + 1))
        self.grad_norm = torch.zeros(1, device="cuda")
        self.norm_space = torch.empty(V.vGradNormWorkspace(self.list, self.comm), dtype=torch.uint8, device="cuda")
        self.back_space = torch.empty(V.vRmsNormBackwardWorkspace(self.desc, self.comm), dtype=torch.uint8,
                                      device="cuda")

    def _rows(self, rows):
        return torch.empty(rows, self.hidden, dtype=self.dtype, device="cuda")

    # ---- forward ------------------------------------------------------------------------------

    def forward(self, x):
        """The last norm's output on every rank, and what the backward pass needs."""
        n, rows = self.n, x.shape[0]
        kept = []
        # the stack's input is no partial sum: rank 0 sends it, the others zeros
        partial = [x] + [torch.zeros_like(x) for _ in range(n - 1)]
        stream = None
        for layer in range(self.layers + 1):
            out, normed, rstd = self._rows(rows), [self._rows(rows) for _ in range(n)], torch.empty(rows, device="cuda")
            V.vAllReduceRmsNorm(self.desc, partial, stream, self.norm[layer][0], out, normed, rstd, self.comm)
            stream = out
            if layer == self.layers:
                kept.append((stream, rstd, normed, None, None))
                break
            wide = [normed[r] @ self.up[layer][r] for r in range(n)]
            active = [torch.relu(w) for w in wide]
            partial = [active[r] @ self.down[layer][r] for r in range(n)]
            kept.append((stream, rstd, normed, wide, active))
        return kept[-1][2], kept

    # ---- backward -------------------------------------------------------------------------------

    def backward(self, kept, d_normed):
        """Fills self.grads from the gradient of the last norm's output (on rank 0; the others'
        partial gradients are zero)."""
        n, layers = self.n, self.layers
        partial = [d_normed] + [torch.zeros_like(d_normed) for _ in range(n - 1)]
        d_stream = None
        for layer in range(layers, -1, -1):
            stream, rstd, normed, wide, active = kept[layer]
            out, weight_grad = [self._rows(self.rows) for _ in range(n)], torch.empty(self.hidden, device="cuda")
            if layer < layers:
                # through this layer's products, each rank on its own part
                partial = []
                for r in range(n):
                    d_active = d_stream[r] @ self.down[layer][r].t()
                    torch.mm(active[r].t(), d_stream[r], out=self.grads[r][layers + layer])
                    d_wide = d_active * (wide[r] > 0)
                    torch.mm(normed[r].t(), d_wide, out=self.grads[r][layer])
                    partial.append(d_wide @ self.up[layer][r].t())
            V.vAllReduceRmsNormBackward(self.desc, partial, stream, rstd, self.norm[layer][0],
                                        None if d_stream is None else d_stream[0], out, weight_grad, self.back_space,
                                        self.comm)
            for r in range(n):
                self.grads[r][2 * layers + layer].copy_(weight_grad)
            d_stream = out
        return d_stream[0]

    def step(self, rate: float, max_norm: float):
        """Clip all ranks' gradients by their common norm and take a step; returns that norm."""
        V.vClipGradNorm(self.list, max_norm, self.grad_norm, self.norm_space, self.comm)
        for params, grads in zip(self.parameters(), self.grads):
            torch._foreach_add_(params, grads, alpha=-rate)
        return self.grad_norm

    # ---- one token ------------------------------------------------------------------------------

    def decode_quantised(self, partial, stream, layer: int):
        """The norm before `layer` for a few tokens, in 8 bits: (values, scales, stream)."""
        n, rows = self.n, partial[0].shape[0]
        desc = V.vRmsNormDesc(rows, self.hidden, self.dtype, torch.float32, EPS, quant_group=128)
        q = [torch.empty(rows, self.hidden, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(n)]
        scales = [torch.empty(rows, -(-self.hidden // 128), device="cuda") for _ in range(n)]
        out = self._rows(rows)
        V.vAllReduceRmsNormQuant(desc, partial, stream, self.norm[layer][0], out, q, scales, None, self.comm)
        return q, scales, out


def train(ranks: int = 4, layers: int = 3, hidden: int = 512, ffn: int = 2048, rows: int = 256, steps: int = 20):
    """Fits a fixed random target; returns the loss of every step."""
    comm = V.vcommInit(ranks)
    try:
        block = Block(comm, layers, hidden, ffn)
        block.prepare_training(rows)
        gen = torch.Generator().manual_seed(1)
        x = torch.randn(rows, hidden, generator=gen).to(block.dtype).cuda()
        target = torch.randn(rows, hidden, generator=gen).to(block.dtype).cuda()
        losses = []
        for _ in range(steps):
            normed, kept = block.forward(x)
            diff = normed[0].float() - target.float()
            losses.append(diff.square().mean())
            block.backward(kept, (diff * (2 / diff.numel())).to(block.dtype))
            block.step(rate=0.5, max_norm=1.0)
        losses = [v.item() for v in losses]

        # one token through the first layer, its normed input in 8 bits
        token = x[:1].contiguous()
        zeros = [torch.zeros_like(token) for _ in range(ranks - 1)]
        q, scales, stream = block.decode_quantised([token] + zeros, None, 0)
        value = q[0].float() * scales[0].repeat_interleave(128, 1)[:, :hidden]
        plain = token.float() * (token.float().square().mean() + EPS).rsqrt() * block.norm[0][0]
        error = ((value - plain).norm() / plain.norm()).item()
        return losses, error
    finally:
        V.vcommDestroy(comm)


if __name__ == "__main__":
    losses, error = train()
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    print(f"one token in 8 bits: {100 * error:.1f} % off its normed input")
