"""Decoding with a mixture of experts and a training step with block norms, over virtual ranks.

A layer of the decoder sends every token to a few of its experts, which are split over N ranks: each
rank ends it with a partial sum.  The next token comes of logits whose vocabulary is split the same way.

  decoding   vMoeRoute                   the normed tokens -> every token's experts and weights
             vMoeExperts                 -> every rank's partial sum
             vAllReduceBlockNorm         -> residual stream, normed input of the next layer on every rank
             vSample                     every rank's columns of the logits -> the next token on every rank
  training   vAllReduceBlockNorm         behind a feed-forward block split over the ranks
             vAllReduceBlockNormBackward partial input gradients -> gradients of the stream, of every
                                         rank's partial sum, of both norms' weights and of the gate

    python examples/experts_decoder.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from collective_communication_virtual_gb300 import vcomm as V  # noqa: E402

EPS = 1e-6


def matrix(gen, *shape, dtype):
    return (torch.randn(*shape, generator=gen) * shape[-1] ** -0.5).to(dtype).cuda()


class Norms:
    """The weights around one block: the norm after it, its gate, the norm before the next one."""

    def __init__(self, gen, hidden):
        self.post, self.gate, self.pre = ((1 + 0.1 * torch.randn(hidden, generator=gen)).cuda() for _ in range(3))

    def weights(self):
        return self.post, self.gate, self.pre


class Decoder:
    """Layers of experts over a batch of sequences, one token of each at a time.  All buffers are made
    once, so that a step can be captured."""

    def __init__(self, comm, rows, layers, hidden, ffn, experts, top_k, vocab, dtype=torch.bfloat16, scale=1.0, seed=0):
        self.comm, self.n = comm, V.vcommCount(comm)
        n, gen = self.n, torch.Generator().manual_seed(seed)
        share = -(-experts // n)
        held = [max(0, min(experts, (r + 1) * share) - r * share) for r in range(n)]
        self.part = -(-vocab // n)
        columns = [max(0, min(vocab, (r + 1) * self.part) - r * self.part) for r in range(n)]
        self.embedding = torch.randn(vocab, hidden, generator=gen).to(dtype).cuda()
        self.router = [matrix(gen, experts, hidden, dtype=torch.float32) for _ in range(layers)]
        self.up = [[matrix(gen, held[r], 2 * ffn, hidden, dtype=dtype) if held[r] else None for r in range(n)] for _ in range(layers)]
        self.down = [[matrix(gen, held[r], hidden, ffn, dtype=dtype) if held[r] else None for r in range(n)] for _ in range(layers)]
        self.norms = [Norms(gen, hidden) for _ in range(layers)]
        self.first = torch.ones(hidden, device="cuda")
        self.head = [matrix(gen, c, hidden, dtype=dtype) for c in columns]

        self.moe = V.vMoeDesc(rows, hidden, ffn, experts, top_k, dtype, torch.float32)
        self.block = V.vBlockNormDesc(rows, hidden, dtype, torch.float32, EPS, scale)
        self.norm = V.vRmsNormDesc(rows, hidden, dtype, torch.float32, EPS)
        self.draw = V.vSampleDesc(rows, vocab, dtype, self.part)

        def empty(*shape, of=dtype):
            return torch.empty(*shape, dtype=of, device="cuda")

        self.stream, self.zero = empty(rows, hidden), torch.zeros(rows, hidden, dtype=dtype, device="cuda")
        self.normed, self.partial = ([empty(rows, hidden) for _ in range(n)] for _ in range(2))
        self.ids, self.weights = empty(rows, top_k, of=torch.int32), empty(rows, top_k, of=torch.float32)
        self.space = empty(V.vMoeExpertsWorkspace(self.moe, comm), of=torch.uint8)
        self.logits = [torch.zeros(rows, self.part, dtype=dtype, device="cuda") for _ in range(n)]
        self.tokens = [empty(rows, of=torch.int32).zero_() for _ in range(n)]
        self.logprob, self.uniform = empty(rows, of=torch.float32), empty(rows, of=torch.float32)

    def step(self, temperature=None, top_k=None, top_p=None, min_p=None, seen=None):
        """self.tokens -> the next ones, by the random numbers in self.uniform.  `seen` is called with a
        name and its buffers behind each operator."""
        seen = seen or (lambda *_: None)
        self.stream.copy_(self.embedding[self.tokens[0].long()])
        # the embedding is no partial sum: rank 0 sends it, the others zeros
        V.vAllReduceRmsNorm(self.norm, [self.stream] + [self.zero] * (self.n - 1), None, self.first, None, self.normed, None, self.comm)
        for layer, norms in enumerate(self.norms):
            x = self.normed[0]
            V.vMoeRoute(self.moe, x, self.router[layer], None, self.ids, self.weights, self.comm)
            seen("route", layer, x, self.ids, self.weights)
            V.vMoeExperts(self.moe, x, self.ids, self.weights, self.up[layer], self.down[layer], self.partial, self.space, self.comm)
            seen("experts", layer, x, self.ids, self.weights, self.partial, self.stream)
            V.vAllReduceBlockNorm(self.block, self.partial, self.stream, *norms.weights(), None, self.stream, self.normed, None,
                                  self.comm)
            seen("norm", layer, self.stream, self.normed)
        for r in range(self.n):
            torch.mm(self.normed[r], self.head[r].t(), out=self.logits[r][:, :self.head[r].shape[0]])
        V.vSample(self.draw, self.logits, temperature, top_k, top_p, min_p, self.uniform, self.tokens, self.logprob, self.comm)
        seen("sample", self.logits, self.uniform, self.tokens, self.logprob)


class Block:
    """Feed-forward blocks split over the ranks with the norms around each, and their backward pass."""

    def __init__(self, comm, layers, hidden, ffn, dtype=torch.bfloat16, scale=1.0, seed=0):
        self.comm, self.n, self.dtype, self.scale = comm, V.vcommCount(comm), dtype, scale
        gen, part = torch.Generator().manual_seed(seed), ffn // self.n
        self.up = [[matrix(gen, part, hidden, dtype=dtype) for _ in range(self.n)] for _ in range(layers)]
        self.down = [[matrix(gen, hidden, part, dtype=dtype) for _ in range(self.n)] for _ in range(layers)]
        self.norms = [Norms(gen, hidden) for _ in range(layers)]

    def forward(self, x):
        """x: the stream, taken as the first block's input as it is.  The last norm's output on every
        rank, and what the backward pass needs."""
        rows, hidden = x.shape
        desc = V.vBlockNormDesc(rows, hidden, self.dtype, torch.float32, EPS, self.scale)
        stream, normed, kept = x, [x] * self.n, []
        for up, down, norms in zip(self.up, self.down, self.norms):
            wide = [normed[r] @ up[r].t() for r in range(self.n)]
            partial = [torch.relu(wide[r]) @ down[r].t() for r in range(self.n)]
            block, out, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(2, rows, device="cuda")
            after = [torch.empty_like(x) for _ in range(self.n)]
            V.vAllReduceBlockNorm(desc, partial, stream, *norms.weights(), block, out, after, rstd, self.comm)
            kept.append((normed, wide, block, out, rstd))
            stream, normed = out, after
        return normed, kept

    def backward(self, kept, d_normed):
        """The gradients of x, of every layer's matrices ([layer][rank]) and of its (post, gate, pre), from
        the last norm's output's gradient."""
        rows, hidden = d_normed.shape
        desc = V.vBlockNormDesc(rows, hidden, self.dtype, torch.float32, EPS, self.scale)
        space = torch.empty(V.vBlockNormBackwardWorkspace(desc, self.comm), dtype=torch.uint8, device="cuda")
        # rank 0 sends the gradient, the others zeros; behind that, each rank its own part
        partial, d_stream = [d_normed] + [torch.zeros_like(d_normed)] * (self.n - 1), None
        d_up, d_down, d_norms = [], [], []
        for up, down, norms, (normed, wide, block, out, rstd) in zip(*(reversed(v) for v in (self.up, self.down, self.norms, kept))):
            d_block, d_residual = torch.empty_like(d_normed), torch.empty_like(d_normed)
            d_weights = [torch.empty(hidden, device="cuda") for _ in range(3)]
            # every rank's partial sum has the same gradient: one copy serves all ranks
            V.vAllReduceBlockNormBackward(desc, partial, out, block, rstd, *norms.weights(), d_stream, d_residual,
                                          [d_block] + [None] * (self.n - 1), *d_weights, space, self.comm)
            d_wide = [(d_block @ down[r]) * (wide[r] > 0) for r in range(self.n)]
            d_down.insert(0, [d_block.t() @ torch.relu(wide[r]) for r in range(self.n)])
            d_up.insert(0, [d_wide[r].t() @ normed[r] for r in range(self.n)])
            d_norms.insert(0, d_weights)
            partial, d_stream = [d_wide[r] @ up[r] for r in range(self.n)], d_residual
        return d_stream + torch.stack(partial).sum(0), d_up, d_down, d_norms


def decode(ranks: int = 4, rows: int = 4, steps: int = 16, layers: int = 3, hidden: int = 512, ffn: int = 256, experts: int = 16,
           vocab: int = 4000):
    """Draws `steps` tokens for every sequence, the step captured in a graph; returns them, [steps, rows]."""
    comm = V.vcommInit(ranks)
    try:
        model = Decoder(comm, rows, layers, hidden, ffn, experts, 4, vocab)
        filters = (torch.full((rows,), 0.8, device="cuda"), torch.full((rows,), 50, dtype=torch.int32, device="cuda"),
                   torch.full((rows,), 0.95, device="cuda"))
        gen = torch.Generator(device="cuda").manual_seed(1)
        drawn = torch.rand(steps, rows, generator=gen, device="cuda")
        model.uniform.copy_(drawn[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            model.step(*filters)                      # once before the capture, for the library's products
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            model.step(*filters)
        for t in model.tokens:
            t.zero_()
        out = torch.empty(steps, rows, dtype=torch.int32, device="cuda")
        for i in range(steps):
            model.uniform.copy_(drawn[i])
            graph.replay()
            out[i].copy_(model.tokens[0])
        return out.cpu()
    finally:
        torch.cuda.synchronize()
        V.vcommDestroy(comm)


def train(ranks: int = 4, rows: int = 256, steps: int = 10, layers: int = 2, hidden: int = 512, ffn: int = 1024):
    """Fits a fixed random target; returns the loss of every step."""
    comm = V.vcommInit(ranks)
    try:
        block = Block(comm, layers, hidden, ffn)
        gen = torch.Generator().manual_seed(2)
        x, target = (torch.randn(rows, hidden, generator=gen).to(block.dtype).cuda() for _ in range(2))
        losses = []
        for _ in range(steps):
            normed, kept = block.forward(x)
            diff = normed[0].float() - target.float()
            losses.append(diff.square().mean())
            _, *grads = block.backward(kept, (diff * (2 / diff.numel())).to(block.dtype))
            for params, ds in zip((block.up, block.down, [n.weights() for n in block.norms]), grads):
                for ps, gs in zip(params, ds):
                    torch._foreach_add_(list(ps), gs, alpha=-0.5)
        return [v.item() for v in losses]
    finally:
        torch.cuda.synchronize()
        V.vcommDestroy(comm)


if __name__ == "__main__":
    print("tokens of the first sequence: " + " ".join(map(str, decode()[:, 0].tolist())))
    print("loss " + " ".join(f"{v:.4f}" for v in train()))
