"""The tensor-parallel example: its hand-written step has autograd's gradients, and it learns."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("tensor_parallel_step",
                                                  os.path.join(ROOT, "examples", "tensor_parallel_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ranks,hidden,rows", [(1, 64, 8), (4, 96, 33), (2, 100, 5)])
def test_gradients_equal_autograd(ranks, hidden, rows):
    ex = load_example()
    comm = V.vcommInit(ranks)
    try:
        block = ex.Block(comm, 2, hidden, 8 * ranks * 4, dtype=torch.float32, seed=3)
        block.prepare_training(rows)
        gen = torch.Generator().manual_seed(4)
        x = torch.randn(rows, hidden, generator=gen).cuda()
        a = torch.randn(rows, hidden, generator=gen).cuda()
        before = torch.backends.cuda.matmul.allow_tf32
        torch.backends.cuda.matmul.allow_tf32 = False
        normed, kept = block.forward(x)
        d_x = block.backward(kept, a)
        torch.backends.cuda.matmul.allow_tf32 = before

        # the same stack whole, in 64 bits
        up = [torch.cat([m.double() for m in ms], 1).requires_grad_() for ms in block.up]
        down = [torch.cat([m.double() for m in ms], 0).requires_grad_() for ms in block.down]
        norm = [w[0].double().requires_grad_() for w in block.norm]
        x64 = x.double().requires_grad_()
        stream = x64
        for layer in range(3):
            y = stream * (stream.square().mean(1, keepdim=True) + ex.EPS).rsqrt() * norm[layer]
            if layer < 2:
                stream = stream + torch.relu(y @ up[layer]) @ down[layer]
        (y * a.double()).sum().backward()

        def near(got, want, what):
            # sums of at most hidden, rows or ffn fp32 terms in a chain of six products
            assert ((got.double() - want).norm() / want.norm()).item() < 2.0 ** -24 * 6 * 128, what

        for r in range(ranks):
            near(normed[r], y.detach(), "output")
        near(d_x, x64.grad, "input")
        for layer in range(2):
            near(torch.cat([block.grads[r][layer] for r in range(ranks)], 1), up[layer].grad, "up")
            near(torch.cat([block.grads[r][2 + layer] for r in range(ranks)], 0), down[layer].grad, "down")
        for layer in range(3):
            near(block.grads[ranks - 1][4 + layer], norm[layer].grad, "norm")
        total = torch.stack([g.square().sum() for g in [*(w.grad for w in up + down), *(w.grad for w in norm)]]).sum().sqrt()
        assert abs(block.step(0.0, 1e9).item() - total.item()) < 2.0 ** -24 * 6 * 128 * total.item()
    finally:
        V.vcommDestroy(comm)


def test_the_example_learns_and_decodes():
    losses, error = load_example().train(steps=12)
    assert losses[-1] < losses[0]
    assert error < 2.0 ** -4                 # half a step of e4m3, relative to the largest in a group
