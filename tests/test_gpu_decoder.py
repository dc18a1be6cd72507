"""The operators together, as a decoder and a training step use them: every operator's results against
its formula in 64 bits from the inputs that it was given, eager, captured, and without early launches."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V
from tests import block_ref as B
from tests import moe_ref as M
from tests import norm_ref as R
from tests import sample_ref as S
from tests.test_gpu_moe import choose

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("experts_decoder", os.path.join(ROOT, "examples", "experts_decoder.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def cpu(v):
    return [cpu(t) for t in v] if isinstance(v, list) else v.detach().cpu().clone()


@pytest.mark.parametrize("pdl", ["1", "0"])
@pytest.mark.parametrize("ranks,rows,hidden,ffn,experts,vocab,dtype", [(1, 1, 64, 40, 5, 100, BF16), (4, 3, 256, 128, 9, 1001, BF16),
                                                                       (3, 17, 130, 33, 4, 4000, F16), (2, 70, 512, 256, 16, 5000, BF16),
                                                                       (8, 2, 100, 30, 6, 37, F32)])
def test_every_operator_of_a_decoding_step(ex, monkeypatch, ranks, rows, hidden, ffn, experts, vocab, dtype, pdl):
    monkeypatch.setenv("VCOMM_PDL", pdl)
    comm = V.vcommInit(ranks)
    try:
        model = ex.Decoder(comm, rows, 2, hidden, ffn, experts, 3, vocab, dtype, scale=0.9, seed=11)
        gen = torch.Generator().manual_seed(12)
        for t in model.tokens:
            t.copy_(torch.arange(rows) % vocab)
        model.uniform.copy_(torch.rand(rows, generator=gen))
        heat = (0.5 + torch.rand(rows, generator=gen)).cuda()
        top_k = torch.randint(0, 40, (rows,), generator=gen, dtype=torch.int32).cuda()
        top_p = (0.5 + torch.rand(rows, generator=gen)).cuda()
        start = [t.clone() for t in model.tokens]
        log = []
        model.step(heat, top_k, top_p, seen=lambda name, *v: log.append((name, [x if isinstance(x, int) else cpu(x) for x in v])))
        assert [name for name, _ in log] == ["route", "experts", "norm"] * 2 + ["sample"]
        for name, v in log:
            if name == "route":
                layer, x, ids, _ = v
                want, _ = choose(x.double() @ model.router[layer].cpu().double().t(), None, 3, True)
                assert torch.equal(ids.long(), want)
            elif name == "experts":
                layer, x, ids, weights, partial, before = v
                none = [torch.empty(0, 2 * ffn, hidden), torch.empty(0, hidden, ffn)]
                up, down = ([none[i] if t is None else t.cpu() for t in ts] for i, ts in enumerate((model.up[layer], model.down[layer])))
                want, slack = M.layer(x, ids.long(), weights, up, down)
                for r in range(ranks):
                    R.assert_close(partial[r], want[r], slack[r], dtype, f"layer {layer} rank {r}")
            elif name == "norm":
                layer, stream, normed = v
                post, gate, pre = (w.cpu() for w in model.norms[layer].weights())
                ref = B.forward(torch.stack(partial), before, post, gate, pre, float(np.float32(0.9)), float(np.float32(ex.EPS)))
                R.assert_close(stream, ref["h"], ref["dh"], dtype, "stream")
                for y in normed:
                    R.assert_close(y, ref["y"], ref["dy"], dtype, "normed")
            else:
                logits, uniform, tokens, _ = v
                whole = torch.cat(logits, 1)[:, :vocab].float().numpy()
                for t in range(rows):
                    assert S.matches(int(tokens[0][t]), whole[t], float(uniform[t]), temperature=float(heat[t]),
                                     top_k=int(top_k[t]), top_p=float(top_p[t]))
                assert all(torch.equal(t, tokens[0]) for t in tokens)
        # a captured step, replayed twice from the same tokens, gives the same bits
        want, share, stream = cpu(model.tokens), cpu(model.logprob), cpu(model.stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            model.step(heat, top_k, top_p)
        for _ in range(2):
            for t, s in zip(model.tokens, start):
                t.copy_(s)
            model.logprob.fill_(-77)
            model.stream.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(cpu(model.tokens), want))
            assert torch.equal(cpu(model.logprob), share) and torch.equal(cpu(model.stream), stream)
        assert V.vcommGetAsyncError(comm) == V.vSuccess
    finally:
        torch.cuda.synchronize()
        V.vcommDestroy(comm)


def test_two_decoders_at_once(ex):
    # one communicator, two streams, each with its own buffers and workspace
    comm = V.vcommInit(4)
    try:
        models = [ex.Decoder(comm, rows, 2, 256, 128, 8, 3, 3001, seed=rows) for rows in (1, 40)]
        streams = [torch.cuda.Stream() for _ in models]
        for m in models:
            m.uniform.fill_(0.4)
        want = []
        for m in models:                              # one behind the other
            for t in m.tokens:
                t.fill_(5)
            for _ in range(6):
                m.step()
            want.append((cpu(m.tokens), cpu(m.stream)))
        for m in models:
            for t in m.tokens:
                t.fill_(5)
        torch.cuda.synchronize()
        for _ in range(6):
            for m, s in zip(models, streams):
                with torch.cuda.stream(s):
                    m.step()
        torch.cuda.synchronize()
        for m, (tokens, stream) in zip(models, want):
            assert all(torch.equal(a, b) for a, b in zip(cpu(m.tokens), tokens)) and torch.equal(cpu(m.stream), stream)
    finally:
        torch.cuda.synchronize()
        V.vcommDestroy(comm)


@pytest.mark.parametrize("ranks,hidden,rows", [(1, 64, 8), (4, 96, 33), (2, 100, 5)])
def test_gradients_equal_autograd(ex, ranks, hidden, rows):
    comm = V.vcommInit(ranks)
    before = torch.backends.cuda.matmul.allow_tf32
    try:
        torch.backends.cuda.matmul.allow_tf32 = False
        block = ex.Block(comm, 2, hidden, 32 * ranks, F32, scale=0.8, seed=3)
        gen = torch.Generator().manual_seed(4)
        x, a = (torch.randn(rows, hidden, generator=gen).cuda() for _ in range(2))
        normed, kept = block.forward(x)
        d_x, d_up, d_down, d_norms = block.backward(kept, a)

        # the same stack whole, in 64 bits
        up = [torch.cat([m.double() for m in ms]).requires_grad_() for ms in block.up]
        down = [torch.cat([m.double() for m in ms], 1).requires_grad_() for ms in block.down]
        norms = [[w.double().requires_grad_() for w in n.weights()] for n in block.norms]
        x64 = x.double().requires_grad_()

        def unit(v):
            return v * (v.square().mean(1, keepdim=True) + ex.EPS).rsqrt()

        stream = y = x64
        for layer, (post, gate, pre) in enumerate(norms):
            stream = 0.8 * stream + gate * post * unit(torch.relu(y @ up[layer].t()) @ down[layer].t())
            y = unit(stream) * pre
        (y * a.double()).sum().backward()

        def near(got, want, what):
            # sums of at most hidden, rows or 32 fp32 terms in a chain of six products, twice for two norms
            assert ((got.double() - want).norm() / want.norm()).item() < 2.0 ** -24 * 12 * 128, what

        for r in range(ranks):
            near(normed[r], y.detach(), "output")
        near(d_x, x64.grad, "input")
        for layer in range(2):
            near(torch.cat(d_up[layer]), up[layer].grad, "up")
            near(torch.cat(d_down[layer], 1), down[layer].grad, "down")
            for got, w, what in zip(d_norms[layer], norms[layer], ("post", "gate", "pre")):
                near(got, w.grad, what)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = before
        torch.cuda.synchronize()
        V.vcommDestroy(comm)


def test_the_example_runs(ex):
    tokens = ex.decode(steps=6)
    assert tokens.shape == (6, 4) and (tokens >= 0).all() and (tokens < 4000).all()
    assert torch.equal(tokens, ex.decode(steps=6))
    assert all(v == v for v in ex.train(steps=2))
