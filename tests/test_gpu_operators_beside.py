"""The operators beside other work: collectives on other streams, other host threads, captures,
and buffers that are input and output at once."""
from __future__ import annotations

import threading

import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V
from tests import norm_ref as R
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.mark.parametrize("captured", [False, True])
def test_few_rows_backward_beside_a_long_all_to_all(captured):
    # more backward calls of few rows on one stream than the communicator has pairs of all-to-all
    # counters (64), while one long all-to-all runs on another
    n, block, rows, hidden = 4, 1 << 24, 5, 512
    comm = V.vcommInit(n)
    try:
        gen = torch.Generator().manual_seed(61)
        send = [torch.arange(n * block, dtype=F32, device=DEV).add_(r * 0.25) for r in range(n)]
        recv = [torch.full((n * block,), -7.0, device=DEV) for _ in range(n)]
        counts = torch.full((n, n), block, dtype=torch.int32, device=DEV)
        at = (torch.arange(n, dtype=torch.int32, device=DEV) * block).expand(n, n).contiguous()
        dys = torch.randn(n, rows, hidden, generator=gen).to(BF16)
        hid = torch.randn(rows, hidden, generator=gen).to(BF16)
        rstd = (hid.float().square().mean(1) + EPS).rsqrt()
        w = torch.ones(hidden)
        desc = V.vRmsNormDesc(rows, hidden, BF16, F32, EPS)
        space = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
        args = ([d.to(DEV) for d in dys], hid.to(DEV), rstd.to(DEV), w.to(DEV), None)
        outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
        dws = [torch.full((hidden,), 77.0, device=DEV) for _ in range(150)]
        one, two = torch.cuda.Stream(), torch.cuda.Stream()

        def both():
            here = torch.cuda.current_stream()
            one.wait_stream(here)
            two.wait_stream(here)
            V.vAllToAllv(send, recv, counts, at, at, F32, comm, stream=one)
            for dw in dws:
                V.vAllReduceRmsNormBackward(desc, *args, outs, dw, space, comm, stream=two)
            here.wait_stream(one)
            here.wait_stream(two)

        both()
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                both()
        ref = R.backward(dys, hid, rstd, w, None)
        for _ in range(3):
            for t in recv:
                t.fill_(-7.0)
            for dw in dws:
                dw.fill_(77.0)
            if captured:
                graph.replay()
            else:
                both()
            torch.cuda.synchronize()
            for j in range(n):
                for i in range(n):
                    assert torch.equal(recv[j][i * block:(i + 1) * block], send[i][j * block:(j + 1) * block]), (i, j)
            R.assert_close(dws[0], ref["dw"], ref["ddw"], F32, "weight gradient")
            assert all(torch.equal(dw, dws[0]) for dw in dws)
        assert V.vcommGetAsyncError(comm) == V.vSuccess
    finally:
        torch.cuda.synchronize()
        V.vcommDestroy(comm)


@pytest.mark.parametrize("op", ["norm", "quant", "backward"])
def test_two_host_threads_with_shapes_of_different_shared_memory(op):
    # one instance of the kernel, launched with 40 KiB a CTA by one thread and with twice that by
    # the other, each on its own communicator
    rows, hidden = 3000, 4096
    got = {}

    def work(n):
        torch.cuda.set_device(0)
        comm = V.vcommInit(n)
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                gen = torch.Generator().manual_seed(n)
                xs = torch.randn(n, rows, hidden, generator=gen).to(BF16)
                hid = torch.randn(rows, hidden, generator=gen).to(BF16)
                desc = V.vRmsNormDesc(rows, hidden, BF16, eps=EPS)
                send, recv = xs.to(DEV), torch.empty(n, rows, hidden, dtype=BF16, device=DEV)
                if op == "quant":
                    recv = torch.empty(n, rows, hidden, dtype=torch.uint8, device=DEV)
                sends, recvs = V.vBuffers(send.unbind()), V.vBuffers(recv.unbind())
                scale = torch.empty(n, rows, device=DEV)
                scales = V.vBuffers(scale.unbind())
                w = torch.ones(hidden, dtype=BF16, device=DEV)
                other = hid.to(DEV)
                rstd = (other.float().square().mean(1) + EPS).rsqrt()
                dw = torch.empty(hidden, dtype=BF16, device=DEV)
                space = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
            stream.synchronize()
            for i in range(3000):
                if op == "norm":
                    V.vAllReduceRmsNorm(desc, sends, other, w, None, recvs, None, comm, stream=stream)
                elif op == "quant":
                    V.vAllReduceRmsNormQuant(desc, sends, other, w, None, recvs, scales, None, comm, stream=stream)
                else:
                    V.vAllReduceRmsNormBackward(desc, sends, other, rstd, w, None, recvs, dw, space, comm, stream=stream)
            stream.synchronize()
            first = recv[0].cpu()
            if op == "norm":
                ref = R.forward(xs, hid, w.cpu(), EPS)
                R.assert_close(first, ref["y"], ref["dy"], BF16, "output")
            elif op == "quant":
                R.assert_quantised(first.view(torch.float8_e4m3fn).double(), scale[0].double().cpu()[:, None],
                                   R.forward(xs, hid, w.cpu(), EPS), 0, "output")
            else:
                ref = R.backward(xs, hid, rstd.cpu(), w.cpu(), None)
                R.assert_close(first, ref["dh"], ref["ddh"], BF16, "gradient")
            got[n] = V.vcommGetAsyncError(comm)
        except Exception as e:       # reported below, by the thread that counts
            got[n] = e
        finally:
            torch.cuda.synchronize()
            V.vcommDestroy(comm)

    threads = [threading.Thread(target=work, args=(n,)) for n in (3, 8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got == {3: V.vSuccess, 8: V.vSuccess}


def test_a_list_that_is_lost_while_a_graph_is_captured():
    comm = V.vcommInit(1)
    try:
        grad = torch.full((1000,), 2.0, device=DEV)
        kept = V.vTensorList([[grad]])
        lost = [V.vTensorList([[torch.ones(10, device=DEV)]])]
        space = torch.empty(V.vGradNormWorkspace(kept, comm), dtype=torch.uint8, device=DEV)
        norm = torch.zeros(1, device=DEV)
        V.vGradNorm(kept, norm, space, comm)
        torch.cuda.synchronize()
        norm.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lost.clear()
            V.vGradNorm(kept, norm, space, comm)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(norm.item() - 4000 ** 0.5) <= R.NORM_REL * 1.01 * 4000 ** 0.5
        V.vTensorList([[grad]]).close()
        assert V.vcommGetAsyncError(comm) == V.vSuccess
    finally:
        torch.cuda.synchronize()
        V.vcommDestroy(comm)
