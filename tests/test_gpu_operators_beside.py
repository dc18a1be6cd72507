"""The operators beside other work: collectives on other streams, other host threads, captures,
and buffers that are input and output at once."""
from __future__ import annotations

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
