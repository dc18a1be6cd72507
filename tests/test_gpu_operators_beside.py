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


# ---- sums that are exact --------------------------------------------------------------------

# rows of teams of part of a warp, a warp and a CTA, dealt out unevenly; few rows; rows shared by a
# cluster; (ranks, rows, hidden)
EXACT = [(1, 45000, 64), (1, 44999, 64), (1, 45001, 71), (2, 9001, 200), (2, 3001, 257), (1, 16001, 1024), (3, 2003, 2048),
         (1, 9001, 2047), (8, 1301, 4096), (1, 40, 512), (2, 331, 1001), (1, 401, 32776), (8, 331, 16384), (3, 291, 24001),
         (2, 231, 65536)]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,rows,hidden", EXACT)
def test_the_weight_gradient_of_small_integers_is_exact(n, rows, hidden, dtype, offset):
    # with rstd = 1 every term and every partial sum is a whole number below 2^24, so no row may be
    # missing or counted twice, whatever the order
    gen = torch.Generator().manual_seed(rows + hidden)
    dys = torch.randint(-2, 3, (n, rows, hidden), generator=gen, dtype=torch.int8)
    hid = torch.randint(-3, 4, (rows, hidden), generator=gen, dtype=torch.int8)

    def place(t):
        flat = torch.empty(t.numel() + offset, dtype=dtype, device=DEV)
        flat[offset:].copy_(t.flatten())
        return flat[offset:].view(t.shape)

    comm = V.vcommInit(n)
    try:
        desc = V.vRmsNormDesc(rows, hidden, dtype, F32, EPS)
        space = torch.full((V.vRmsNormBackwardWorkspace(desc, comm),), 0xFF, dtype=torch.uint8, device=DEV)
        dw = torch.full((hidden,), 77.0, device=DEV)
        outs = [None] * (n - 1) + [torch.empty(rows, hidden, dtype=dtype, device=DEV)]
        V.vAllReduceRmsNormBackward(desc, [place(d) for d in dys], place(hid), torch.ones(rows, device=DEV),
                                    torch.ones(hidden, device=DEV), None, outs, dw, space, comm)
        torch.cuda.synchronize()
    finally:
        V.vcommDestroy(comm)
    want = (dys.to(torch.int32).sum(0) * hid.to(torch.int32)).sum(0)
    assert want.abs().max() < 1 << 24
    assert torch.equal(dw.cpu().to(torch.int32), want.to(torch.int32)) and (dw == dw.round()).all()


# ---- in place, and values that are not finite ---------------------------------------------------

# rows that one CTA stages, and rows shared by a cluster, aligned and not
SHARED = [(3, 37, 2048), (2, 3000, 1001), (1, 400, 32776), (8, 330, 16384), (3, 290, 24001), (2, 230, 65536), (64, 90, 4096),
          (40, 161, 2100)]


def make(n, rows, hidden, seed):
    gen = torch.Generator().manual_seed(seed)
    xs = (torch.randn(n, rows, hidden, generator=gen) / n ** 0.5).to(BF16)
    other, more = (torch.randn(rows, hidden, generator=gen).to(BF16) for _ in range(2))
    w = 1 + 0.2 * torch.randn(hidden, generator=gen)
    return xs, other, more, w


@pytest.mark.parametrize("n,rows,hidden", SHARED)
def test_forward_in_place(n, rows, hidden):
    xs, res, _, w = make(n, rows, hidden, 71)
    comm = V.vcommInit(n)
    try:
        send, stream = [x.to(DEV) for x in xs], res.to(DEV)
        V.vAllReduceRmsNorm(V.vRmsNormDesc(rows, hidden, BF16, F32, EPS), send, stream, w.to(DEV), stream, send, None, comm)
        torch.cuda.synchronize()
    finally:
        V.vcommDestroy(comm)
    ref = R.forward(xs, res, w, EPS)
    R.assert_close(stream, ref["h"], ref["dh"], BF16, "stream")
    for r in range(n):
        R.assert_close(send[r], ref["y"], ref["dy"], BF16, f"rank {r}")


@pytest.mark.parametrize("over", ["send", "residual"])
@pytest.mark.parametrize("n,rows,hidden", SHARED)
def test_backward_in_place(n, rows, hidden, over):
    dys, hid, dres, w = make(n, rows, hidden, 72)
    rstd = (hid.float().square().mean(1) + EPS).rsqrt()
    comm = V.vcommInit(n)
    try:
        desc = V.vRmsNormDesc(rows, hidden, BF16, F32, EPS)
        space = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
        send, grad, dw = [d.to(DEV) for d in dys], dres.to(DEV), torch.empty(hidden, device=DEV)
        outs = send if over == "send" else [None] * (n - 1) + [grad]
        V.vAllReduceRmsNormBackward(desc, send, hid.to(DEV), rstd.to(DEV), w.to(DEV), grad, outs, dw, space, comm)
        torch.cuda.synchronize()
    finally:
        V.vcommDestroy(comm)
    ref = R.backward(dys, hid, rstd, w, dres)
    R.assert_close(dw, ref["dw"], ref["ddw"], F32, "weight gradient")
    for o in outs:
        if o is not None:
            R.assert_close(o, ref["dh"], ref["ddh"], BF16, "gradient")


@pytest.mark.parametrize("n,rows,hidden", [(2, 9, 96), (1, 40, 1003), (2, 2700, 1000), (1, 9001, 200), (2, 230, 65536),
                                           (3, 290, 24001)])
def test_backward_rows_with_infinities_and_nans(n, rows, hidden):
    # a bad element spoils its own row of the gradient and its own column of the weight's, no other
    dys, hid, dres, w = make(n, rows, hidden, 73)
    dys[0, 2, hidden // 2] = float("nan")
    dys[n - 1, 4, hidden - 1] = float("inf")
    hid[6, 1] = float("-inf")
    dres[8, 3] = float("nan")
    rstd = (hid.float().square().mean(1) + EPS).rsqrt()      # 0 where the row holds an infinity
    comm = V.vcommInit(n)
    try:
        desc = V.vRmsNormDesc(rows, hidden, BF16, F32, EPS)
        space = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
        outs, dw = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)], torch.empty(hidden, device=DEV)
        V.vAllReduceRmsNormBackward(desc, [d.to(DEV) for d in dys], hid.to(DEV), rstd.to(DEV), w.to(DEV), dres.to(DEV), outs,
                                    dw, space, comm)
        torch.cuda.synchronize()
    finally:
        V.vcommDestroy(comm)
    ref = R.backward(dys, hid, rstd, w, dres)
    for got, want, slack, dtype, what in ((outs[n - 1], ref["dh"], ref["ddh"], BF16, "gradient"),
                                          (dw, ref["dw"], ref["ddw"], F32, "weight gradient")):
        got = got.double().cpu()
        fine = want.isfinite()
        R.assert_close(got[fine], want[fine], slack[fine], dtype, what)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf()), what
    spoilt = ~ref["dh"].isfinite()
    assert spoilt[[2, 4, 6]].all() and spoilt[8].sum() == 1 and not spoilt[[0, 1, 3, 5, 7]].any()
