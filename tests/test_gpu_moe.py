"""The experts' router and their layer for a few tokens, against the formulas in 64 bits."""
from __future__ import annotations

import time

import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V
from tests import moe_ref as M
from tests import norm_ref as R
from tests.gpu_util import DEV
from tests.test_gpu_norm import BF16, CANARY, F16, F32, check_outside, place, rows_buffer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def comms():
    made = {}

    def get(n):
        if n not in made:
            made[n] = V.vcommInit(n)
        return made[n]

    yield get
    for c in made.values():
        V.vcommDestroy(c)


# ---- the router ----------------------------------------------------------------------------

def choose(logits, bias, k, normalize):
    """ids and weights from 64-bit logits; ties to the lower index, NaN last."""
    score = logits if bias is None else logits + bias.double()
    key = torch.where(score.isnan(), -float("inf"), score)
    ids = torch.empty(logits.shape[0], k, dtype=torch.int64)
    for t in range(logits.shape[0]):
        order = sorted(range(logits.shape[1]), key=lambda e: (bool(score[t, e].isnan()), -float(key[t, e]), e))
        ids[t] = torch.tensor(order[:k])
    chosen = logits.gather(1, ids)
    top = chosen.amax(1, keepdim=True)
    total = ((chosen if normalize else logits) - top).exp().sum(1, keepdim=True)
    return ids, (chosen - top).exp() / total


def run_route(comm, rows, hidden, experts, k, dtype, wtype, seed, normalize=True, bias=False, pad=0, offset=0, x=None, w=None):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, hidden, generator=gen).to(dtype) if x is None else x
    w = (torch.randn(experts, hidden, generator=gen) * hidden ** -0.5).to(wtype) if w is None else w
    b = torch.randn(experts, generator=gen) * 0.2 if bias else None
    _, dx = rows_buffer(rows, hidden, dtype, hidden + pad, offset)
    dx.copy_(x)
    ids = torch.full((rows * k + 4,), -7, dtype=torch.int32, device=DEV)
    weights = torch.full((rows * k + 4,), CANARY, device=DEV)
    desc = V.vMoeDesc(rows, hidden, 8, experts, k, dtype, wtype, normalize, hidden + pad)
    V.vMoeRoute(desc, dx, place(w, offset), None if b is None else place(b), ids, weights, comm)
    torch.cuda.synchronize()
    logits = x.double() @ w.double().t()
    want, share = choose(logits, b, k, normalize)
    assert torch.equal(ids[:rows * k].cpu().view(rows, k).long(), want)
    # the logits are rounded to fp32 as differences, exp and the quotient add a few u each.  The logits
    # that no choice hangs on are sums of up to 32 products in two fp32 chains: 17 roundings a product,
    # so up to 17 u of the products' magnitudes off, which add up to at most |x| |w|; a weight depends on
    # its own logit and on those that it is a share of.  (The first version of this bound left that out:
    # with logits of 20, sums of 64 products of 1 and more, it allowed 30 u, where they take up 17 * 64.)
    got = weights[:rows * k].cpu().double().view(rows, k)
    sums = 2 * 17 * x.double().norm(dim=1, keepdim=True) * w.double().norm(dim=1).max()
    slack = share * R.U32 * (16 + 2 * (logits.gather(1, want) - logits.amax(1, keepdim=True)).abs() + sums)
    assert ((got - share).abs() <= slack + 1e-38).all()
    assert (ids[rows * k:] == -7).all() and (weights[rows * k:] == CANARY).all()


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("rows,hidden,experts,k", [(1, 8, 1, 1), (1, 4096, 64, 4), (2, 100, 7, 7), (3, 33, 9, 2), (5, 256, 65, 6),
                                                   (8, 64, 8, 8), (9, 1000, 128, 8), (64, 2048, 256, 8), (17, 1, 40, 3),
                                                   (250, 513, 31, 5), (3, 64, 1024, 32), (1024, 40, 16, 2)])
def test_route(comms, rows, hidden, experts, k, dtype, wtype):
    run_route(comms(1), rows, hidden, experts, k, dtype, wtype, seed=hidden + experts)
    run_route(comms(2), rows, hidden, experts, k, dtype, wtype, seed=hidden, normalize=False, bias=True)


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,hidden,experts,k", [(5, 264, 128, 8), (7, 130, 100, 3), (64, 96, 60, 4), (77, 96, 60, 4), (9, 512, 129, 4),
                                                   (64, 256, 256, 8), (80, 250, 200, 5), (700, 96, 20, 3), (1024, 72, 33, 2)])
def test_route_of_a_warp_an_expert_and_of_tiles(comms, rows, hidden, experts, k, dtype, wtype):
    run_route(comms(1), rows, hidden, experts, k, dtype, wtype, seed=rows + hidden, bias=rows % 2 == 1)


@pytest.mark.parametrize("kw", [dict(pad=3), dict(offset=1), dict(pad=8), dict(pad=5, offset=3)])
@pytest.mark.parametrize("hidden", [64, 250])
def test_route_strides_and_offsets(comms, hidden, kw):
    for dtype in (BF16, F32):
        run_route(comms(1), 11, hidden, 20, 4, dtype, F32, 5, **kw)


def test_route_ties_go_to_the_lower_index(comms):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(9, 64, generator=gen).to(BF16)
    x[4] = 0                                          # every score the same
    w = torch.randn(48, 64, generator=gen).to(BF16)
    w[30] = w[5]
    w[31] = w[5]
    w[2] = w[40]
    run_route(comms(1), 9, 64, 48, 12, BF16, BF16, 0, x=x, w=w)
    run_route(comms(1), 9, 64, 48, 12, BF16, BF16, 0, normalize=False, x=x, w=w)


@pytest.mark.parametrize("hidden", [512, 4096])
def test_route_tells_neighbouring_scores_apart(comms, hidden):
    # experts in pairs whose logits differ by some 10^-7 of themselves, less than an fp32 sum's error
    gen = torch.Generator().manual_seed(hidden)
    x = torch.randn(16, hidden, generator=gen).to(BF16)
    w = torch.randn(64, hidden, generator=gen) * hidden ** -0.5
    w[1::2] = w[::2]
    w[1::2, 7] += 2.0 ** -20 * torch.randn(32, generator=gen)
    run_route(comms(1), 16, hidden, 64, 8, BF16, F32, 0, x=x, w=w)


def test_route_values_that_are_not_finite(comms):
    gen = torch.Generator().manual_seed(3)
    rows, hidden, experts, k = 6, 32, 20, 4
    x = torch.randn(rows, hidden, generator=gen)
    w = torch.randn(experts, hidden, generator=gen)
    x[1, 5] = float("nan")                            # no score: the first k experts
    w[6, 0] = float("nan")                            # an expert that nobody chooses
    w[9, 1] = float("inf")
    ids = torch.empty(rows, k, dtype=torch.int32, device=DEV)
    weights = torch.empty(rows, k, device=DEV)
    V.vMoeRoute(V.vMoeDesc(rows, hidden, 8, experts, k, F32), place(x), place(w), None, ids, weights, comms(1))
    want, share = choose(x.double() @ w.double().t(), None, k, True)
    assert torch.equal(ids.cpu().long(), want)
    assert torch.isnan(weights[1]).all() and ids[1].tolist() == [0, 1, 2, 3]
    low = [t for t in range(rows) if t != 1 and x[t, 1] < 0]     # there expert 9 has minus infinity
    assert low and torch.allclose(weights.cpu()[low].double(), share[low], rtol=1e-5)


# ---- the experts -----------------------------------------------------------------------------

def make(ranks, rows, hidden, ffn, experts, k, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, hidden, generator=gen).to(dtype)
    ids = torch.stack([torch.randperm(experts, generator=gen)[:k] for _ in range(rows)]).to(torch.int32)
    weights = torch.rand(rows, k, generator=gen)
    up = [(torch.randn(len(M.held(experts, ranks, r)), 2 * ffn, hidden, generator=gen) * hidden ** -0.5).to(dtype) for r in range(ranks)]
    down = [(torch.randn(len(M.held(experts, ranks, r)), hidden, ffn, generator=gen) * ffn ** -0.5).to(dtype) for r in range(ranks)]
    return x, ids, weights, up, down


def run_experts(comm, x, ids, weights, up, down, pad=0, recv_pad=0, offset=0, weight_offset=0, recv_offset=0):
    ranks, (rows, hidden), k, dtype = len(up), x.shape, ids.shape[1], x.dtype
    ffn = down[0].shape[2]
    experts = sum(u.shape[0] for u in up)
    desc = V.vMoeDesc(rows, hidden, ffn, experts, k, dtype, row_stride=hidden + pad, recv_stride=hidden + recv_pad)
    _, dx = rows_buffer(rows, hidden, dtype, hidden + pad, offset)
    dx.copy_(x)
    outs = [rows_buffer(rows, hidden, dtype, hidden + recv_pad, recv_offset, CANARY) for _ in range(ranks)]
    need = V.vMoeExpertsWorkspace(desc, comm)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)      # NaNs, and a canary behind
    dup, ddown = ([place(t, weight_offset) if t.numel() else None for t in ts] for ts in (up, down))
    V.vMoeExperts(desc, dx, place(ids), place(weights), dup, ddown, [o[1] for o in outs], (ws.data_ptr(), need), comm)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xFF).all(), "written behind the workspace"
    want, slack = M.layer(x, ids.long(), weights, up, down)
    for r, o in enumerate(outs):
        R.assert_close(o[1], want[r], slack[r], dtype, f"rank {r}")
        check_outside(*o, CANARY, f"rank {r}: written outside its rows")


# (ranks, tokens, hidden, ffn, experts, topk): one of everything, odd sizes, ranks without experts,
# widths around the tiles' and steps' sizes, many tokens on few experts
CASES = [(1, 1, 8, 8, 1, 1), (1, 1, 1, 1, 2, 2), (1, 1, 64, 32, 4, 2), (3, 13, 100, 36, 10, 3), (2, 7, 33, 17, 5, 2),
         (8, 5, 64, 48, 3, 2), (4, 1, 2048, 1024, 16, 4), (4, 64, 256, 128, 16, 4), (8, 33, 1024, 512, 64, 8),
         (2, 16, 136, 72, 6, 3), (1, 17, 264, 200, 3, 1), (2, 48, 120, 56, 4, 4), (1, 200, 128, 64, 2, 2),
         (3, 70, 1032, 328, 7, 2), (2, 130, 520, 136, 4, 2), (64, 9, 64, 64, 100, 8), (1, 1024, 72, 40, 8, 3),
         (2, 3, 4104, 2056, 5, 2)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("ranks,rows,hidden,ffn,experts,k", CASES)
def test_experts(comms, ranks, rows, hidden, ffn, experts, k, dtype):
    run_experts(comms(ranks), *make(ranks, rows, hidden, ffn, experts, k, dtype, hidden + rows))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [dict(pad=3), dict(pad=8), dict(recv_pad=5), dict(offset=1), dict(weight_offset=1),
                                dict(recv_offset=3), dict(pad=1, recv_pad=2, offset=3, weight_offset=5, recv_offset=1)])
@pytest.mark.parametrize("rows,hidden,ffn", [(1, 256, 128), (21, 256, 128), (6, 130, 70)])
def test_experts_strides_and_offsets(comms, rows, hidden, ffn, dtype, kw):
    run_experts(comms(2), *make(2, rows, hidden, ffn, 9, 3, dtype, 7), **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hidden,ffn", [(128, 64), (130, 63)])
def test_padding_repeats_and_crowds(comms, hidden, ffn, dtype):
    # ids that are no expert, tokens of none, an expert named twice, all tokens on one expert, no expert at all
    x, ids, weights, up, down = make(3, 90, hidden, ffn, 8, 4, dtype, 11)
    ids[3] = -1
    ids[5, 1:] = 8
    ids[6, 0] = 1 << 30
    ids[7, 2] = -(1 << 31)
    ids[9] = ids[9, 0]
    ids[10, 3] = ids[10, 1]
    run_experts(comms(3), x, ids, weights, up, down)
    run_experts(comms(3), x, torch.full_like(ids, 6), weights, up, down)
    run_experts(comms(3), x, torch.full_like(ids, -1), weights, up, down)
    run_experts(comms(3), x[:1], torch.full_like(ids[:1], 8), weights[:1], up, down)


@pytest.mark.parametrize("hidden,ffn", [(128, 64), (131, 65)])
def test_tokens_that_are_not_finite_stay_alone(comms, hidden, ffn):
    x, ids, weights, up, down = make(2, 24, hidden, ffn, 6, 2, BF16, 13)
    x[5, 3], x[11, 0], weights[17, 1] = float("nan"), float("inf"), float("nan")
    desc = V.vMoeDesc(24, hidden, ffn, 6, 2, BF16)
    outs = [torch.empty(24, hidden, dtype=BF16, device=DEV) for _ in range(2)]
    ws = torch.empty(V.vMoeExpertsWorkspace(desc, comms(2)), dtype=torch.uint8, device=DEV)
    V.vMoeExperts(desc, place(x), place(ids), place(weights), [place(t) for t in up], [place(t) for t in down], outs, ws, comms(2))
    fine = [t for t in range(24) if t not in (5, 11, 17)]
    want, slack = M.layer(x[fine], ids[fine].long(), weights[fine], up, down)
    for r in range(2):
        got = outs[r].cpu()
        R.assert_close(got[fine], want[r], slack[r], BF16, f"rank {r}")
        for t, touched in ((5, (ids[5] // 3 == r).any()), (17, ids[17, 1] // 3 == r)):
            assert torch.isnan(got[t].float()).all() if touched else torch.isfinite(got[t].float()).all()


@pytest.mark.parametrize("ranks,rows,hidden,ffn,experts,k", [(2, 1024, 64, 64, 16, 8), (1, 1024, 72, 40, 64, 32), (3, 700, 64, 32, 1000, 20),
                                                             (1, 1001, 40, 24, 32, 32), (2, 500, 64, 64, 1024, 1)])
def test_many_slots(comms, ranks, rows, hidden, ffn, experts, k):
    run_experts(comms(ranks), *make(ranks, rows, hidden, ffn, experts, k, BF16, seed=rows + k))


@pytest.mark.parametrize("ffn", [64, 63])
@pytest.mark.parametrize("dtype,scale", [(F16, 300.0), (BF16, 1e18)])
def test_inner_values_near_the_end_of_the_type(comms, ffn, dtype, scale):
    # silu(g) u of 50,000 to 130,000 (fp16: largest value 65504, twice that at most), or to 1.4e36
    gen = torch.Generator().manual_seed(91)
    rows, hidden, experts = 5, 64, 2
    x = torch.full((rows, hidden), 16.0).to(dtype)
    one = scale * (0.75 + 0.43 * torch.rand(experts, 2 * ffn, 1, generator=gen)) / (16 * hidden)
    up = one.expand(-1, -1, hidden).to(dtype)
    down = (torch.randn(experts, hidden, ffn, generator=gen) * 2.0 ** -12 / scale).to(dtype)
    ids, weights = torch.tensor([[0], [1], [0], [1], [1]], dtype=torch.int32), torch.ones(rows, 1)
    desc = V.vMoeDesc(rows, hidden, ffn, experts, 1, dtype)
    out = torch.empty(rows, hidden, dtype=dtype, device=DEV)
    ws = torch.empty(V.vMoeExpertsWorkspace(desc, comms(1)), dtype=torch.uint8, device=DEV)
    V.vMoeExperts(desc, place(x), place(ids), place(weights), [place(up)], [place(down)], [out], ws, comms(1))
    want, slack = M.layer(x, ids.long(), weights, [up], [down])
    # the second of two fp16 values is below 65504, so off by half a step of 2^-11 of that at most: 16, and
    # the values are above 2^16
    wide = (x.double()[:, None] @ up[ids[:, 0].long()].double().transpose(1, 2))[:, 0]
    a = wide[:, :ffn] / (1 + (-wide[:, :ffn]).exp()) * wide[:, ffn:]
    more = 2.0 ** -12 * (a[:, None] * down[ids[:, 0].long()].double().abs()).sum(2) if dtype == F16 else 0
    R.assert_close(out, want[0], slack[0] + more, dtype, "output")
    # beyond: with fp16 infinite (aligned rows), and what comes of it is not finite
    if dtype == F16 and ffn == 64:
        V.vMoeExperts(desc, place(x * 2), place(ids), place(weights), [place(up)], [place(down.abs())], [out], ws, comms(1))
        assert not out.isfinite().any()


def test_the_same_bits_again(comms):
    for hidden, ffn in ((1024, 256), (1001, 255)):
        x, ids, weights, up, down = make(4, 40, hidden, ffn, 12, 4, BF16, 15)
        args = (place(x), place(ids), place(weights), [place(t) for t in up], [place(t) for t in down])
        desc = V.vMoeDesc(40, hidden, ffn, 12, 4, BF16)
        got = []
        for _ in range(4):
            outs = torch.empty(4, 40, hidden, dtype=BF16, device=DEV)
            ws = torch.empty(V.vMoeExpertsWorkspace(desc, comms(4)), dtype=torch.uint8, device=DEV)
            V.vMoeExperts(desc, *args, list(outs), ws, comms(4))
            got.append(outs)
        assert all(torch.equal(g, got[0]) for g in got)


@pytest.mark.parametrize("hidden,ffn", [(512, 256), (500, 251)])
def test_streams_a_group_and_a_graph(comms, hidden, ffn):
    # router and experts one behind the other, on two streams at once, grouped, and replayed on new tokens
    ranks, rows, experts, k = 2, 20, 10, 3
    comm = comms(ranks)
    x, _, _, up, down = make(ranks, rows, hidden, ffn, experts, k, BF16, 17)
    gen = torch.Generator().manual_seed(18)
    router = (torch.randn(experts, hidden, generator=gen) * hidden ** -0.5).to(BF16)
    desc = V.vMoeDesc(rows, hidden, ffn, experts, k, BF16)
    drouter, dup, ddown = place(router), [place(t) for t in up], [place(t) for t in down]

    class Run:
        def __init__(self, x):
            self.x = x
            self.dx = place(x)
            self.ids = torch.zeros(rows, k, dtype=torch.int32, device=DEV)
            self.weights = torch.zeros(rows, k, device=DEV)
            self.outs = [torch.zeros(rows, hidden, dtype=BF16, device=DEV) for _ in range(ranks)]
            self.ws = torch.empty(V.vMoeExpertsWorkspace(desc, comm), dtype=torch.uint8, device=DEV)

        def go(self, stream=None):
            V.vMoeRoute(desc, self.dx, drouter, None, self.ids, self.weights, comm, stream=stream)
            V.vMoeExperts(desc, self.dx, self.ids, self.weights, dup, ddown, self.outs, self.ws, comm, stream=stream)

        def check(self):
            torch.cuda.synchronize()
            ids, _ = choose(self.x.double() @ router.double().t(), None, k, True)
            assert torch.equal(self.ids.cpu().long(), ids)
            want, slack = M.layer(self.x, ids, self.weights.cpu(), up, down)
            for r in range(ranks):
                R.assert_close(self.outs[r], want[r], slack[r], BF16, f"rank {r}")

    both = [(Run(x), torch.cuda.Stream()), (Run(x.flip(0)), torch.cuda.Stream())]
    torch.cuda.synchronize()
    for _ in range(3):
        for run, side in both:
            run.go(side)
    for run, _ in both:
        run.check()
    run = Run(x.flip(1))
    V.vcommGroupStart(comm)
    run.go()
    torch.cuda.synchronize()
    assert (run.outs[0] == 0).all()                   # recorded, not run
    V.vcommGroupEnd(comm)
    run.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.go()
    for seed in range(3):
        run.x = torch.randn(rows, hidden, generator=gen).to(BF16)
        run.dx.copy_(run.x)
        graph.replay()
        run.check()


def test_refusals(comms):
    comm = comms(2)
    rows, hidden, ffn, experts, k = 4, 64, 32, 6, 2
    buf = [torch.full((rows, hidden), CANARY, dtype=BF16, device=DEV) for _ in range(3)]
    w = torch.zeros(experts, 2 * ffn, hidden, dtype=BF16, device=DEV)
    ids, weights = torch.zeros(rows, k, dtype=torch.int32, device=DEV), torch.zeros(rows, k, device=DEV)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    good = dict(rows=rows, hidden=hidden, ffn=ffn, experts=experts, top_k=k, datatype=BF16)

    def refused(call, *args):
        with pytest.raises(V.VcommError) as e:
            call(*args)
        assert e.value.code == V.vInvalidArgument

    for change in (dict(rows=1025), dict(hidden=65537), dict(ffn=65537), dict(experts=0), dict(experts=1025), dict(top_k=0),
                   dict(top_k=7), dict(experts=64, top_k=33), dict(datatype=torch.int32), dict(router_type=F16),
                   dict(row_stride=63), dict(recv_stride=1), dict(recv_stride=1 << 62)):
        d = V.vMoeDesc(**{**good, **change})
        refused(V.vMoeRoute, d, buf[0], w, None, ids, weights, comm)
        refused(V.vMoeExpertsWorkspace, d, comm)
        refused(V.vMoeExperts, d, buf[0], ids, weights, [w, w], [w, w], buf[1:], ws, comm)
    for change in (dict(hidden=0), dict(ffn=0)):
        d = V.vMoeDesc(**{**good, **change})
        if change.get("hidden") == 0:
            refused(V.vMoeRoute, d, buf[0], w, None, ids, weights, comm)
        else:
            refused(V.vMoeExperts, d, buf[0], ids, weights, [w, w], [w, w], buf[1:], ws, comm)
    d = V.vMoeDesc(**good)
    odd = buf[0].data_ptr() + 1
    fine = [buf[0], w, None, ids, weights]
    for i, value in [(0, None), (0, odd), (1, None), (1, odd), (2, odd), (3, None), (3, odd), (4, None), (4, odd)]:
        refused(V.vMoeRoute, d, *fine[:i], value, *fine[i + 1:], comm)
    need = V.vMoeExpertsWorkspace(d, comm)
    fine = [buf[0], ids, weights, [w, w], [w, w], buf[1:], ws]
    for i, value in [(0, None), (0, odd), (1, None), (1, odd), (2, None), (2, odd), (3, [None, w]), (3, [w, odd]), (3, [w]),
                     (4, [w, None]), (4, [odd, w]), (5, [None, buf[1]]), (5, [buf[1], odd]), (6, (None, 1 << 20)),
                     (6, (ws.data_ptr(), need - 1)), (6, (ws.data_ptr() + 4, 1 << 19))]:
        refused(V.vMoeExperts, d, *fine[:i], value, *fine[i + 1:], comm)
    zero = V.vMoeDesc(**{**good, "rows": 0})
    V.vMoeRoute(zero, None, None, None, None, None, comm)
    V.vMoeExperts(zero, None, None, None, [None] * 2, [None] * 2, [None] * 2, (None, 0), comm)
    torch.cuda.synchronize()
    assert all((b == CANARY).all() for b in buf) and V.vcommGetAsyncError(comm) == V.vSuccess
    V.vcommGroupStart(comm)
    V.vMoeExperts(d, None, ids, weights, [w, w], [w, w], buf[1:], ws, comm)
    refused(V.vcommGroupEnd, comm)


@pytest.mark.parametrize("inner", [1e-3, 1e-5, 1e-6, 1e-8])
@pytest.mark.parametrize("rows,ffn", [(5, 1024), (5, 1023), (40, 600), (200, 1024), (200, 333)])
def test_small_inner_values_of_fp16(comms, monkeypatch, rows, ffn, inner):
    # silu(g) u far below what steps of 2^-24 resolve, under down weights around 1: held to 2^-22 of itself, or to
    # 2^-35 (the second of the two values in units of 2^-10, its smallest step 2^-24, half of it lost)
    monkeypatch.setitem(M.SPLIT, F16, (2.0 ** -22, 2.0 ** -35))
    x, ids, weights, up, _ = make(2, rows, 64, ffn, 2, 1, F16, 101)
    gen = torch.Generator().manual_seed(102)
    down = [torch.randn(1, 64, ffn, generator=gen).to(F16) for _ in range(2)]
    run_experts(comms(2), (x * (2 * inner) ** 0.5).to(F16), ids, weights, up, down)


def neighbours(rows, hidden, experts, seed):
    """Experts in pairs whose logits differ by some 10^-7 of themselves, less than an fp32 sum's error."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, hidden, generator=gen).to(BF16)
    w = torch.randn(experts, hidden, generator=gen) * hidden ** -0.5
    w[1::2] = w[::2]
    w[1::2, 7] += 2.0 ** -20 * torch.randn(experts // 2, generator=gen)
    return x, w


@pytest.mark.parametrize("tokens_by,weights_by", [(1.0, 1.0), (2.0 ** -80, 2.0 ** 54), (2.0 ** 60, 2.0 ** -80), (2.0 ** 70, 2.0 ** -70)])
@pytest.mark.parametrize("rows,hidden,experts", [(16, 512, 64), (200, 1024, 64), (200, 600, 130)])
def test_route_tells_neighbouring_scores_apart_at_any_scale(comms, rows, hidden, experts, tokens_by, weights_by):
    # squares of the tokens or of the weights below fp32's smallest value, or above its largest
    x, w = neighbours(rows, hidden, experts, hidden)
    run_route(comms(1), rows, hidden, experts, 8, BF16, F32, 0, x=x * tokens_by, w=w * weights_by)


@pytest.mark.parametrize("rows", [3, 200])
def test_route_of_large_tokens_by_experts_of_zeros(comms, rows):
    # one expert whose logit is some 2^-25 of its products' magnitudes, all others zero: its sign decides
    hidden, experts = 512, 40
    for seed in range(12):
        gen = torch.Generator().manual_seed(seed)
        x0 = torch.randn(hidden, generator=gen).to(BF16)
        w = torch.zeros(experts, hidden)
        w[17] = torch.randn(hidden, generator=gen)
        for j in range(3):                            # down to the last bit of one weight after another
            w[17, j] -= float(w[17].double() @ x0.double() / x0[j].double())
        run_route(comms(1), rows, hidden, experts, 1, BF16, F32, 0, x=(x0 * 2.0 ** 70).expand(rows, -1), w=w)


@pytest.mark.parametrize("rows,hidden,ffn,experts,k,stall", [(1, 2048, 1024, 16, 4, 0), (1, 2048, 1024, 16, 4, 1), (1, 2048, 1024, 16, 4, 3),
                                                             (4, 33, 17, 5, 2, 0), (64, 512, 256, 8, 4, 2), (300, 500, 250, 4, 2, 1)])
def test_a_wait_that_runs_out_ends_the_call_with_an_error(comms, rows, hidden, ffn, experts, k, stall):
    # one CTA of both launches gets nothing to multiply: its waits, and those of the others that wait for it,
    # give up after the communicator's limit, and the call is over
    args = make(4, rows, hidden, ffn, experts, k, BF16, 21)
    x, ids, weights = (place(t) for t in args[:3])
    up, down = ([place(t) for t in ts] for ts in args[3:])
    desc = V.vMoeDesc(rows, hidden, ffn, experts, k, BF16)
    outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(4)]
    comm = V.vcommInit(4)
    try:
        V.vcommSetTimeoutMs(comm, 100)
        V.vcommTestSetStallRank(comm, stall)
        ws = torch.empty(V.vMoeExpertsWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        V.vMoeExperts(desc, x, ids, weights, up, down, outs, ws, comm)
        torch.cuda.synchronize()
        # in each launch the stalled CTA's, then that of a CTA that waits for its sums
        assert 0.1 <= time.perf_counter() - t0 < 1.0
        assert V.vcommGetAsyncError(comm) == V.vTimeout
        with pytest.raises(V.VcommError) as e:
            V.vMoeExperts(desc, x, ids, weights, up, down, outs, ws, comm)
        assert e.value.code == V.vTimeout
    finally:
        V.vcommDestroy(comm)
    # the context and the tensor cores are as usable as before
    run_experts(comms(4), *args)


@pytest.mark.parametrize("hidden,ffn", [(65536, 64), (65535, 63), (72, 65536), (71, 65535)])
def test_the_shortest_limit_is_long_enough_for_the_longest_rows(hidden, ffn):
    # a tile's 512 stages take up to a millisecond, in which there is progress
    comm = V.vcommInit(1)
    try:
        V.vcommSetTimeoutMs(comm, 1)
        args = make(1, 70, hidden, ffn, 2, 1, BF16, 31)
        for _ in range(3):
            run_experts(comm, *args)
        assert V.vcommGetAsyncError(comm) == V.vSuccess
    finally:
        V.vcommDestroy(comm)
