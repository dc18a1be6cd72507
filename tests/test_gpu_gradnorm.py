"""The global gradient norm and clipping against the formula in 64 bits: many tensors of mixed
types and odd sizes, split and replicated ones, alignments, special values and refusals."""
from __future__ import annotations

import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V
from tests import norm_ref as R
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


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


def packed(sizes, dtypes, gen, scale=1.0, pad=0):
    """Tensors of one rank cut from one buffer per type, one behind the other from element
    `pad` on, so that they start at every alignment; canaries before and behind them."""
    out, flats = [None] * len(sizes), []
    for dt in dict.fromkeys(dtypes):
        mine = [i for i, d in enumerate(dtypes) if d == dt]
        total = sum(sizes[i] for i in mine)
        flat = torch.full((pad + total + 16,), 3.0, dtype=dt, device=DEV)
        if total:
            flat[pad:pad + total] = (torch.randn(total, generator=gen) * scale).to(dt).to(DEV)
        at = pad
        for i in mine:
            out[i] = flat[at:at + sizes[i]]
            at += sizes[i]
        flats.append((flat, pad, at))
    return out, flats


def run(comm, n, sizes, dtypes, replicated, max_norm, seed, scale=1.0, pad=0, out_pad=0, in_place=False):
    gen = torch.Generator().manual_seed(seed)
    ranks = [packed(sizes, dtypes, gen, scale, pad) for _ in range(n)]
    grads = [t for t, _ in ranks]
    for t, rep in enumerate(replicated or []):
        if rep:
            for r in range(1, n):
                grads[r][t].copy_(grads[0][t])
    before = [[t.double().cpu() for t in g] for g in grads]
    counted = [before[r][t] for r in range(n) for t in range(len(sizes)) if r == 0 or not (replicated and replicated[t])]
    want = R.grad_norm(counted).item()
    outs = None if in_place else [packed(sizes, dtypes, gen, scale, out_pad) for _ in range(n)]
    tensors = V.vTensorList(grads, None if in_place else [o for o, _ in outs], replicated)
    need = V.vGradNormWorkspace(tensors, comm)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    norm = torch.full((3,), 5.0, device=DEV)
    V.vGradNorm(tensors, norm, (ws.data_ptr(), need), comm)
    assert abs(norm[0].item() - want) <= R.NORM_REL * 1.01 * want
    norm[0] = -1
    V.vClipGradNorm(tensors, max_norm, norm, (ws.data_ptr(), need), comm)
    torch.cuda.synchronize()
    assert abs(norm[0].item() - want) <= R.NORM_REL * 1.01 * want
    assert (norm[1:] == 5.0).all() and (ws[need:] == 0xFF).all()
    factor = min(1.0, max_norm / (want + 1e-6))
    sides = ranks if in_place else outs
    for r in range(n):
        for t, g in enumerate(before[r]):
            value = g * factor
            R.assert_close(sides[r][0][t], value, R.CLIP_REL * value.abs(), dtypes[t], f"rank {r} tensor {t}")
            if not in_place:
                assert torch.equal(grads[r][t].double().cpu(), g), "a gradient was written"
        for flat, lo, hi in sides[r][1]:
            assert (flat[:lo] == 3.0).all() and (flat[hi:] == 3.0).all(), "written outside the tensors"


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16383, 1, 16385], [0, 5, 0, 9], [100_003, 2, 40_000], [3] * 130])
@pytest.mark.parametrize("in_place", [False, True])
def test_one_type(comms, n, dtype, sizes, in_place):
    run(comms(n), n, sizes, [dtype] * len(sizes), None, 0.5, seed=len(sizes), in_place=in_place)


@pytest.mark.parametrize("pad,out_pad", [(0, 0), (1, 1), (0, 3), (5, 2)])
@pytest.mark.parametrize("max_norm", [1.0, 1e9, 0.0, float("inf")])
def test_mixed_types_replicated_and_offsets(comms, pad, out_pad, max_norm):
    sizes = [4097, 33, 1, 70_000, 512, 8, 32_769, 5]
    dtypes = [BF16, F32, F16, F32, BF16, F32, F16, BF16]
    rep = [False, True, False, False, True, True, False, True]
    run(comms(4), 4, sizes, dtypes, rep, max_norm, seed=pad, pad=pad, out_pad=out_pad)
    run(comms(4), 4, sizes, dtypes, rep, max_norm, seed=pad, pad=pad, in_place=True)


@pytest.mark.parametrize("n,count", [(1, 120), (1, 121), (1, 1000), (1, 1001), (2, 1700), (8, 300)])
def test_many_tensors(comms, n, count):
    gen = torch.Generator().manual_seed(count)
    sizes = torch.randint(0, 90, (count,), generator=gen).tolist()
    dtypes = [(F32, BF16)[i % 2] for i in range(count)]
    run(comms(n), n, sizes, dtypes, [i % 3 == 0 for i in range(count)], 1.0, seed=count)


@pytest.mark.parametrize("total", [1 << 20, (1 << 22) + 13, 30_000_001])
def test_sizes_between_a_few_ctas_and_many_waves(comms, total):
    run(comms(2), 2, [total, total // 3], [BF16, F32], [False, True], 2.0, seed=3, scale=0.1)


def test_a_tensor_past_two_to_the_31_elements(comms):
    count = (1 << 31) + 4099
    g = torch.empty(count, dtype=BF16, device=DEV).normal_(0, 0.01)
    out = torch.empty_like(g)
    tensors = V.vTensorList([[g]], [[out]])
    ws = torch.empty(V.vGradNormWorkspace(tensors, comms(1)), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    V.vClipGradNorm(tensors, 1.0, norm, ws, comms(1))
    want = sum(c.double().square().sum().item() for c in g.split(1 << 28)) ** 0.5
    assert abs(norm.item() - want) <= R.NORM_REL * 1.01 * want
    for at in (0, 1 << 30, count - 5000):
        value = g[at:at + 5000].double() / (want + 1e-6)
        R.assert_close(out[at:at + 5000], value, R.CLIP_REL * value.abs(), BF16, f"at {at}")


def test_values_that_are_not_finite(comms):
    comm = comms(1)
    for bad, kept in ((float("inf"), 0.0), (float("nan"), float("nan"))):
        g = torch.ones(1000, device=DEV)
        g[500] = bad
        tensors = V.vTensorList([[g]])
        ws = torch.empty(V.vGradNormWorkspace(tensors, comm), dtype=torch.uint8, device=DEV)
        norm = torch.empty(1, device=DEV)
        V.vClipGradNorm(tensors, 1.0, norm, ws, comm)
        got = g.cpu()
        assert torch.equal(norm.cpu(), torch.tensor([bad]).abs()) or torch.isnan(norm).item() and bad != bad
        assert torch.isnan(got[500])
        rest = torch.cat([got[:500], got[501:]])
        assert torch.isnan(rest).all() if kept != kept else (rest == 0).all()


def test_no_tensors_is_a_norm_of_zero(comms):
    comm = comms(2)
    empty = torch.empty(0, device=DEV)
    for tensors in (V.TensorList(2, [], [], None, [], None), V.vTensorList([[empty], [empty]])):
        ws = torch.empty(V.vGradNormWorkspace(tensors, comm), dtype=torch.uint8, device=DEV)
        norm = torch.full((1,), 5.0, device=DEV)
        V.vGradNorm(tensors, norm, ws, comm)
        assert norm.item() == 0.0
        norm.fill_(5.0)
        V.vClipGradNorm(tensors, 1.0, norm, ws, comm)
        assert norm.item() == 0.0


@pytest.mark.parametrize("sizes", [[5000, 77], [3_000_000, 500_001]])
def test_the_same_bits_again_in_a_group_and_in_a_graph(comms, sizes):
    n, comm = 2, comms(2)
    gen = torch.Generator().manual_seed(5)
    grads = [packed(sizes, [F32, BF16], gen)[0] for _ in range(n)]
    outs = [packed(sizes, [F32, BF16], gen)[0] for _ in range(n)]
    tensors = V.vTensorList(grads, outs)
    ws = torch.empty(V.vGradNormWorkspace(tensors, comm), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    V.vClipGradNorm(tensors, 1.0, norm, ws, comm)
    first = [norm.clone()] + [t.clone() for o in outs for t in o]

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(x, y) for x, y in zip(first, [norm] + [t for o in outs for t in o]))

    def wipe():
        for o in outs:
            for t in o:
                t.zero_()
        norm.zero_()

    wipe()
    V.vcommGroupStart(comm)
    V.vClipGradNorm(tensors, 1.0, norm, ws, comm)
    torch.cuda.synchronize()
    assert norm.item() == 0.0
    V.vcommGroupEnd(comm)
    assert same()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        V.vClipGradNorm(tensors, 1.0, norm, ws, comm)
    for _ in range(3):
        wipe()
        graph.replay()
        assert same()


def test_clipping_follows_a_reduction_on_the_stream(comms):
    # reduce-scatter, norm and clipping launched without waits: each sees the one before
    n, count = 4, 100_000
    comm = comms(n)
    gen = torch.Generator().manual_seed(9)
    xs = [torch.randn(n * count, generator=gen) for _ in range(n)]
    send = [x.to(DEV) for x in xs]
    shard = [torch.zeros(count, device=DEV) for _ in range(n)]
    tensors = V.vTensorList([[s] for s in shard])
    ws = torch.empty(V.vGradNormWorkspace(tensors, comm), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    torch.cuda.synchronize()
    V.vReduceScatterScaleCast(send, shard, count, F32, "sum", F32, 1.0 / n, comm)
    V.vClipGradNorm(tensors, 1.0, norm, ws, comm)
    torch.cuda.synchronize()
    mean = torch.stack(xs).double().sum(0) / n
    want = mean.square().sum().sqrt().item()
    # the shards carry n fp32 additions of their own
    assert abs(norm.item() - want) <= (R.NORM_REL + 2 * n * R.U32) * want
    value = mean[-count:] / want
    slack = (R.CLIP_REL + 2 * n * R.U32) * value.abs() + n * R.U32 * torch.stack(xs).double().abs().sum(0)[-count:] / n / want
    R.assert_close(shard[-1], value, slack, F32, "clipped shard")


def test_refusals(comms):
    n, comm = 2, comms(2)
    g = [[torch.full((64,), 2.0, device=DEV), torch.full((8,), 2.0, dtype=BF16, device=DEV)] for _ in range(n)]
    good = V.vTensorList(g)
    norm = torch.full((1,), 5.0, device=DEV)
    need = V.vGradNormWorkspace(good, comm)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)

    def refused(call):
        with pytest.raises(V.VcommError) as e:
            call()
        assert e.value.code == V.vInvalidArgument

    ptrs = [t.data_ptr() for r in g for t in r]
    counts, types = [64, 8], [V.vFloat32, V.vBFloat16]
    for bad in ((n, counts, [V.vFloat32, V.vInt32], None, ptrs, None), (n, counts, types, None, [None] + ptrs[1:], None),
                (n, counts, types, None, [ptrs[0] + 2] + ptrs[1:], None), (n, counts, types, None, ptrs, [None] + ptrs[1:]),
                (n, counts, types, None, ptrs, ptrs[:3] + [ptrs[3] + 1]), (n, [64, 1 << 41], types, None, ptrs, None),
                (n, [64, (1 << 64) - 1], types, None, ptrs, None), (0, counts, types, None, [], None)):
        refused(lambda: V.TensorList(*bad))
    gone = V.vTensorList(g)
    gone.close()
    refused(lambda: V.vGradNorm(gone, norm, ws, comm))
    refused(lambda: V.vGradNormWorkspace(gone, comm))
    refused(lambda: V.vGradNorm(good, None, ws, comm))
    refused(lambda: V.vGradNorm(good, norm.data_ptr() + 2, ws, comm))
    refused(lambda: V.vGradNorm(good, norm, (None, need), comm))
    refused(lambda: V.vGradNorm(good, norm, (ws.data_ptr(), need - 1), comm))
    refused(lambda: V.vGradNorm(good, norm, (ws.data_ptr() + 8, need), comm))
    for m in (-1.0, float("nan")):
        refused(lambda: V.vClipGradNorm(good, m, norm, ws, comm))
    refused(lambda: V.vGradNorm(V.vTensorList(g[:1]), norm, ws, comm))
    torch.cuda.synchronize()
    assert norm.item() == 5.0 and all((t == 2).all() for r in g for t in r)
    assert V.vcommGetAsyncError(comm) == V.vSuccess
