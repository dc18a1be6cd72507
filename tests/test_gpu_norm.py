"""All-reduce + residual + RMS norm, its 8-bit output and its backward pass against the plain
formulas in 64 bits, at the sizes, alignments, strides and values where they can go wrong."""
from __future__ import annotations

import ctypes

import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V
from tests import norm_ref as R
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5
CANARY = 77.0

# (ranks, rows, hidden): one element, parts of a warp, one warp, a CTA, the longest a CTA
# holds, clusters; odd sizes around each boundary
SIZES = [(1, 1, 1), (2, 5, 1), (1, 3, 7), (3, 17, 8), (1, 200, 31), (2, 33, 64), (4, 7, 100), (1, 70, 127), (8, 9, 128),
         (1, 9, 129), (2, 40, 255), (1, 65, 512), (5, 11, 1000), (1, 3, 1023), (2, 301, 1024), (1, 2, 1025),
         (8, 1, 4096), (3, 160, 4096), (2, 170, 4097), (1, 1, 5120), (64, 2, 640), (2, 155, 8200), (1, 160, 16384),
         (2, 3, 20480), (1, 160, 20481), (1, 2, 40961), (1, 2, 65535), (2, 3, 65536)]
# enough rows for CTAs to take several: parts of a warp, whole warps, long rows, rows of which
# one fills an SM's share (aligned and not), rows that are too much to stage
MANY = [(8, 400, 4096), (8, 401, 4099), (16, 330, 8192), (24, 310, 9001), (1, 45000, 64), (2, 9001, 200), (1, 5003, 520), (3, 3001, 1000), (8, 1301, 1024), (1, 2601, 1031), (2, 1400, 4097),
        (1, 700, 16384)]
TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)]


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


def rows_buffer(rows, hidden, dtype, stride, offset=0, fill=None):
    """A [rows, hidden] view whose rows are `stride` apart, `offset` elements into memory that
    is filled with `fill`."""
    flat = torch.empty(offset + rows * stride + 64, dtype=dtype, device=DEV)
    if fill is not None:
        flat.fill_(fill)
    view = flat[offset:offset + rows * stride].view(rows, stride)[:, :hidden]
    return flat, view


def make(n, rows, hidden, dtype, wtype, seed, residual=True, stride=None, offset=0):
    gen = torch.Generator().manual_seed(seed)
    xs = (torch.randn(n, rows, hidden, generator=gen) / n ** 0.5).to(dtype)
    if rows > 4:
        xs[:, 3] = 0
    res = (torch.randn(rows, hidden, generator=gen) * 2).to(dtype) if residual else None
    if residual and rows > 4:
        res[3] = 0                                    # a row of zeros: 1 / sqrt(eps)
    w = (1 + 0.2 * torch.randn(hidden, generator=gen)).to(wtype)
    sends = []
    for r in range(n):
        _, v = rows_buffer(rows, hidden, dtype, stride or hidden, offset)
        v.copy_(xs[r])
        sends.append(v)
    return xs, res, w, sends


def place(t, offset=0):
    """A device copy that starts `offset` elements into its allocation."""
    flat = torch.empty(t.numel() + offset, dtype=t.dtype, device=DEV)
    v = flat[offset:].view(t.shape)
    v.copy_(t)
    return v


def check_outside(flat, view, fill, what):
    """Nothing but the view's rows was written."""
    mask = torch.ones_like(flat, dtype=torch.bool)
    start = (view.data_ptr() - flat.data_ptr()) // flat.element_size()
    idx = start + torch.arange(view.shape[0], device=DEV)[:, None] * view.stride(0) + torch.arange(view.shape[1], device=DEV)
    mask[idx.flatten()] = False
    assert (flat[mask].float() == fill).all(), what


def run_forward(comm, n, rows, hidden, dtype, wtype, seed, residual=True, send_pad=0, res_pad=0, recv_pad=0, offset=0,
                recv_offset=0, weight_offset=0, skip=()):
    xs, res, w, sends = make(n, rows, hidden, dtype, wtype, seed, residual, hidden + send_pad, offset)
    desc = V.vRmsNormDesc(rows, hidden, dtype, wtype, EPS, hidden + send_pad, hidden + res_pad, hidden + recv_pad)
    dres = None
    if residual:
        _, dres = rows_buffer(rows, hidden, dtype, hidden + res_pad, offset)
        dres.copy_(res)
    hflat, hout = rows_buffer(rows, hidden, dtype, hidden + res_pad, offset, CANARY)
    outs = [None if r in skip else rows_buffer(rows, hidden, dtype, hidden + recv_pad, recv_offset, CANARY) for r in range(n)]
    rstd = torch.empty(rows, device=DEV)
    V.vAllReduceRmsNorm(desc, sends, dres, place(w, weight_offset), hout, [o and o[1] for o in outs], rstd, comm)
    torch.cuda.synchronize()
    ref = R.forward(xs, res, w, EPS)
    R.assert_close(hout, ref["h"], ref["dh"], dtype, "stream")
    R.assert_close(rstd, ref["rstd"], ref["drstd"], F32, "rstd")
    for r, o in enumerate(outs):
        if o is not None:
            R.assert_close(o[1], ref["y"], ref["dy"], dtype, f"rank {r}")
            check_outside(*o, CANARY, f"rank {r}: written outside its rows")
    check_outside(hflat, hout, CANARY, "stream: written outside its rows")


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("n,rows,hidden", SIZES + MANY)
def test_forward(comms, n, rows, hidden, dtype, wtype):
    run_forward(comms(n), n, rows, hidden, dtype, wtype, seed=hidden + n)


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("kw", [dict(send_pad=3), dict(res_pad=5), dict(recv_pad=1), dict(offset=1), dict(recv_offset=3),
                                dict(weight_offset=1), dict(send_pad=8, res_pad=16, recv_pad=24),
                                dict(send_pad=1, res_pad=2, recv_pad=3, offset=5, recv_offset=2, weight_offset=7)])
@pytest.mark.parametrize("n,rows,hidden", [(3, 21, 96), (2, 5, 1000), (1, 300, 1030), (2, 3, 4099), (1, 2, 33000),
                                           (2, 9000, 136), (1, 2700, 1030), (3, 900, 4099)])
def test_forward_strides_and_offsets(comms, n, rows, hidden, dtype, wtype, kw):
    run_forward(comms(n), n, rows, hidden, dtype, wtype, seed=7, **kw)


@pytest.mark.parametrize("hidden", [512, 515])
def test_forward_optional_arguments(comms, hidden):
    run_forward(comms(4), 4, 20, hidden, BF16, BF16, 3, residual=False)
    run_forward(comms(4), 4, 20, hidden, BF16, BF16, 4, skip=(0, 2, 3))
    xs, _, w, sends = make(4, 20, hidden, BF16, BF16, 5, residual=False)
    outs = [torch.empty(20, hidden, dtype=BF16, device=DEV) for _ in range(4)]
    V.vAllReduceRmsNorm(V.vRmsNormDesc(20, hidden, BF16, eps=EPS), sends, None, place(w), None, outs, None, comms(4))
    ref = R.forward(xs, None, w, EPS)
    for o in outs:
        R.assert_close(o, ref["y"], ref["dy"], BF16, "no stream, no rstd")


@pytest.mark.parametrize("rows,hidden", [(37, 256), (37, 1001), (37, 2048), (37, 30000), (3000, 256), (3000, 1001)])
def test_forward_in_place(comms, rows, hidden):
    n = 3
    xs, res, w, sends = make(n, rows, hidden, BF16, F32, 11)
    stream = place(res)
    V.vAllReduceRmsNorm(V.vRmsNormDesc(rows, hidden, BF16, F32, EPS), sends, stream, place(w), stream, sends, None, comms(n))
    ref = R.forward(xs, res, w, EPS)
    R.assert_close(stream, ref["h"], ref["dh"], BF16, "stream")
    for s in sends:
        R.assert_close(s, ref["y"], ref["dy"], BF16, "in place")


@pytest.mark.parametrize("rows,hidden", [(9, 96), (9, 1000), (9, 1003), (9, 24000), (2700, 1000), (2700, 1003)])
def test_rows_with_infinities_and_nans_stay_alone(comms, rows, hidden):
    n = 2
    xs, res, w, _ = make(n, rows, hidden, BF16, BF16, 13)
    xs[1, 2, hidden // 2] = float("nan")
    xs[0, 5, hidden - 1] = float("inf")
    res[7, 0] = float("-inf")
    sends = [place(x) for x in xs]
    outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
    rstd = torch.empty(rows, device=DEV)
    V.vAllReduceRmsNorm(V.vRmsNormDesc(rows, hidden, BF16, eps=EPS), sends, place(res), place(w), None, outs, rstd, comms(n))
    out = outs[1].double().cpu()
    fine = [r for r in range(rows) if r not in (2, 5, 7)]
    ref = R.forward(xs[:, fine], res[fine], w, EPS)
    R.assert_close(out[fine], ref["y"], ref["dy"], BF16, "other rows")
    assert torch.isnan(out[2]).all() and torch.isnan(rstd[2])
    for row, col in ((5, hidden - 1), (7, 0)):        # 0 everywhere, infinity times 0 at the element
        assert rstd[row].item() == 0.0 and torch.isnan(out[row, col])
        keep = torch.arange(hidden) != col
        assert (out[row][keep] == 0).all()


def test_no_rows_and_no_elements(comms):
    buf = torch.full((8,), CANARY, device=DEV)
    for rows, hidden in ((0, 8), (3, 0)):
        desc = V.vRmsNormDesc(rows, hidden, F32)
        V.vAllReduceRmsNorm(desc, [buf], None, buf, None, [buf], None, comms(1))
    torch.cuda.synchronize()
    assert (buf == CANARY).all()
    # a weight gradient that sums over no rows is zero
    desc = V.vRmsNormDesc(0, 8, F32)
    ws = torch.empty(V.vRmsNormBackwardWorkspace(desc, comms(1)), dtype=torch.uint8, device=DEV)
    V.vAllReduceRmsNormBackward(desc, [buf], buf, buf, buf, None, [buf], buf, ws, comms(1))
    assert (buf == 0).all()


@pytest.mark.parametrize("general", [False, True])
def test_forward_rows_past_two_to_the_31_elements(comms, general):
    hidden, stride = (8192, 8192) if not general else (8191, 8193)
    rows = (1 << 31) // stride + 5
    x = torch.empty(rows * stride, dtype=BF16, device=DEV).normal_().view(rows, stride)[:, :hidden]
    w = torch.ones(hidden, dtype=BF16, device=DEV)
    out = torch.zeros(rows * stride, dtype=BF16, device=DEV).view(rows, stride)[:, :hidden]
    V.vAllReduceRmsNorm(V.vRmsNormDesc(rows, hidden, BF16, eps=EPS, send_stride=stride, recv_stride=stride),
                        [x], None, w, None, [out], None, comms(1))
    pick = [0, 1, rows // 2, rows - 6, rows - 2, rows - 1]
    ref = R.forward(x[pick].cpu()[None], None, w.cpu(), EPS)
    R.assert_close(out[pick], ref["y"], ref["dy"], BF16, "sampled rows")
    if general:
        assert (out.as_strided((rows, stride - hidden), (stride, 1), hidden) == 0).all()


# ---- 8-bit output --------------------------------------------------------------------------

def run_quant(comm, n, rows, hidden, dtype, wtype, group, seed, send_pad=0, recv_pad=0, recv_offset=0, offset=0):
    xs, res, w, sends = make(n, rows, hidden, dtype, wtype, seed, True, hidden + send_pad, offset)
    desc = V.vRmsNormDesc(rows, hidden, dtype, wtype, EPS, hidden + send_pad, 0, hidden + recv_pad, group)
    groups = -(-hidden // group) if group else 1
    outs = [rows_buffer(rows, hidden, torch.uint8, hidden + recv_pad, recv_offset, 77) for _ in range(n)]
    scales = [torch.full((rows * groups + 8,), CANARY, device=DEV) for _ in range(n)]
    hout = torch.empty(rows, hidden, dtype=dtype, device=DEV)
    rstd = torch.empty(rows, device=DEV)
    V.vAllReduceRmsNormQuant(desc, sends, place(res), place(w), hout, [o[1] for o in outs], scales, rstd, comm)
    torch.cuda.synchronize()
    ref = R.forward(xs, res, w, EPS)
    R.assert_close(hout, ref["h"], ref["dh"], dtype, "stream")
    R.assert_close(rstd, ref["rstd"], ref["drstd"], F32, "rstd")
    for r in range(n):
        q = outs[r][1].contiguous().view(torch.float8_e4m3fn).double().cpu()
        R.assert_quantised(q, scales[r][:rows * groups].view(rows, groups).double().cpu(), ref, group, f"rank {r}")
        check_outside(*outs[r], 77, f"rank {r}: written outside its rows")
        assert (scales[r][rows * groups:] == CANARY).all()


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("n,rows,hidden", SIZES + MANY)
def test_quantised(comms, n, rows, hidden, dtype, wtype, group):
    run_quant(comms(n), n, rows, hidden, dtype, wtype, group, seed=hidden)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [dict(send_pad=3), dict(recv_pad=5), dict(recv_offset=1), dict(offset=1),
                                dict(recv_offset=3, recv_pad=2, send_pad=1, offset=2)])
@pytest.mark.parametrize("n,rows,hidden", [(2, 21, 96), (1, 6, 300), (3, 4, 1029), (1, 2, 33000), (2, 9000, 136),
                                           (3, 2000, 1029)])
def test_quantised_strides_and_offsets(comms, n, rows, hidden, dtype, group, kw):
    run_quant(comms(n), n, rows, hidden, dtype, dtype, group, 5, **kw)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("hidden", [64, 384, 1000, 1001, 24000])
def test_quantised_special_values(comms, group, hidden):
    # a row of zeros, one with a NaN, and one whose other groups are zero
    rows = 5
    x = torch.randn(1, rows, hidden, generator=torch.Generator().manual_seed(1)).to(BF16)
    x[0, 1] = 0
    x[0, 2, hidden // 2] = float("nan")
    x[0, 3, min(128, hidden - 1):] = 0
    w = torch.ones(hidden, dtype=BF16)
    groups = -(-hidden // group) if group else 1
    q = torch.empty(rows, hidden, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, groups, device=DEV)
    V.vAllReduceRmsNormQuant(V.vRmsNormDesc(rows, hidden, BF16, eps=EPS, quant_group=group), [place(x[0])], None,
                             place(w), None, [q], [scales], None, comms(1))
    q, scales = q.view(torch.float8_e4m3fn).double().cpu(), scales.double().cpu()
    assert (q[1] == 0).all() and (scales[1].float() == torch.tensor(2.0 ** -64) / 448).all()
    assert torch.isnan(q[2]).all() and torch.isnan(scales[2]).all()      # rstd is NaN, so all is
    fine = [0, 3, 4]
    R.assert_quantised(q[fine], scales[fine], R.forward(x[:, fine], None, w, EPS), group, "other rows")
    assert q[0].abs().max() == 448.0


# ---- backward ------------------------------------------------------------------------------

def run_backward(comm, n, rows, hidden, dtype, wtype, seed, residual=True, send_pad=0, res_pad=0, recv_pad=0, offset=0,
                 recv_offset=0, weight_offset=0, skip=()):
    gen = torch.Generator().manual_seed(seed)
    dys, dres, w, sends = make(n, rows, hidden, dtype, wtype, seed, residual, hidden + send_pad, offset)
    hid = torch.randn(rows, hidden, generator=gen).to(dtype)
    rstd = (hid.float().square().mean(1) + EPS).rsqrt()
    desc = V.vRmsNormDesc(rows, hidden, dtype, wtype, EPS, hidden + send_pad, hidden + res_pad, hidden + recv_pad)
    _, dhid = rows_buffer(rows, hidden, dtype, hidden + res_pad, offset)
    dhid.copy_(hid)
    ddres = None
    if residual:
        _, ddres = rows_buffer(rows, hidden, dtype, hidden + res_pad, offset)
        ddres.copy_(dres)
    outs = [None if r in skip else rows_buffer(rows, hidden, dtype, hidden + recv_pad, recv_offset, CANARY) for r in range(n)]
    dw = torch.full((hidden + 4,), CANARY, dtype=wtype, device=DEV)
    need = V.vRmsNormBackwardWorkspace(desc, comm)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)      # NaNs, and a canary behind
    V.vAllReduceRmsNormBackward(desc, sends, dhid, rstd.to(DEV), place(w, weight_offset), ddres, [o and o[1] for o in outs],
                                dw, (ws.data_ptr(), need), comm)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xFF).all(), "written behind the workspace"
    assert (dw[hidden:] == CANARY).all()
    ref = R.backward(dys, hid, rstd, w, dres)
    R.assert_close(dw[:hidden], ref["dw"], ref["ddw"], wtype, "weight gradient")
    for r, o in enumerate(outs):
        if o is not None:
            R.assert_close(o[1], ref["dh"], ref["ddh"], dtype, f"rank {r}")
            check_outside(*o, CANARY, f"rank {r}: written outside its rows")


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("n,rows,hidden", SIZES + MANY + [(1, 5000, 64), (2, 3001, 257), (1, 2000, 2048)])
def test_backward(comms, n, rows, hidden, dtype, wtype):
    run_backward(comms(n), n, rows, hidden, dtype, wtype, seed=hidden + n)


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("kw", [dict(send_pad=3), dict(res_pad=5), dict(recv_pad=1), dict(offset=1), dict(recv_offset=3),
                                dict(weight_offset=1), dict(residual=False),
                                dict(send_pad=1, res_pad=2, recv_pad=3, offset=5, recv_offset=2, weight_offset=7)])
@pytest.mark.parametrize("n,rows,hidden", [(3, 21, 96), (2, 5, 1000), (1, 900, 1030), (2, 3, 4099), (1, 200, 21003),
                                           (2, 9000, 136), (3, 2000, 1030)])
def test_backward_strides_and_offsets(comms, n, rows, hidden, dtype, wtype, kw):
    run_backward(comms(n), n, rows, hidden, dtype, wtype, seed=9, **kw)


def test_backward_optional_arguments_and_in_place(comms):
    run_backward(comms(3), 3, 50, 256, BF16, F32, 4, skip=(0, 2))
    n, rows, hidden = 2, 40, 1001
    dys, dres, w, sends = make(n, rows, hidden, BF16, BF16, 21)
    hid = torch.randn(rows, hidden, generator=torch.Generator().manual_seed(2)).to(BF16)
    rstd = (hid.float().square().mean(1) + EPS).rsqrt()
    desc = V.vRmsNormDesc(rows, hidden, BF16, eps=EPS)
    ws = torch.empty(V.vRmsNormBackwardWorkspace(desc, comms(n)), dtype=torch.uint8, device=DEV)
    dw = torch.empty(hidden, dtype=BF16, device=DEV)
    ddres = place(dres)
    ref = R.backward(dys, hid, rstd, w, dres)
    V.vAllReduceRmsNormBackward(desc, sends, place(hid), rstd.to(DEV), place(w), ddres, [None, ddres], dw, ws, comms(n))
    R.assert_close(ddres, ref["dh"], ref["ddh"], BF16, "in place of the residual's gradient")
    ddres = place(dres)
    V.vAllReduceRmsNormBackward(desc, sends, place(hid), rstd.to(DEV), place(w), ddres, sends, dw, ws, comms(n))
    for s in sends:
        R.assert_close(s, ref["dh"], ref["ddh"], BF16, "in place of the partial gradients")
    R.assert_close(dw, ref["dw"], ref["ddw"], BF16, "weight gradient")


@pytest.mark.parametrize("n,rows,hidden", [(1, 700, 64), (2, 333, 1001), (4, 1000, 2048), (2, 3000, 1001), (1, 45000, 72)])
def test_backward_gives_the_same_bits_again(comms, n, rows, hidden):
    dys, dres, w, sends = make(n, rows, hidden, BF16, F32, 23)
    hid = place(torch.randn(rows, hidden).to(BF16))
    rstd = (hid.float().square().mean(1) + EPS).rsqrt()
    desc = V.vRmsNormDesc(rows, hidden, BF16, F32, EPS)
    got = []
    for _ in range(3):
        ws = torch.empty(V.vRmsNormBackwardWorkspace(desc, comms(n)), dtype=torch.uint8, device=DEV)
        dw = torch.empty(hidden, device=DEV)
        outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
        V.vAllReduceRmsNormBackward(desc, sends, hid, rstd, place(w), place(dres), outs, dw, ws, comms(n))
        got.append((dw, outs[-1]))
    for dw, o in got[1:]:
        assert torch.equal(dw, got[0][0]) and torch.equal(o, got[0][1])


@pytest.mark.parametrize("n,rows,hidden", [(2, 5, 512), (1, 64, 96), (3, 17, 1001)])
def test_backward_of_few_rows_many_times_and_replayed(comms, n, rows, hidden):
    # the pass whose last CTA adds up the weight's gradient: more calls than counters, with other
    # calls between, and replays of a capture between eager calls
    comm = comms(n)
    dys, dres, w, sends = make(n, rows, hidden, BF16, F32, 25)
    hid = torch.randn(rows, hidden, generator=torch.Generator().manual_seed(3)).to(BF16)
    rstd = (hid.float().square().mean(1) + EPS).rsqrt()
    desc = V.vRmsNormDesc(rows, hidden, BF16, F32, EPS)
    ws = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
    args = (sends, place(hid), rstd.to(DEV), place(w), place(dres))
    ref = R.backward(dys, hid, rstd, w, dres)
    outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]

    def run(dw):
        V.vAllReduceRmsNormBackward(desc, *args, outs, dw, ws, comm)

    captured = torch.empty(hidden, device=DEV)
    run(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(captured)
    got = []
    for i in range(150):
        got.append(torch.full((hidden,), CANARY, device=DEV))
        run(got[-1])
        if i % 50 == 0:
            captured.zero_()
            graph.replay()
            got.append(captured.clone())
    torch.cuda.synchronize()
    R.assert_close(got[0], ref["dw"], ref["ddw"], F32, "weight gradient")
    R.assert_close(outs[0], ref["dh"], ref["ddh"], BF16, "gradient")
    assert all(torch.equal(g, got[0]) for g in got)


@pytest.mark.parametrize("n,rows,hidden", [(2, 4, 40), (1, 4, 301), (3, 3, 1024)])
def test_backward_against_differences_of_the_forward_pass(comms, n, rows, hidden):
    """dL of L = sum(y a) + sum(h b) along a random direction of each input, against the
    central difference of the kernel's own fp32 forward pass.  With directions of unit
    elements and steps of d = 2^-5, the difference is off by d^2/6 of the third derivative (a
    few times the first for rows of unit scale: allowed 16 d^2/6) and by the fp32 rounding of
    the outputs over d."""
    comm, gen = comms(n), torch.Generator().manual_seed(n * hidden)
    xs, res, w, _ = make(n, rows, hidden, F32, F32, 31)
    a, b = (torch.randn(rows, hidden, generator=gen) for _ in range(2))
    desc = V.vRmsNormDesc(rows, hidden, F32, eps=EPS)

    def loss(x, r, weight):
        y = [None] * (n - 1) + [torch.empty(rows, hidden, device=DEV)]
        h = torch.empty(rows, hidden, device=DEV)
        rstd = torch.empty(rows, device=DEV)
        V.vAllReduceRmsNorm(desc, [place(t) for t in x], place(r), place(weight), h, y, rstd, comm)
        return ((y[-1].double().cpu() * a).sum() + (h.double().cpu() * b).sum()).item(), h, rstd

    _, h, rstd = loss(xs, res, w)
    # the gradient of y reaches the norm as n partial gradients that add up to a
    parts = torch.randn(n, rows, hidden, generator=gen)
    parts[-1] = a - parts[:-1].sum(0)
    ws = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
    dw = torch.empty(hidden, device=DEV)
    dh = [torch.empty(rows, hidden, device=DEV) for _ in range(n)]
    V.vAllReduceRmsNormBackward(desc, [place(p) for p in parts], h, rstd, place(w), place(b), dh, dw, ws, comm)
    d = 2.0 ** -5
    for what in ("x", "residual", "weight"):
        v = torch.randn(hidden, generator=gen) if what == "weight" else torch.randn(rows, hidden, generator=gen)

        def at(s):
            x, r, weight = xs.clone(), res, w
            if what == "x":
                x[n // 2] += s * d * v
            elif what == "residual":
                r = res + s * d * v
            else:
                weight = w + s * d * v
            return loss(x, r, weight)[0]

        numeric = (at(1) - at(-1)) / (2 * d)
        grad = (dw if what == "weight" else dh[n // 2]).double().cpu()
        analytic = (grad * v).sum().item()
        scale = (grad.abs() * v.abs()).sum().item()
        noise = 64 * R.U32 * (rows * hidden) ** 0.5 * 4 / d
        assert abs(numeric - analytic) <= 16 * d * d / 6 * scale + noise, what


# ---- streams, groups, graphs -----------------------------------------------------------------

def test_on_another_stream_in_a_group_and_in_a_graph(comms):
    n, rows, hidden = 2, 64, 2048
    comm = comms(n)
    xs, res, w, sends = make(n, rows, hidden, BF16, BF16, 41)
    desc = V.vRmsNormDesc(rows, hidden, BF16, eps=EPS)
    dres, dw_ = place(res), place(w)
    ref = R.forward(xs, res, w, EPS)
    side = torch.cuda.Stream()
    outs = [torch.zeros(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
    side.wait_stream(torch.cuda.current_stream())
    V.vAllReduceRmsNorm(desc, sends, dres, dw_, None, outs, None, comm, stream=side)
    side.synchronize()
    R.assert_close(outs[0], ref["y"], ref["dy"], BF16, "side stream")

    for o in outs:
        o.zero_()
    rstd = torch.empty(rows, device=DEV)
    stream = torch.empty(rows, hidden, dtype=BF16, device=DEV)
    V.vcommGroupStart(comm)
    V.vAllReduceRmsNorm(desc, list(sends), dres, dw_, stream, list(outs), rstd, comm)
    torch.cuda.synchronize()
    assert (outs[1] == 0).all()                       # recorded, not run
    V.vcommGroupEnd(comm)
    R.assert_close(outs[1], ref["y"], ref["dy"], BF16, "group")

    # forward and backward captured together, replayed on new contents of the same buffers
    ws = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
    dh = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
    gw = torch.empty(hidden, dtype=BF16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        V.vAllReduceRmsNorm(desc, sends, dres, dw_, stream, outs, rstd, comm)
        V.vAllReduceRmsNormBackward(desc, outs, stream, rstd, dw_, None, dh, gw, ws, comm)
    for s, x in zip(sends, xs):
        s.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    ref = R.forward(xs.flip(1), res, w, EPS)
    R.assert_close(outs[0], ref["y"], ref["dy"], BF16, "replay")
    back = R.backward(torch.stack([o.cpu() for o in outs]), stream.cpu(), rstd.cpu(), w, None)
    R.assert_close(dh[0], back["dh"], back["ddh"], BF16, "replayed backward")
    R.assert_close(gw, back["dw"], back["ddw"], BF16, "replayed weight gradient")


def test_two_streams_and_plain_launches(monkeypatch):
    # the same calls on two streams at once, on a communicator without early launches
    monkeypatch.setenv("VCOMM_PDL", "0")
    n, rows, hidden = 2, 3000, 1024
    comm = V.vcommInit(n)
    try:
        desc = V.vRmsNormDesc(rows, hidden, BF16, eps=EPS)
        runs = []
        for seed in (51, 52):
            xs, res, w, sends = make(n, rows, hidden, BF16, BF16, seed)
            outs = [torch.zeros(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
            dh = [torch.zeros(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
            ws = torch.empty(V.vRmsNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
            runs.append((xs, res, w, sends, place(res), place(w), torch.zeros(rows, hidden, dtype=BF16, device=DEV), outs,
                         torch.zeros(rows, device=DEV), dh, torch.zeros(hidden, dtype=BF16, device=DEV), ws,
                         torch.cuda.Stream()))
        torch.cuda.synchronize()
        for _ in range(3):
            for xs, res, w, sends, dres, dw, stream, outs, rstd, dh, gw, ws, side in runs:
                V.vAllReduceRmsNorm(desc, sends, dres, dw, stream, outs, rstd, comm, stream=side)
                V.vAllReduceRmsNormBackward(desc, outs, stream, rstd, dw, None, dh, gw, ws, comm, stream=side)
        torch.cuda.synchronize()
        for xs, res, w, sends, dres, dw, stream, outs, rstd, dh, gw, ws, side in runs:
            ref = R.forward(xs, res, w, EPS)
            R.assert_close(outs[1], ref["y"], ref["dy"], BF16, "output")
            back = R.backward(torch.stack([o.cpu() for o in outs]), stream.cpu(), rstd.cpu(), w, None)
            R.assert_close(dh[0], back["dh"], back["ddh"], BF16, "gradient")
            R.assert_close(gw, back["dw"], back["ddw"], BF16, "weight gradient")
    finally:
        V.vcommDestroy(comm)


def test_a_chain_without_waits_keeps_stream_order(comms):
    # every step reads what the one before wrote, the weight included
    n, rows, hidden = 2, 512, 1024
    comm = comms(n)
    xs, res, w, sends = make(n, rows, hidden, F32, F32, 43)
    desc = V.vRmsNormDesc(rows, hidden, F32, eps=EPS)
    for _ in range(5):
        weight = torch.zeros(hidden, device=DEV)
        a = [torch.zeros(rows, hidden, device=DEV) for _ in range(n)]
        b = [torch.zeros(rows, hidden, device=DEV) for _ in range(n)]
        src = place(w)
        torch.cuda.synchronize()
        V.vBroadcast([src, None], [weight, torch.empty_like(src)], hidden, F32, "sum", 0, comm)
        V.vAllReduceRmsNorm(desc, sends, None, weight, None, a, None, comm)
        V.vAllReduceRmsNorm(desc, a, None, weight, None, b, None, comm)
        torch.cuda.synchronize()
        ref = R.forward(xs, None, w, EPS)
        R.assert_close(a[0], ref["y"], ref["dy"], F32, "first")
        two = R.forward(torch.stack([t.cpu() for t in a]), None, w, EPS)
        R.assert_close(b[1], two["y"], two["dy"], F32, "second")


# ---- refusals ------------------------------------------------------------------------------

def test_refusals(comms):
    n, rows, hidden = 2, 4, 64
    comm = comms(n)
    bufs = [torch.full((rows, hidden), CANARY, dtype=BF16, device=DEV) for _ in range(6)]
    w, rstd = torch.ones(hidden, dtype=BF16, device=DEV), torch.ones(rows, device=DEV)
    good = dict(rows=rows, hidden=hidden, datatype=BF16)
    sends, recvs = bufs[:2], bufs[2:4]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    scales = [torch.zeros(rows, device=DEV)] * 2

    def refused(call, code=V.vInvalidArgument):
        with pytest.raises(V.VcommError) as e:
            call()
        assert e.value.code == code

    for change in (dict(datatype=torch.int32), dict(hidden=65537), dict(rows=1 << 31), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(eps=float("inf")), dict(send_stride=63), dict(residual_stride=1), dict(recv_stride=2),
                   dict(recv_stride=1 << 62), dict(weight_type=torch.float16), dict(quant_group=64), dict(quant_group=-1)):
        d = V.vRmsNormDesc(**{**good, **change})
        refused(lambda: V.vAllReduceRmsNorm(d, sends, None, w, None, recvs, None, comm))
        refused(lambda: V.vAllReduceRmsNormQuant(d, sends, None, w, None, recvs, scales, None, comm))
        refused(lambda: V.vAllReduceRmsNormBackward(d, sends, bufs[4], rstd, w, None, recvs, w, ws, comm))
        refused(lambda: V.vRmsNormBackwardWorkspace(d, comm))
    d = V.vRmsNormDesc(**good)
    odd = bufs[0].data_ptr() + 1
    for s, res, weight, out, recv, r in [([None, bufs[1]], None, w, None, recvs, None), ([odd, bufs[1]], None, w, None, recvs, None),
                                         (sends, odd, w, None, recvs, None), (sends, None, None, None, recvs, None),
                                         (sends, None, odd, None, recvs, None), (sends, None, w, odd, recvs, None),
                                         (sends, None, w, None, [None, None], None), (sends, None, w, None, [odd, None], None),
                                         (sends, None, w, None, recvs, odd), (sends[:1], None, w, None, recvs, None),
                                         (sends, None, w, None, recvs + recvs, None)]:
        refused(lambda: V.vAllReduceRmsNorm(d, s, res, weight, out, recv, r, comm))
    refused(lambda: V.vAllReduceRmsNormQuant(d, sends, None, w, None, recvs, [None, scales[0]], None, comm))
    need = V.vRmsNormBackwardWorkspace(d, comm)
    for hid, r, weight, dres, recv, dw, space in [(None, rstd, w, None, recvs, w, ws), (bufs[4], None, w, None, recvs, w, ws),
                                                  (bufs[4], rstd, None, None, recvs, w, ws), (bufs[4], rstd, w, odd, recvs, w, ws),
                                                  (bufs[4], rstd, w, None, recvs, None, ws), (bufs[4], rstd, w, None, recvs, w, (None, 1 << 20)),
                                                  (bufs[4], rstd, w, None, recvs, w, (ws.data_ptr(), need - 1)),
                                                  (bufs[4], rstd, w, None, recvs, w, (ws.data_ptr() + 4, 1 << 19)),
                                                  (bufs[4], rstd, w, None, [None, None], w, ws)]:
        refused(lambda: V.vAllReduceRmsNormBackward(d, sends, hid, r, weight, dres, recv, dw, space, comm))
    lib = V.lib()
    arr = (ctypes.c_void_p * 2)(*[b.data_ptr() for b in sends])
    assert lib.vAllReduceRmsNorm(None, arr, None, w.data_ptr(), None, arr, None, comm, None) == V.vInvalidArgument
    assert lib.vAllReduceRmsNorm(ctypes.addressof(d), None, None, w.data_ptr(), None, arr, None, comm, None) == V.vInvalidArgument
    # nothing was launched, and nothing sticks
    torch.cuda.synchronize()
    assert all((b == CANARY).all() for b in bufs)
    assert V.vcommGetAsyncError(comm) == V.vSuccess
    # a group reports a recorded call's error at its end
    V.vcommGroupStart(comm)
    V.vAllReduceRmsNorm(d, sends, None, None, None, recvs, None, comm)
    refused(lambda: V.vcommGroupEnd(comm))


# rows too long for one CTA to stage, and enough of them that each cluster takes several
LONG = [(1, 400, 32776), (8, 330, 16384), (3, 290, 24001), (2, 230, 65536), (16, 170, 12296), (64, 90, 4096), (40, 161, 2100)]


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("kw", [dict(), dict(send_pad=1, recv_offset=3, offset=5, weight_offset=1)])
@pytest.mark.parametrize("n,rows,hidden", LONG)
def test_long_rows_forward(comms, n, rows, hidden, dtype, wtype, kw):
    run_forward(comms(n), n, rows, hidden, dtype, wtype, seed=hidden + n, **kw)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("kw", [dict(), dict(send_pad=1, recv_offset=3, offset=5)])
@pytest.mark.parametrize("n,rows,hidden", LONG)
def test_long_rows_quantised(comms, n, rows, hidden, dtype, wtype, group, kw):
    run_quant(comms(n), n, rows, hidden, dtype, wtype, group, seed=hidden, **kw)


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("kw", [dict(), dict(send_pad=1, recv_offset=3, offset=5, weight_offset=1)])
@pytest.mark.parametrize("n,rows,hidden", LONG)
def test_long_rows_backward(comms, n, rows, hidden, dtype, wtype, kw):
    run_backward(comms(n), n, rows, hidden, dtype, wtype, seed=hidden + n, **kw)
