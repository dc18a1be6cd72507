"""The norms after and before a block with its gate and the scaled residual, and their backward pass,
against the plain formulas in 64 bits, at the sizes, alignments, strides and values where they can go
wrong."""
from __future__ import annotations

import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V
from tests import block_ref as B
from tests import norm_ref as R
from tests.gpu_util import DEV
from tests.test_gpu_norm import BF16, CANARY, EPS, F16, F32, check_outside, place, rows_buffer

pytestmark = pytest.mark.gpu

# (ranks, rows, hidden): one element, parts of a warp, one warp, a CTA, clusters; odd sizes around each
# boundary; a row that fills a CTA's threads with two sums a column
SIZES = [(1, 1, 1), (2, 5, 1), (1, 3, 7), (3, 17, 8), (1, 200, 31), (2, 33, 64), (4, 7, 100), (8, 9, 128), (1, 9, 129),
         (5, 11, 1000), (1, 3, 1023), (2, 301, 1024), (8, 1, 8192), (3, 160, 4096), (2, 170, 4097), (2, 155, 8200),
         (1, 160, 16384), (2, 3, 20480), (1, 160, 20481), (1, 2, 40961), (1, 2, 65535), (2, 3, 65536)]
# enough rows for CTAs to take several, of every way to lay out a row
MANY = [(8, 400, 4096), (8, 401, 4099), (16, 330, 8192), (1, 9001, 64), (2, 9001, 200), (1, 5003, 520), (3, 3001, 1000),
        (1, 2601, 1031), (2, 1400, 4097), (1, 700, 16384), (1, 400, 32776), (3, 290, 24001), (64, 90, 4096)]
TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)]
PADS = [dict(send_pad=3), dict(res_pad=5), dict(recv_pad=1), dict(offset=1), dict(recv_offset=3), dict(weight_offset=1),
        dict(send_pad=8, res_pad=16, recv_pad=24),
        dict(send_pad=1, res_pad=2, recv_pad=3, offset=5, recv_offset=2, weight_offset=7)]


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


def weights(hidden, wtype, gen, gate=True):
    post, pre = ((1 + 0.2 * torch.randn(hidden, generator=gen)).to(wtype) for _ in range(2))
    return post, (0.5 + 0.3 * torch.randn(hidden, generator=gen)).to(wtype) if gate else None, pre


def spread(xs, stride, offset):
    """Device copies whose rows are `stride` apart."""
    got = []
    for x in xs:
        _, v = rows_buffer(x.shape[0], x.shape[1], x.dtype, stride, offset)
        v.copy_(x)
        got.append(v)
    return got


def at(t, offset=0):
    return None if t is None else place(t, offset)


def run_forward(comm, n, rows, hidden, dtype, wtype, seed, residual=True, gate=True, alpha=0.75, send_pad=0, res_pad=0,
                recv_pad=0, offset=0, recv_offset=0, weight_offset=0, skip=()):
    gen = torch.Generator().manual_seed(seed)
    xs = (torch.randn(n, rows, hidden, generator=gen) / n ** 0.5).to(dtype)
    res = (torch.randn(rows, hidden, generator=gen) * 2).to(dtype) if residual else None
    if rows > 4:
        xs[:, 3] = 0                                  # a block output of zeros: 1 / sqrt(eps)
    post, g, pre = weights(hidden, wtype, gen, gate)
    desc = V.vBlockNormDesc(rows, hidden, dtype, wtype, EPS, alpha, hidden + send_pad, hidden + res_pad, hidden + recv_pad)
    sends = spread(xs, hidden + send_pad, offset)
    dres = spread([res], hidden + res_pad, offset)[0] if residual else None
    bflat, bout = rows_buffer(rows, hidden, dtype, hidden + res_pad, offset, CANARY)
    hflat, hout = rows_buffer(rows, hidden, dtype, hidden + res_pad, offset, CANARY)
    outs = [None if r in skip else rows_buffer(rows, hidden, dtype, hidden + recv_pad, recv_offset, CANARY) for r in range(n)]
    rstd = torch.full((2 * rows + 4,), CANARY, device=DEV)
    V.vAllReduceBlockNorm(desc, sends, dres, place(post, weight_offset), at(g, weight_offset), place(pre, weight_offset), bout,
                          hout, [o and o[1] for o in outs], rstd, comm)
    torch.cuda.synchronize()
    ref = B.forward(xs, res, post, g, pre, alpha, EPS)
    R.assert_close(bout, ref["b"], ref["db"], dtype, "block")
    R.assert_close(rstd[:rows], ref["r1"], ref["dr1"], F32, "the block's rstd")
    R.assert_close(hout, ref["h"], ref["dh"], dtype, "stream")
    R.assert_close(rstd[rows:2 * rows], ref["r2"], ref["dr2"], F32, "the stream's rstd")
    assert (rstd[2 * rows:] == CANARY).all()
    for r, o in enumerate(outs):
        if o is not None:
            R.assert_close(o[1], ref["y"], ref["dy"], dtype, f"rank {r}")
            check_outside(*o, CANARY, f"rank {r}: written outside its rows")
    check_outside(hflat, hout, CANARY, "stream: written outside its rows")
    check_outside(bflat, bout, CANARY, "block: written outside its rows")


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("n,rows,hidden", SIZES + MANY)
def test_forward(comms, n, rows, hidden, dtype, wtype):
    run_forward(comms(n), n, rows, hidden, dtype, wtype, seed=hidden + n)


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("kw", PADS)
@pytest.mark.parametrize("n,rows,hidden", [(3, 21, 96), (2, 5, 1000), (2, 3, 4099), (1, 2, 33000), (2, 4000, 136),
                                           (1, 2700, 1030), (3, 290, 20496)])
def test_forward_strides_and_offsets(comms, n, rows, hidden, dtype, wtype, kw):
    run_forward(comms(n), n, rows, hidden, dtype, wtype, seed=7, **kw)


@pytest.mark.parametrize("rows,hidden", [(20, 512), (20, 515), (3000, 512), (3000, 515)])
def test_forward_optional_arguments(comms, rows, hidden):
    run_forward(comms(4), 4, rows, hidden, BF16, BF16, 3, residual=False)
    run_forward(comms(4), 4, rows, hidden, BF16, BF16, 4, skip=(0, 2, 3))
    run_forward(comms(4), 4, rows, hidden, BF16, F32, 5, gate=False, alpha=-1.0)
    run_forward(comms(4), 4, rows, hidden, F16, F16, 6, alpha=0.0)
    gen = torch.Generator().manual_seed(8)
    xs = torch.randn(4, rows, hidden, generator=gen).to(BF16)
    post, _, pre = weights(hidden, BF16, gen)
    outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(4)]
    V.vAllReduceBlockNorm(V.vBlockNormDesc(rows, hidden, BF16, eps=EPS), [place(x) for x in xs], None, place(post), None,
                          place(pre), None, None, outs, None, comms(4))
    ref = B.forward(xs, None, post, None, pre, 1.0, EPS)
    for o in outs:
        R.assert_close(o, ref["y"], ref["dy"], BF16, "nothing kept")


def test_a_residual_that_the_block_cancels(comms):
    # h is a small difference of large parts, which its own mean square must be taken of
    rows, hidden = 6, 1024
    x = torch.randn(rows, hidden, generator=torch.Generator().manual_seed(2))
    ones = torch.ones(hidden)
    res = -(x.double() * ((x.double() ** 2).mean(1, keepdim=True) + EPS).rsqrt()).float()
    res[:, ::2] += 2.0 ** -12
    outs, h = torch.empty(rows, hidden, device=DEV), torch.empty(rows, hidden, device=DEV)
    V.vAllReduceBlockNorm(V.vBlockNormDesc(rows, hidden, F32, eps=0.0), [place(x)], place(res), place(ones), None, place(ones),
                          None, h, [outs], None, comms(1))
    ref = B.forward(x[None], res, ones, None, ones, 1.0, 0.0)
    # the first norm by EPS in the residual, none here: the difference is what stays
    R.assert_close(h, ref["h"], ref["dh"], F32, "stream")
    own = h.double().cpu()
    want = own * (own * own).mean(1, keepdim=True).rsqrt()
    assert ((outs.double().cpu() - want).abs() <= (R.CHAIN + 4) * R.U32 * want.abs() + R.U32 * 8 * want.abs().amax()).all()


@pytest.mark.parametrize("rows,hidden", [(37, 256), (37, 1001), (37, 2048), (37, 30000), (3000, 256), (3000, 1001)])
def test_forward_in_place(comms, rows, hidden):
    n, gen = 3, torch.Generator().manual_seed(11)
    xs, res = torch.randn(n, rows, hidden, generator=gen).to(BF16), torch.randn(rows, hidden, generator=gen).to(BF16)
    post, gate, pre = weights(hidden, F32, gen)
    sends, stream = [place(x) for x in xs], place(res)
    V.vAllReduceBlockNorm(V.vBlockNormDesc(rows, hidden, BF16, F32, EPS, 0.5), sends, stream, place(post), place(gate),
                          place(pre), None, stream, sends, None, comms(n))
    ref = B.forward(xs, res, post, gate, pre, 0.5, EPS)
    R.assert_close(stream, ref["h"], ref["dh"], BF16, "stream")
    for s in sends:
        R.assert_close(s, ref["y"], ref["dy"], BF16, "in place")


@pytest.mark.parametrize("rows,hidden", [(9, 96), (9, 1003), (9, 24000), (2700, 1000), (2700, 1003)])
def test_rows_with_infinities_and_nans_stay_alone(comms, rows, hidden):
    n, gen = 2, torch.Generator().manual_seed(13)
    xs, res = torch.randn(n, rows, hidden, generator=gen).to(BF16), torch.randn(rows, hidden, generator=gen).to(BF16)
    post, gate, pre = weights(hidden, BF16, gen)
    xs[1, 2, hidden // 2] = float("nan")
    xs[0, 5, hidden - 1] = float("inf")
    res[7, 0] = float("-inf")
    outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)]
    rstd = torch.empty(2, rows, device=DEV)
    V.vAllReduceBlockNorm(V.vBlockNormDesc(rows, hidden, BF16, eps=EPS), [place(x) for x in xs], place(res), place(post),
                          place(gate), place(pre), None, None, outs, rstd, comms(n))
    out = outs[1].double().cpu()
    fine = [r for r in range(rows) if r not in (2, 5, 7)]
    ref = B.forward(xs[:, fine], res[fine], post, gate, pre, 1.0, EPS)
    R.assert_close(out[fine], ref["y"], ref["dy"], BF16, "other rows")
    assert torch.isnan(out[2]).all() and torch.isnan(rstd[:, 2]).all()
    # an infinite sum: 0 * infinity in the block's norm, so the stream and all of its row is NaN
    assert rstd[0, 5].item() == 0.0 and torch.isnan(rstd[1, 5]) and torch.isnan(out[5]).all()
    assert rstd[1, 7].item() == 0.0 and torch.isnan(out[7, 0]) and (out[7, 1:] == 0).all()


@pytest.mark.parametrize("general", [False, True])
def test_rows_past_two_to_the_31_elements(comms, general):
    hidden, stride = (8192, 8192) if not general else (8191, 8193)
    rows = (1 << 31) // stride + 5
    x = torch.empty(rows * stride, dtype=BF16, device=DEV).normal_().view(rows, stride)[:, :hidden]
    w = torch.ones(hidden, dtype=BF16, device=DEV)
    out, h, b = (torch.zeros(rows * stride, dtype=BF16, device=DEV).view(rows, stride)[:, :hidden] for _ in range(3))
    V.vAllReduceBlockNorm(V.vBlockNormDesc(rows, hidden, BF16, eps=EPS, residual_scale=0.5, send_stride=stride,
                                           residual_stride=stride, recv_stride=stride), [x], x, w, None, w, b, h, [out], None,
                          comms(1))
    pick = [0, 1, rows // 2, rows - 6, rows - 2, rows - 1]
    one = w.cpu()
    ref = B.forward(x[pick].cpu()[None], x[pick].cpu(), one, None, one, 0.5, EPS)
    for got, name in ((out, "y"), (h, "h"), (b, "b")):
        R.assert_close(got[pick], ref[name], ref["d" + name], BF16, name)
    if general:
        assert (out.as_strided((rows, stride - hidden), (stride, 1), hidden) == 0).all()


# ---- backward ------------------------------------------------------------------------------

def run_backward(comm, n, rows, hidden, dtype, wtype, seed, stream_grad=True, gate=True, residual_grad=True, alpha=0.75,
                 send_pad=0, res_pad=0, recv_pad=0, offset=0, recv_offset=0, weight_offset=0, skip=(), inplace=False):
    gen = torch.Generator().manual_seed(seed)
    dys = (torch.randn(n, rows, hidden, generator=gen) / n ** 0.5).to(dtype)
    hid, block, dstream = (torch.randn(rows, hidden, generator=gen).to(dtype) for _ in range(3))
    rstd = torch.stack([(t.float().square().mean(1) + EPS).rsqrt() for t in (block, hid)])
    post, g, pre = weights(hidden, wtype, gen, gate)
    desc = V.vBlockNormDesc(rows, hidden, dtype, wtype, EPS, alpha, hidden + send_pad, hidden + res_pad, hidden + recv_pad)
    sends = spread(dys, hidden + send_pad, offset)
    dhid, dblock, dds = spread([hid, block, dstream], hidden + res_pad, offset)
    outs = [None if r in skip else rows_buffer(rows, hidden, dtype, hidden + recv_pad, recv_offset, CANARY) for r in range(n)]
    rflat, rout = rows_buffer(rows, hidden, dtype, hidden + res_pad, offset, CANARY)
    if inplace:
        outs, rout, rflat = [(None, s) for s in sends], dds, None
    grads = [torch.full((hidden + 4,), CANARY, dtype=wtype, device=DEV) for _ in range(3)]
    need = V.vBlockNormBackwardWorkspace(desc, comm)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)      # NaNs, and a canary behind
    V.vAllReduceBlockNormBackward(desc, sends, dhid, dblock, rstd.to(DEV), place(post, weight_offset), at(g, weight_offset),
                                  place(pre, weight_offset), dds if stream_grad else None, rout if residual_grad else None,
                                  [o and o[1] for o in outs], grads[0], grads[1] if gate else None, grads[2],
                                  (ws.data_ptr(), need), comm)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xFF).all(), "written behind the workspace"
    ref = B.backward(dys, hid, block, rstd, post, g, pre, dstream if stream_grad else None, alpha)
    for got, name in zip(grads, ("post", "gate", "pre")):
        assert (got[hidden:] == CANARY).all()
        if ref[name] is not None:
            R.assert_close(got[:hidden], ref[name], ref["d" + name], wtype, name)
    if residual_grad:
        R.assert_close(rout, ref["dres"], ref["ddres"], dtype, "residual")
    for r, o in enumerate(outs):
        if o is not None:
            R.assert_close(o[1], ref["db"], ref["ddb"], dtype, f"rank {r}")
            if not inplace:
                check_outside(*o, CANARY, f"rank {r}: written outside its rows")
    if not inplace:
        if residual_grad:
            check_outside(rflat, rout, CANARY, "residual: written outside its rows")
        else:
            assert (rflat == CANARY).all()


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("n,rows,hidden", SIZES + MANY + [(1, 5000, 64), (2, 3001, 257), (1, 2000, 2048)])
def test_backward(comms, n, rows, hidden, dtype, wtype):
    run_backward(comms(n), n, rows, hidden, dtype, wtype, seed=hidden + n)


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("kw", PADS + [dict(stream_grad=False)])
@pytest.mark.parametrize("n,rows,hidden", [(3, 21, 96), (2, 5, 1000), (2, 3, 4099), (1, 200, 21003), (2, 4000, 136),
                                           (3, 2000, 1030)])
def test_backward_strides_and_offsets(comms, n, rows, hidden, dtype, wtype, kw):
    run_backward(comms(n), n, rows, hidden, dtype, wtype, seed=9, **kw)


@pytest.mark.parametrize("rows,hidden", [(50, 256), (50, 1001), (50, 4096), (3000, 256), (3000, 1001)])
def test_backward_optional_arguments_and_in_place(comms, rows, hidden):
    run_backward(comms(3), 3, rows, hidden, BF16, F32, 4, skip=(0, 2))
    run_backward(comms(3), 3, rows, hidden, BF16, F32, 5, gate=False, residual_grad=False)
    run_backward(comms(3), 3, rows, hidden, F32, F32, 6, gate=False, stream_grad=False, alpha=-2.0)
    run_backward(comms(3), 3, rows, hidden, BF16, BF16, 7, inplace=True)


def test_no_rows_and_no_elements(comms):
    buf = torch.full((8,), CANARY, device=DEV)
    for rows, hidden in ((0, 8), (3, 0)):
        desc = V.vBlockNormDesc(rows, hidden, F32)
        V.vAllReduceBlockNorm(desc, [buf], None, buf, None, buf, None, None, [buf], None, comms(1))
    torch.cuda.synchronize()
    assert (buf == CANARY).all()
    desc = V.vBlockNormDesc(0, 8, F32)
    ws = torch.empty(V.vBlockNormBackwardWorkspace(desc, comms(1)), dtype=torch.uint8, device=DEV)
    grads = [torch.full((9,), CANARY, device=DEV) for _ in range(3)]
    V.vAllReduceBlockNormBackward(desc, [buf], buf, buf, buf, buf, buf, buf, None, None, [buf], *grads, ws, comms(1))
    torch.cuda.synchronize()
    assert all((g[:8] == 0).all() and g[8] == CANARY for g in grads) and (buf == CANARY).all()


@pytest.mark.parametrize("n,rows,hidden", [(1, 700, 64), (2, 333, 1001), (4, 1000, 2048), (2, 3000, 1001)])
def test_backward_gives_the_same_bits_again(comms, n, rows, hidden):
    gen = torch.Generator().manual_seed(23)
    sends = [place(torch.randn(rows, hidden, generator=gen).to(BF16)) for _ in range(n)]
    hid, block, ds = (place(torch.randn(rows, hidden, generator=gen).to(BF16)) for _ in range(3))
    rstd = torch.rand(2, rows, generator=gen).to(DEV)
    post, gate, pre = (place(t) for t in weights(hidden, F32, gen))
    desc = V.vBlockNormDesc(rows, hidden, BF16, F32, EPS)
    got = []
    for _ in range(3):
        ws = torch.empty(V.vBlockNormBackwardWorkspace(desc, comms(n)), dtype=torch.uint8, device=DEV)
        grads = [torch.empty(hidden, device=DEV) for _ in range(3)]
        outs = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n + 1)]
        V.vAllReduceBlockNormBackward(desc, sends, hid, block, rstd, post, gate, pre, ds, outs[n], outs[:n], *grads, ws,
                                      comms(n))
        got.append(grads + outs)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(other, got[0]))


@pytest.mark.parametrize("n,rows,hidden", [(2, 4, 40), (1, 4, 301), (3, 3, 1024)])
def test_backward_against_differences_of_the_forward_pass(comms, n, rows, hidden):
    """dL of L = sum(y a) + sum(h c) along a random direction of each input, against the central
    difference of the kernel's own fp32 forward pass, within the step's third-order term (steps of
    d = 2^-5 along unit elements through two norms: allowed 32 d^2/6 of the products' magnitudes) and
    the outputs' fp32 rounding over d."""
    comm, gen = comms(n), torch.Generator().manual_seed(n * hidden)
    start = {"x": torch.randn(n, rows, hidden, generator=gen), "residual": torch.randn(rows, hidden, generator=gen) * 2}
    start["post"], start["gate"], start["pre"] = weights(hidden, F32, gen)
    a, c = (torch.randn(rows, hidden, generator=gen) for _ in range(2))
    alpha = 0.8
    desc = V.vBlockNormDesc(rows, hidden, F32, eps=EPS, residual_scale=alpha)

    def loss(i):
        y = [None] * (n - 1) + [torch.empty(rows, hidden, device=DEV)]
        h, b, rstd = torch.empty(rows, hidden, device=DEV), torch.empty(rows, hidden, device=DEV), torch.empty(2, rows, device=DEV)
        V.vAllReduceBlockNorm(desc, [place(t) for t in i["x"]], place(i["residual"]), place(i["post"]), place(i["gate"]),
                              place(i["pre"]), b, h, y, rstd, comm)
        return ((y[-1].double().cpu() * a).sum() + (h.double().cpu() * c).sum()).item(), h, b, rstd

    _, h, b, rstd = loss(start)
    # the gradient of y reaches the norm as n partial gradients that add up to a
    parts = torch.randn(n, rows, hidden, generator=gen)
    parts[-1] = a - parts[:-1].sum(0)
    ws = torch.empty(V.vBlockNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
    grads = [torch.empty(hidden, device=DEV) for _ in range(3)]
    db, dres = [torch.empty(rows, hidden, device=DEV) for _ in range(n)], torch.empty(rows, hidden, device=DEV)
    V.vAllReduceBlockNormBackward(desc, [place(p) for p in parts], h, b, rstd, place(start["post"]), place(start["gate"]),
                                  place(start["pre"]), place(c), dres, db, *grads, ws, comm)
    by = {"x": db[n // 2], "residual": dres, "post": grads[0], "gate": grads[1], "pre": grads[2]}
    d = 2.0 ** -5
    for what, grad in by.items():
        v = torch.randn(grad.shape, generator=gen)

        def at_step(s):
            moved = dict(start)
            if what == "x":
                moved["x"] = start["x"].clone()
                moved["x"][n // 2] += s * d * v
            else:
                moved[what] = start[what] + s * d * v
            return loss(moved)[0]

        numeric = (at_step(1) - at_step(-1)) / (2 * d)
        grad = grad.double().cpu()
        analytic, scale = (grad * v).sum().item(), (grad.abs() * v.abs()).sum().item()
        noise = 64 * R.U32 * (rows * hidden) ** 0.5 * 4 / d
        assert abs(numeric - analytic) <= 32 * d * d / 6 * scale + noise, what


# ---- streams, groups, graphs, refusals ---------------------------------------------------------

@pytest.mark.parametrize("rows,hidden", [(8, 2048), (2000, 1024)])
def test_on_other_streams_in_a_group_and_in_a_graph(comms, rows, hidden):
    n = 2
    comm, gen = comms(n), torch.Generator().manual_seed(41)
    xs, res = torch.randn(n, rows, hidden, generator=gen).to(BF16), torch.randn(rows, hidden, generator=gen).to(BF16)
    w = weights(hidden, BF16, gen)
    post, gate, pre = (place(t) for t in w)
    sends, dres = [place(x) for x in xs], place(res)
    desc = V.vBlockNormDesc(rows, hidden, BF16, eps=EPS, residual_scale=0.5)
    ref = B.forward(xs, res, *w, 0.5, EPS)

    def room():
        return ([torch.zeros(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)],
                *(torch.zeros(rows, hidden, dtype=BF16, device=DEV) for _ in range(2)), torch.zeros(2, rows, device=DEV))

    both = [(torch.cuda.Stream(), *room()) for _ in range(2)]
    torch.cuda.synchronize()
    for side, outs, b, h, rstd in both:
        V.vAllReduceBlockNorm(desc, sends, dres, post, gate, pre, b, h, outs, rstd, comm, stream=side)
    torch.cuda.synchronize()
    for _, outs, b, h, rstd in both:
        R.assert_close(outs[1], ref["y"], ref["dy"], BF16, "side stream")
    outs, b, h, rstd = room()
    V.vcommGroupStart(comm)
    V.vAllReduceBlockNorm(desc, list(sends), dres, post, gate, pre, b, h, list(outs), rstd, comm)
    torch.cuda.synchronize()
    assert (outs[1] == 0).all()                       # recorded, not run
    V.vcommGroupEnd(comm)
    R.assert_close(outs[1], ref["y"], ref["dy"], BF16, "group")

    # forward and backward captured together, replayed on new contents of the same buffers
    ws = torch.empty(V.vBlockNormBackwardWorkspace(desc, comm), dtype=torch.uint8, device=DEV)
    db, dr = [torch.empty(rows, hidden, dtype=BF16, device=DEV) for _ in range(n)], torch.empty(rows, hidden, dtype=BF16, device=DEV)
    grads = [torch.empty(hidden, dtype=BF16, device=DEV) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        V.vAllReduceBlockNorm(desc, sends, dres, post, gate, pre, b, h, outs, rstd, comm)
        V.vAllReduceBlockNormBackward(desc, outs, h, b, rstd, post, gate, pre, None, dr, db, *grads, ws, comm)
    for s, x in zip(sends, xs):
        s.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    ref = B.forward(xs.flip(1), res, *w, 0.5, EPS)
    R.assert_close(outs[0], ref["y"], ref["dy"], BF16, "replay")
    back = B.backward(torch.stack([o.cpu() for o in outs]), h.cpu(), b.cpu(), rstd.cpu(), *w, None, 0.5)
    R.assert_close(db[0], back["db"], back["ddb"], BF16, "replayed backward")
    R.assert_close(dr, back["dres"], back["ddres"], BF16, "replayed residual")
    for g, name in zip(grads, ("post", "gate", "pre")):
        R.assert_close(g, back[name], back["d" + name], BF16, name)


def test_refusals(comms):
    n, rows, hidden = 2, 4, 64
    comm = comms(n)
    bufs = [torch.full((rows, hidden), CANARY, dtype=BF16, device=DEV) for _ in range(6)]
    w, rstd = torch.ones(hidden, dtype=BF16, device=DEV), torch.ones(2, rows, device=DEV)
    good = dict(rows=rows, hidden=hidden, datatype=BF16)
    s, o = bufs[:2], bufs[2:4]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)

    def refused(call, *args):
        with pytest.raises(V.VcommError) as e:
            call(*args)
        assert e.value.code == V.vInvalidArgument

    for change in (dict(datatype=torch.int32), dict(hidden=65537), dict(rows=1 << 31), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(residual_scale=float("inf")), dict(residual_scale=float("nan")), dict(send_stride=63),
                   dict(residual_stride=1), dict(recv_stride=2), dict(weight_type=torch.float16)):
        d = V.vBlockNormDesc(**{**good, **change})
        refused(V.vAllReduceBlockNorm, d, s, None, w, None, w, None, None, o, None, comm)
        refused(V.vAllReduceBlockNormBackward, d, s, bufs[4], bufs[5], rstd, w, None, w, None, None, o, w, None, w, ws, comm)
        refused(V.vBlockNormBackwardWorkspace, d, comm)
    d = V.vBlockNormDesc(**good)
    odd = bufs[0].data_ptr() + 1
    fine = [s, None, w, None, w, None, None, o, None]
    for i, value in [(0, [None, bufs[1]]), (0, [odd, bufs[1]]), (0, s[:1]), (1, odd), (2, None), (2, odd), (3, odd), (4, None),
                     (4, odd), (5, odd), (6, odd), (7, [None, None]), (7, [odd, None]), (8, odd)]:
        refused(V.vAllReduceBlockNorm, d, *fine[:i], value, *fine[i + 1:], comm)
    need = V.vBlockNormBackwardWorkspace(d, comm)
    fine = [s, bufs[4], bufs[5], rstd, w, w, w, None, None, o, w, w, w, ws]
    for i, value in [(0, [None, bufs[1]]), (1, None), (1, odd), (2, None), (3, None), (4, None), (5, None), (5, odd), (6, None),
                     (7, odd), (8, odd), (9, [None, None]), (10, None), (10, odd), (11, None), (11, odd), (12, None),
                     (13, (None, 1 << 20)), (13, (ws.data_ptr(), need - 1)), (13, (ws.data_ptr() + 4, 1 << 19))]:
        refused(V.vAllReduceBlockNormBackward, d, *fine[:i], value, *fine[i + 1:], comm)
    torch.cuda.synchronize()
    assert all((b == CANARY).all() for b in bufs)
    assert V.vcommGetAsyncError(comm) == V.vSuccess
    V.vcommGroupStart(comm)
    V.vAllReduceBlockNorm(d, s, None, None, None, w, None, None, o, None, comm)
    refused(V.vcommGroupEnd, comm)
