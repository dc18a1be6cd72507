"""The norms and the clipping in 64 bits, and bounds on what fp32 arithmetic may differ.

u = 2^-24 is fp32's unit roundoff, U the output type's.  A sum of n fp32 terms in any order is
within n u of its value relative to the sum of the terms' magnitudes; products and roots add
a few u.  The bounds below are those, with the constants rounded up, plus U |value| for the one
rounding to the output type (and half of fp16's smallest step).
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
# terms that one thread adds in a row (32), the two shuffle trees (10), a cluster (8), and the
# roots, products and divisions after them
CHAIN = 64


def forward(xs, residual, weight, eps):
    """xs: [N, rows, hidden].  Returns a dict of 64-bit results and error bounds."""
    x = xs.double()
    h, mag = x.sum(0), x.abs().sum(0)
    if residual is not None:
        h = h + residual.double()
        mag = mag + residual.double().abs()
    n = xs.shape[0] + 1
    w = weight.double()
    mean = (h * h).mean(1, keepdim=True) + eps
    rstd = mean.rsqrt()
    y = h * rstd * w
    dh = n * U32 * mag                                     # of h
    drstd = CHAIN * U32 + n * U32 * (mag * mag).mean(1, keepdim=True).sqrt() * rstd * 2   # relative
    dy = (dh * rstd + h.abs() * rstd * drstd) * w.abs() + 4 * U32 * y.abs()
    return {"h": h, "dh": dh, "rstd": rstd[:, 0], "drstd": (drstd * rstd)[:, 0], "y": y, "dy": dy}


def assert_close(got, want, slack, dtype, what):
    got = got.double().cpu()
    want = want.cpu()
    bound = slack.cpu() * 1.01 + UNIT[dtype] * want.abs() * 1.01 + TINY[dtype]
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got {got[i].item()!r}, "
                             f"want {want[i].item()!r} within {bound[i].item():.3g}")


def group_amax(y, group):
    rows, hidden = y.shape
    if group == 0:
        return y.abs().amax(1, keepdim=True)
    return torch.stack([y[:, i:i + group].abs().amax(1) for i in range(0, hidden, group)], 1)


def per_element(per_group, hidden, group):
    if group == 0:
        return per_group.expand(-1, hidden)
    return per_group.repeat_interleave(group, 1)[:, :hidden]


def assert_quantised(q, scales, ref, group, what):
    """q: e4m3 values as double, scales as double, against the 64-bit y of `ref`."""
    y, dy = ref["y"].cpu(), ref["dy"].cpu()
    rows, hidden = y.shape
    amax = group_amax(y, group).clamp(min=2.0 ** -64)
    want = amax / 448
    damax = group_amax(dy, group) / 448 + 8 * U32 * want
    assert (scales - want).abs().le(damax * 1.01).all(), f"{what}: scales"
    s = per_element(want, hidden, group)
    v = y / s
    # half the spacing of e4m3 at the value (2^-10 below its normals), plus the fp32 error of v
    # (8 u of it again, for the scale's and the factor's roundings)
    slack = dy / s + v.abs() * (per_element(damax / want, hidden, group) + 16 * U32)
    reach = (v.abs() + slack).clamp(max=448.0)
    spacing = torch.pow(2.0, torch.floor(torch.log2(reach.clamp(min=2.0 ** -6))) - 3)
    off = (q - v).abs()
    bad = ~(off <= spacing / 2 + slack)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} e4m3 values outside, first at {i}: got {q[i].item()!r}, "
                             f"want {v[i].item()!r}")


def backward(dys, hidden, rstd, weight, dres):
    d = dys.double()
    dy, mag = d.sum(0), d.abs().sum(0)
    n = dys.shape[0] + 1
    w, r = weight.double(), rstd.double()[:, None]
    xhat = hidden.double() * r
    g, gm = dy * w, mag * w.abs()
    c = (g * xhat).mean(1, keepdim=True)
    cm = (gm * xhat.abs()).mean(1, keepdim=True)
    dh = r * (g - xhat * c)
    slack = (n + CHAIN) * U32 * r.abs() * (gm + xhat.abs() * cm)
    if dres is not None:
        dh = dh + dres.double()
        slack = slack + 2 * U32 * dres.double().abs() + 2 * U32 * dh.abs()
    dw = (dy * xhat).sum(0)
    dslack = (n + 8 + dys.shape[1]) * U32 * (mag * xhat.abs()).sum(0)
    return {"dh": dh, "ddh": slack, "dw": dw, "ddw": dslack}


# norm of gradients: at most 64 squares are added in fp32 (16 in each of 4 chains, then 2
# additions), the rest in fp64; half of that after the root, then one rounding
NORM_REL = 16 * U32
# the factor adds a sum, a quotient and the product
CLIP_REL = NORM_REL + 4 * U32


def grad_norm(tensors):
    return torch.stack([t.double().square().sum() for t in tensors] or [torch.zeros((), dtype=torch.float64)]).sum().sqrt()
