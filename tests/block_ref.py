"""The block norm in 64 bits, and bounds on what fp32 arithmetic may differ (units as in norm_ref).

The first norm's bounds are norm_ref's; what they leave uncertain in h (dh) goes through the second
norm: its mean square is off by at most 2 rms(h) rms(dh), so its root by rms(dh) rstd relative.
"""
from __future__ import annotations

import torch

from tests import norm_ref as R

U32, CHAIN = R.U32, R.CHAIN


def forward(xs, residual, post, gate, pre, alpha, eps):
    """xs: [N, rows, hidden]; gate and residual may be None.  64-bit results and error bounds."""
    one = R.forward(xs, None, post if gate is None else post.double() * gate.double(), eps)
    h, dh = one["y"], one["dy"] + 4 * U32 * one["y"].abs()
    if residual is not None:
        kept = alpha * residual.double()
        dh = dh + 2 * U32 * (kept.abs() + h.abs())
        h = h + kept
    rstd = ((h * h).mean(1, keepdim=True) + eps).rsqrt()
    drstd = CHAIN * U32 + 2 * (dh * dh).mean(1, keepdim=True).sqrt() * rstd
    y = h * rstd * pre.double()
    dy = (dh * rstd + h.abs() * rstd * drstd) * pre.double().abs() + 4 * U32 * y.abs()
    return {"b": one["h"], "db": one["dh"], "r1": one["rstd"], "dr1": one["drstd"], "h": h, "dh": dh,
            "r2": rstd[:, 0], "dr2": (drstd * rstd)[:, 0], "y": y, "dy": dy}


def backward(dys, hidden, block, rstd, post, gate, pre, dstream, alpha):
    """rstd: [2, rows].  A sum of rows products is within (rows + 8) u of its terms' magnitudes, plus
    what the terms themselves are off by."""
    two = R.backward(dys, hidden, rstd[1], pre, dstream)
    dh, ddh = two["dh"], two["ddh"]
    r1 = rstd[0].double()[:, None]
    x1 = block.double() * r1
    scale = post.double() if gate is None else post.double() * gate.double()
    g = dh * scale
    dg = ddh * scale.abs() + 4 * U32 * g.abs()
    c = (g * x1).mean(1, keepdim=True)
    dc = (dg * x1.abs()).mean(1, keepdim=True) + CHAIN * U32 * (g * x1).abs().mean(1, keepdim=True)
    db = r1 * (g - x1 * c)
    ddb = r1.abs() * (dg + x1.abs() * dc + 8 * U32 * (g.abs() + (x1 * c).abs()))
    q = (dh * x1).sum(0)
    dq = (ddh * x1.abs()).sum(0) + (8 + dys.shape[1]) * U32 * (dh * x1).abs().sum(0)
    got = {"db": db, "ddb": ddb, "dres": alpha * dh, "ddres": abs(alpha) * (ddh + 2 * U32 * dh.abs()),
           "pre": two["dw"], "dpre": two["ddw"], "gate": None}
    if gate is None:
        return {**got, "post": q, "dpost": dq}
    got["post"], got["dpost"] = q * gate.double(), (dq + 4 * U32 * q.abs()) * gate.double().abs()
    return {**got, "gate": q * post.double(), "dgate": (dq + 4 * U32 * q.abs()) * post.double().abs()}
