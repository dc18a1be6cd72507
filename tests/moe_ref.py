"""The experts' layer in 64 bits, and bounds on what fp32 arithmetic may differ.

A sum of n products in fp32 is within n u of its value relative to the products' magnitudes where the
additions round (u = 2^-24), and within 2 n u where they cut off, as a matrix unit may.  silu has a
slope of at most 1.1.  What goes into the way down is in fp32, or, next to 16-bit weights, the sum of
two values of the weights' type: the first is off by half a step of that type, the second by half a
step of what is left, 2^-18 of the value (bf16), or 2^-25 where the type ends (fp16).
"""
from __future__ import annotations

import torch

from tests import norm_ref as R

U32 = R.U32
SPLIT = {torch.float32: (0.0, 0.0), torch.bfloat16: (2.0 ** -18, 0.0), torch.float16: (2.0 ** -22, 2.0 ** -25)}


def held(experts, ranks, rank):
    share = -(-experts // ranks)
    return range(min(rank * share, experts), min((rank + 1) * share, experts))


def layer(x, ids, weights, up, down):
    """x: [T, H]; ids, weights: [T, K]; up, down: every rank's [experts, 2F, H] and [experts, H, F].
    Returns each rank's partial sums and their bounds, [N, T, H]."""
    ranks, (t, h), k = len(up), x.shape, ids.shape[1]
    rel, tiny = SPLIT[x.dtype]
    x64, w64 = x.double(), weights.double()
    out = torch.zeros(ranks, t, h, dtype=torch.float64)
    slack = torch.zeros_like(out)
    share = -(-sum(u.shape[0] for u in up) // ranks)
    for r in range(ranks):
        for i in range(up[r].shape[0]):
            tokens, places = (ids == r * share + i).nonzero(as_tuple=True)
            if tokens.numel() == 0:
                continue
            wide, mag = x64[tokens] @ up[r][i].double().t(), x64[tokens].abs() @ up[r][i].double().abs().t()
            f = wide.shape[1] // 2
            dwide = 2 * h * U32 * mag
            g, u = wide[:, :f], wide[:, f:]
            s = g / (1 + (-g).exp())
            a = s * u
            da = (1.1 * dwide[:, :f] + 8 * U32 * s.abs()) * (u.abs() + dwide[:, f:]) + s.abs() * dwide[:, f:]
            da = da + 4 * U32 * a.abs() + rel * a.abs() + tiny
            d = down[r][i].double()
            y, ym = a @ d.t(), a.abs() @ d.abs().t()
            dy = da @ d.abs().t() + 2 * 2 * f * U32 * ym
            w = w64[tokens, places][:, None]
            out[r].index_add_(0, tokens, w * y)
            slack[r].index_add_(0, tokens, w.abs() * (dy + (k + 2) * U32 * ym))
    return out, slack
