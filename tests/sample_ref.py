"""Sampling in 64 bits.

Weights are carried to d = 2^-28.8 of themselves, so a share s of a sum of them is off by at most
2 d s (1 - s) < 2^-29, and a weight next to the largest by d.  A drawn number within 2^-28 of a token's border
(in shares of the kept sum), and a filter whose border is that close to a running sum, may go either way:
`matches` accepts those, and nothing else.
"""
from __future__ import annotations

import math

import numpy as np

NEAR = 2.0 ** -28


def kept(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, slack=0.0):
    """64-bit weights e (of all tokens), and the tokens that the filters keep, as a mask.  slack moves
    topP's and minP's borders by that share."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    n = x.size
    top = x.max()
    greedy = not temperature > 0
    heat = 1.0 if greedy else float(np.float32(temperature))
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        e = np.where(x == top, 1.0, np.exp((x - top) / heat))
    if math.isinf(top):
        e = (x == top).astype(np.float64)
    order = np.lexsort((np.arange(n), -x))            # largest first, ties to the lower index
    count = 1 if greedy else n if top_k <= 0 else min(n, top_k)
    if not greedy and top_p < 1:
        mass = e[order[:count]].cumsum()
        goal = max(0.0, float(np.float32(top_p))) * mass[-1] * (1 + slack)
        before = np.concatenate([[0.0], mass[:-1]])
        count = max(1, int((before < goal).sum()))
    mask = np.zeros(n, dtype=bool)
    mask[order[:count]] = True
    if not greedy and min_p > 0:
        mask &= e >= min(1.0, float(np.float32(min_p))) * (1 - slack)
    return e, mask & (e > 0)


def draw(e, mask, u):
    """The token, and the borders of every token's share of the kept sum."""
    mass = np.where(mask, e, 0.0).cumsum()
    hi = mass / mass[-1]
    lo = np.concatenate([[0.0], hi[:-1]])
    u = min(max(float(u), 0.0), 1 - 2.0 ** -53) if u == u else 0.0
    return int(np.searchsorted(hi, u, side="right")), lo, hi, u


def logprob(e, logits, token, temperature):
    x = logits.astype(np.float64)
    top = np.nanmax(np.where(np.isnan(x), -np.inf, x))
    heat = float(np.float32(temperature)) if temperature > 0 else 1.0
    z = 0.0 if x[token] == top else (x[token] - top) / heat
    return z - math.log1p(e.sum() - 1.0)


def matches(token, logits, u, **filters):
    """Whether `token` may come of this row."""
    for slack in (0.0, NEAR, -NEAR):
        e, mask = kept(logits, **filters, slack=slack)
        want, lo, hi, u = draw(e, mask, u)
        if token == want or (0 <= token < e.size and mask[token] and lo[token] - NEAR <= u <= hi[token] + NEAR):
            return True
    return False
