"""Measured cases of the operators that run next to the collectives in a parallel training or
serving step: the all-reduce fused with the residual's addition and an RMS norm (its plain
and its 8-bit output), that norm's backward pass, and the global gradient norm with clipping.

A case's "op" names the operator.  Norm cases have ranks, rows, hidden, dtype, wtype (the
weight's type), residual (whether a residual stream is added), pad (elements between the rows
of the ranks' partial sums) and, for the 8-bit output, group (0: one scale a row).  Gradient
cases stand for a decoder of `layers` layers of width `width` and feed-forward width `ffn`,
whose matrices are split over the ranks and whose norm weights every rank holds.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
LEAST_AMAX = 2.0 ** -64        # a row or group of zeros gets this over 448 as its scale
CLIP_EPS = 1e-6
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
MOST_BYTES = 6e8               # of a drawn norm case
MOST_GRADS = 4e8               # elements of a drawn gradient case, all ranks

_comms: dict = {}


# ---- cases ---------------------------------------------------------------------------------

def _norm(op, name, ranks, rows, hidden, dtype, wtype, residual=True, pad=0, group=0):
    return {"op": op, "name": name, "ranks": ranks, "rows": rows, "hidden": hidden, "dtype": dtype,
            "wtype": wtype, "residual": residual, "pad": pad, "group": group}


def _grads(op, name, ranks, layers, width, ffn, dtype, vtype, max_norm=1.0):
    return {"op": op, "name": name, "ranks": ranks, "layers": layers, "width": width, "ffn": ffn,
            "dtype": dtype, "vtype": vtype, "max_norm": max_norm}


def listed():
    return [
        # one decoded token of a wide model on 8 ranks: all latency
        _norm("norm", "norm_token_8x1x8192_bf16", 8, 1, 8192, "bf16", "bf16"),
        # a long prompt on 8 ranks of 4096 tokens and hidden size 4096: all bandwidth
        _norm("norm", "norm_prompt_8x4096x4096_bf16", 8, 4096, 4096, "bf16", "bf16"),
        # an odd hidden size, where no row but the first starts on a 16-byte boundary
        _norm("norm", "norm_ragged_3x1537x2731_fp16", 3, 1537, 2731, "fp16", "fp32"),
        # a small decoding batch on 4 ranks, 8-bit output scaled by groups of 128
        _norm("quant", "quant_batch_4x24x5120_bf16", 4, 24, 5120, "bf16", "bf16", group=128),
        # a long prompt on one rank, 8-bit output with one scale a token
        _norm("quant", "quant_prompt_1x16384x4096_bf16", 1, 16384, 4096, "bf16", "bf16"),
        # the training step of the long prompt
        _norm("backward", "backward_8x4096x4096_bf16", 8, 4096, 4096, "bf16", "bf16"),
        # a training step in fp32 on one rank
        _norm("backward", "backward_1x8192x2048_fp32", 1, 8192, 2048, "fp32", "fp32"),
        # a small step with odd sizes
        _norm("backward", "backward_ragged_2x331x1001_fp16", 2, 331, 1001, "fp16", "fp32"),
        # the gradients of a toy model: all latency
        _grads("gradnorm", "gradnorm_small_1x2x64_bf16", 1, 2, 64, 171, "bf16", "fp32"),
        # reduce-scattered shards of 8 ranks
        _grads("gradnorm", "gradnorm_shards_8x4x2048_bf16", 8, 4, 2048, 8192, "bf16", "fp32"),
        # hundreds of small tensors of odd sizes on 2 ranks
        _grads("clip", "clip_many_2x96x65_fp32", 2, 96, 65, 173, "fp32", "fp32"),
        # half a billion fp32 gradients on one rank
        _grads("clip", "clip_large_1x8x2048_fp32", 1, 8, 2048, 8192, "fp32", "fp32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "quant", "backward", "backward", "gradnorm", "clip"])
    if op in ("gradnorm", "clip"):
        while True:
            case = _grads(op, "", rng.choice([1, 1, 2, 3, 4, 8]), _spread(rng, 1, 100), _spread(rng, 24, 4096),
                          0, rng.choice(["fp32", "bf16", "bf16", "fp16"]), rng.choice(["fp32", "bf16"]),
                          rng.choice([0.5, 1.0, 1e6]))
            case["ffn"] = int(case["width"] * rng.uniform(2.0, 4.5))
            if sum(map(sum, _sizes(case))) * case["ranks"] <= MOST_GRADS:
                break
    else:
        while True:
            dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            hidden = _spread(rng, 48, 16384)
            if rng.random() < 0.6:
                hidden = max(64, hidden // 64 * 64)
            case = _norm(op, "", rng.choice([1, 1, 2, 3, 4, 6, 8, 16]), _spread(rng, 1, 16384), hidden, dtype,
                         rng.choice([dtype, "fp32"]), rng.random() < 0.8, rng.choice([0, 0, 64, 5]),
                         rng.choice([0, 128]) if op == "quant" else 0)
            if work(case)["bytes"] <= MOST_BYTES:
                break
    del case["name"]
    return case


def _sizes(case):
    """Elements of each tensor that one rank holds: (pieces of split matrices, whole vectors)."""
    w, f, n = case["width"], case["ffn"], case["ranks"]
    layer = [-(-x // n) for x in (w * w, w * w, w * w, w * w, w * f, w * f, w * f)]
    return layer * case["layers"], [w, w] * case["layers"]


def _bytes_of(name):
    return 4 if name == "fp32" else 2


def work(case):
    n = case["ranks"]
    if case["op"] in ("gradnorm", "clip"):
        split, whole = (sum(s) for s in _sizes(case))
        # the norm reads every piece of a split tensor and one copy of a whole one
        read = n * split * _bytes_of(case["dtype"]) + whole * _bytes_of(case["vtype"])
        if case["op"] == "gradnorm":
            return {"bytes": read + 4, "flops": 2 * (n * split + whole)}
        both = n * (split * _bytes_of(case["dtype"]) + whole * _bytes_of(case["vtype"]))
        return {"bytes": 2 * both + 4, "flops": 3 * n * (split + whole)}
    t, h, e, we = case["rows"], case["hidden"], _bytes_of(case["dtype"]), _bytes_of(case["wtype"])
    if case["op"] == "backward":
        read = n * t * h * e + t * h * e * (2 if case["residual"] else 1) + 4 * t + h * we
        return {"bytes": read + n * t * h * e + h * we, "flops": t * h * (n + 9)}
    read = n * t * h * e + (t * h * e if case["residual"] else 0) + h * we
    write = t * h * e + 4 * t
    if case["op"] == "norm":
        write += n * t * h * e
    else:
        groups = -(-h // case["group"]) if case["group"] else 1
        write += n * (t * h + 4 * t * groups)
    return {"bytes": read + write, "flops": t * h * (n + 5)}


# ---- inputs --------------------------------------------------------------------------------

def _randn(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen).mul_(scale)


def _inputs(case, seed):
    """The tensors that a case starts from, made from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, dt = case["ranks"], DTYPES[case["dtype"]]
    if case["op"] in ("gradnorm", "clip"):
        split, whole = (sum(s) for s in _sizes(case))
        return {"split": _randn((n, split), dt, gen, 0.01),
                "whole": _randn((1, whole), DTYPES[case["vtype"]], gen, 0.1).repeat(n, 1)}
    t, h = case["rows"], case["hidden"]
    wide = _randn((n, t, h + case["pad"]), dt, gen, n ** -0.5)
    if case["op"] != "backward":
        wide[:, 3::97] = 0                        # tokens of padding
    got = {"wide": wide, "weight": (1 + 0.1 * torch.randn(h, device="cuda", generator=gen)).to(DTYPES[case["wtype"]])}
    stream = torch.randn((t, h), device="cuda", generator=gen)
    stream[:, 1::61] *= 20                        # a few channels of large values
    if case["op"] == "backward":
        got["hidden"] = stream.to(dt)
        got["rstd"] = (got["hidden"].float().square().mean(1) + EPS).rsqrt()
        if case["residual"]:
            got["grad"] = _randn((t, h), dt, gen)
    elif case["residual"]:
        stream[3::97] = 0
        got["residual"] = stream.to(dt)
    return got


def _communicator(n):
    from collective_communication_virtual_gb300 import vcomm as V
    if n not in _comms:
        _comms[n] = V.vcommInit(n)
    return _comms[n]


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if not own:
        return state
    from collective_communication_virtual_gb300 import vcomm as V
    n, dt = case["ranks"], DTYPES[case["dtype"]]
    comm = state["comm"] = _communicator(n)
    if case["op"] in ("gradnorm", "clip"):
        sizes, vsizes = _sizes(case)

        def pieces(split, whole):
            return [list(split[r].split(sizes)) + list(whole[r].split(vsizes)) for r in range(n)]

        state["norm"] = torch.empty(1, device="cuda")
        outs = None
        if case["op"] == "clip":
            state["out"] = [torch.empty_like(state["split"]), torch.empty_like(state["whole"])]
            outs = pieces(*state["out"])
        state["list"] = V.vTensorList(pieces(state["split"], state["whole"]), outs,
                                      replicated=[False] * len(sizes) + [True] * len(vsizes))
        state["workspace"] = torch.empty(V.vGradNormWorkspace(state["list"], comm), dtype=torch.uint8, device="cuda")
        return state
    t, h, pad = case["rows"], case["hidden"], case["pad"]
    state["desc"] = V.vRmsNormDesc(t, h, dt, DTYPES[case["wtype"]], eps=EPS, send_stride=h + pad,
                                   quant_group=case["group"])
    state["send"] = V.vBuffers(state["wide"][r] for r in range(n))
    out = torch.empty((n, t, h), dtype=torch.float8_e4m3fn if case["op"] == "quant" else dt, device="cuda")
    state["out"], state["recv"] = out, V.vBuffers(out[r] for r in range(n))
    if case["op"] == "backward":
        state["grad_weight"] = torch.empty_like(state["weight"])
        state["workspace"] = torch.empty(V.vRmsNormBackwardWorkspace(state["desc"], comm), dtype=torch.uint8,
                                         device="cuda")
        return state
    state["stream"] = torch.empty((t, h), dtype=dt, device="cuda")
    state["rstd"] = torch.empty(t, device="cuda")
    if case["op"] == "quant":
        groups = -(-h // case["group"]) if case["group"] else 1
        state["scales"] = torch.empty((n, t, groups), device="cuda")
        state["scale_bufs"] = V.vBuffers(state["scales"][r] for r in range(n))
    return state


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from collective_communication_virtual_gb300 import vcomm as V
    op, comm = s["case"]["op"], s["comm"]
    if op == "norm":
        V.vAllReduceRmsNorm(s["desc"], s["send"], s.get("residual"), s["weight"], s["stream"], s["recv"], s["rstd"],
                            comm)
        return {"normed": s["out"], "stream": s["stream"], "rstd": s["rstd"]}
    if op == "quant":
        V.vAllReduceRmsNormQuant(s["desc"], s["send"], s.get("residual"), s["weight"], s["stream"], s["recv"],
                                 s["scale_bufs"], s["rstd"], comm)
        return {"normed": s["out"], "scales": s["scales"], "stream": s["stream"], "rstd": s["rstd"]}
    if op == "backward":
        V.vAllReduceRmsNormBackward(s["desc"], s["send"], s["hidden"], s["rstd"], s["weight"], s.get("grad"),
                                    s["recv"], s["grad_weight"], s["workspace"], comm)
        return {"grad": s["out"], "grad_weight": s["grad_weight"]}
    if op == "gradnorm":
        V.vGradNorm(s["list"], s["norm"], s["workspace"], comm)
        return {"norm": s["norm"]}
    V.vClipGradNorm(s["list"], s["case"]["max_norm"], s["norm"], s["workspace"], comm)
    return {"norm": s["norm"], "split": s["out"][0], "whole": s["out"][1]}


def _run_plain(s):
    case = s["case"]
    n, op = case["ranks"], case["op"]
    if op in ("gradnorm", "clip"):
        total = s["split"].float().square().sum() + s["whole"][0].float().square().sum()
        norm = total.sqrt().reshape(1)
        if op == "gradnorm":
            return {"norm": norm}
        factor = (case["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
        return {"norm": norm, "split": (s["split"].float() * factor).to(s["split"].dtype),
                "whole": (s["whole"].float() * factor).to(s["whole"].dtype)}
    h, dt = case["hidden"], s["wide"].dtype
    x = s["wide"][:, :, :h].sum(0, dtype=torch.float32)
    weight = s["weight"].float()
    if op == "backward":
        xhat = s["hidden"].float() * s["rstd"][:, None]
        g = x * weight
        grad = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if case["residual"]:
            grad = grad + s["grad"].float()
        return {"grad": grad.to(dt).expand(n, -1, -1).contiguous(),
                "grad_weight": (x * xhat).sum(0).to(s["weight"].dtype)}
    if case["residual"]:
        x = x + s["residual"].float()
    rstd = 1.0 / (x.square().mean(1) + EPS).sqrt()
    normed = x * rstd[:, None] * weight
    if op == "norm":
        return {"normed": normed.to(dt).expand(n, -1, -1).contiguous(), "stream": x.to(dt), "rstd": rstd}
    t, group = case["rows"], case["group"] or h
    groups = -(-h // group)
    padded = torch.nn.functional.pad(normed, (0, groups * group - h)).view(t, groups, group)
    scales = padded.abs().amax(2).clamp(min=LEAST_AMAX) / E4M3_MAX
    q = (padded / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(t, -1)[:, :h].to(torch.float8_e4m3fn)
    return {"normed": q.view(torch.uint8).expand(n, -1, -1).contiguous().view(torch.float8_e4m3fn),
            "scales": scales.expand(n, -1, -1).contiguous(), "stream": x.to(dt), "rstd": rstd}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    n, op = case["ranks"], case["op"]
    if op in ("gradnorm", "clip"):
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for r in range(n):
            for piece in s["split"][r].split(1 << 26):
                total += torch.dot(piece.double(), piece.double())
        total += torch.dot(s["whole"][0].double(), s["whole"][0].double())
        norm = torch.sqrt(total)
        if op == "gradnorm":
            return {"norm": norm.reshape(1)}
        factor = min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
        return {"norm": norm.reshape(1), "split": torch.mul(s["split"].double(), factor),
                "whole": torch.mul(s["whole"].double(), factor)}
    t, h = case["rows"], case["hidden"]
    total = torch.zeros((t, h), dtype=torch.float64, device="cuda")
    for r in range(n):
        total += s["wide"][r, :, :h].double()
    weight = s["weight"].double()
    if op == "backward":
        rstd = s["rstd"].double()
        hidden = s["hidden"].double()
        inner = torch.einsum("th,h,th->t", total, weight, hidden)
        grad = torch.einsum("th,h,t->th", total, weight, rstd)
        grad -= hidden * (inner * rstd ** 3 / h)[:, None]
        if case["residual"]:
            grad += s["grad"].double()
        return {"grad": torch.stack([grad] * n), "grad_weight": torch.einsum("th,th,t->h", total, hidden, rstd)}
    if case["residual"]:
        total += s["residual"].double()
    rstd = torch.pow(torch.einsum("th,th->t", total, total) / h + EPS, -0.5)
    normed = torch.einsum("th,t,h->th", total, rstd, weight)
    if op == "norm":
        return {"normed": torch.stack([normed] * n), "stream": total, "rstd": rstd}
    columns = [normed[:, i:i + (case["group"] or h)] for i in range(0, h, case["group"] or h)]
    scales = [torch.linalg.vector_norm(c, ord=float("inf"), dim=1).clamp(min=LEAST_AMAX) / E4M3_MAX for c in columns]
    values = torch.cat([c / x[:, None] for c, x in zip(columns, scales)], 1)
    return {"normed": torch.stack([values] * n), "scales": torch.stack([torch.stack(scales, 1)] * n),
            "stream": total, "rstd": rstd}
