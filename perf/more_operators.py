"""Measured cases of what a parallel decoder runs between its products: the all-reduce fused with
the norms after and before a block, its gate and the residual's scale, with its backward pass;
the router of a mixture of experts and its experts' layer for a few tokens, the experts split over
the ranks; and sampling from logits whose vocabulary is split over the ranks.

A case's "op" names the operator.  "ranks" is the number of virtual ranks.  Block norm cases have
rows, hidden, dtype, wtype (the weights' type), gate (whether there is one), alpha (the residual's
scale) and pad (elements between the rows of the ranks' partial sums).  Mixture cases have rows
(tokens), hidden, ffn (an expert's inner width), experts, topk, dtype and, for the router, wtype
and whether the weights are normalised over the chosen.  Sampling cases have rows, vocab, dtype and
which of the filters are given.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
MOST_NORM = 6e8                # bytes of a drawn block norm
MOST_EXPERTS = 4.5e9           # bytes of drawn experts, all of them
MOST_LOGITS = 256 * 131072     # of a drawn sampling case
OPS = ["norm", "norm", "backward", "backward", "route", "experts", "experts", "sample", "sample"]

_comms: dict = {}


# ---- cases ---------------------------------------------------------------------------------

def _norm(op, name, ranks, rows, hidden, dtype, wtype, gate=True, alpha=1.0, pad=0):
    return {"op": op, "name": name, "ranks": ranks, "rows": rows, "hidden": hidden, "dtype": dtype,
            "wtype": wtype, "gate": gate, "alpha": alpha, "pad": pad}


def _route(name, rows, hidden, experts, topk, dtype, wtype, normalize=True, bias=False):
    return {"op": "route", "name": name, "ranks": 1, "rows": rows, "hidden": hidden, "ffn": 64, "experts": experts,
            "topk": topk, "dtype": dtype, "wtype": wtype, "normalize": normalize, "bias": bias}


def _experts(name, ranks, rows, hidden, ffn, experts, topk, dtype):
    return {"op": "experts", "name": name, "ranks": ranks, "rows": rows, "hidden": hidden, "ffn": ffn,
            "experts": experts, "topk": topk, "dtype": dtype}


def _sample(name, ranks, rows, vocab, dtype, topk=True, topp=True, minp=False, pad=0):
    return {"op": "sample", "name": name, "ranks": ranks, "rows": rows, "vocab": vocab, "dtype": dtype,
            "topk": topk, "topp": topp, "minp": minp, "pad": pad}


def listed():
    return [
        # one decoded token of a wide model on 8 ranks: all latency
        _norm("norm", "block_token_8x1x8192_bf16", 8, 1, 8192, "bf16", "bf16"),
        # a long prompt on 8 ranks of 4096 tokens and hidden size 4096: all bandwidth
        _norm("norm", "block_prompt_8x4096x4096_bf16", 8, 4096, 4096, "bf16", "bf16", alpha=0.5),
        # the training step of the long prompt
        _norm("backward", "block_backward_8x4096x4096_bf16", 8, 4096, 4096, "bf16", "bf16", alpha=0.5),
        # a training step of odd sizes, where no row but the first starts on a 16-byte boundary
        _norm("backward", "block_backward_3x1537x2731_fp16", 3, 1537, 2731, "fp16", "fp32", alpha=0.7),
        # the router for one decoded token
        _route("route_token_1x4096_of_64_bf16", 1, 4096, 64, 4, "bf16", "bf16"),
        # the router for a decoding batch, fp32 weights and a balancing bias
        _route("route_batch_256x4096_of_128_bf16", 256, 4096, 128, 8, "bf16", "fp32", normalize=False, bias=True),
        # one decoded token: four experts of 64
        _experts("experts_token_4x1x2048x1024_bf16", 4, 1, 2048, 1024, 64, 4, "bf16"),
        # a decoding batch that reaches nearly all of 128 experts
        _experts("experts_batch_8x64x4096x1536_bf16", 8, 64, 4096, 1536, 128, 8, "bf16"),
        # odd sizes, where no expert's rows are aligned
        _experts("experts_ragged_3x13x1001x333_fp16", 3, 13, 1001, 333, 10, 3, "fp16"),
        # one sequence: all latency
        _sample("sample_token_8x1x131072_bf16", 8, 1, 131072, "bf16"),
        # a large decoding batch
        _sample("sample_batch_8x256x131072_bf16", 8, 256, 131072, "bf16"),
        # an odd vocabulary in fp32, every filter
        _sample("sample_ragged_3x33x50001_fp32", 3, 33, 50001, "fp32", minp=True, pad=3),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _even(rng, size, to):
    return max(to, size // to * to) if rng.random() < 0.6 else size


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    ranks = rng.choice([1, 1, 2, 3, 4, 6, 8])
    while True:
        if op in ("norm", "backward"):
            case = _norm(op, "", ranks, _spread(rng, 1, 16384), _even(rng, _spread(rng, 48, 16384), 64), dtype,
                         rng.choice([dtype, "fp32"]), rng.random() < 0.7, round(rng.uniform(0.2, 1.5), 3),
                         rng.choice([0, 0, 64, 5]))
            if work(case)["bytes"] <= MOST_NORM:
                break
        elif op == "route":
            experts = _spread(rng, 8, 512)
            case = _route("", _spread(rng, 1, 512), _even(rng, _spread(rng, 64, 8192), 64), experts,
                          rng.randint(1, min(12, experts)), dtype, rng.choice([dtype, "fp32"]), rng.random() < 0.5,
                          rng.random() < 0.5)
            if case["rows"] * case["hidden"] * experts <= 256 * 4096 * 128:
                break
        elif op == "experts":
            experts = _spread(rng, 4, 128)
            case = _experts("", ranks, _spread(rng, 1, 96), _even(rng, _spread(rng, 128, 6144), 64),
                            _even(rng, _spread(rng, 64, 4096), 64), experts, rng.randint(1, min(8, experts)), dtype)
            if 3 * experts * case["hidden"] * case["ffn"] * _bytes_of(dtype) <= MOST_EXPERTS and \
                    case["rows"] * case["topk"] * case["hidden"] * case["ffn"] <= 64 * 8 * 4096 * 1536 // 2:
                break
        else:
            case = _sample("", ranks, _spread(rng, 1, 512), _spread(rng, 1000, 262144), dtype, rng.random() < 0.6,
                           rng.random() < 0.6, rng.random() < 0.4, rng.choice([0, 0, 8, 3]))
            if case["rows"] * case["vocab"] <= MOST_LOGITS:
                break
    del case["name"]
    return case


def _bytes_of(name):
    return 4 if name == "fp32" else 2


def work(case):
    n, t, e = case["ranks"], case["rows"], _bytes_of(case["dtype"])
    if case["op"] == "sample":
        filters = case["topk"] + case["topp"] + case["minp"]
        return {"bytes": t * case["vocab"] * e + 4 * t * (2 + filters) + 4 * t * (n + 1), "flops": 4 * t * case["vocab"]}
    h = case["hidden"]
    if case["op"] == "route":
        return {"bytes": t * h * e + case["experts"] * h * _bytes_of(case["wtype"]) + 8 * t * case["topk"],
                "flops": 2 * t * h * case["experts"]}
    if case["op"] == "experts":
        f, k = case["ffn"], case["topk"]
        hit = case["experts"] * (1.0 - (1.0 - k / case["experts"]) ** t)      # experts that some token chose, on average
        return {"bytes": int(3 * hit * h * f * e) + t * h * e + 8 * t * k + n * t * h * e, "flops": 6 * t * k * h * f}
    we = _bytes_of(case["wtype"]) * (3 if case["gate"] else 2)
    if case["op"] == "backward":
        read = n * t * h * e + 3 * t * h * e + 8 * t + h * we
        return {"bytes": read + n * t * h * e + t * h * e + h * we, "flops": t * h * (n + 20)}
    read = n * t * h * e + t * h * e + h * we
    return {"bytes": read + n * t * h * e + 2 * t * h * e + 8 * t, "flops": t * h * (n + 10)}


# ---- inputs --------------------------------------------------------------------------------

def _randn(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen).mul_(scale)


def _norm_inputs(case, gen):
    n, t, h, dt, wt = case["ranks"], case["rows"], case["hidden"], DTYPES[case["dtype"]], DTYPES[case["wtype"]]
    got = {"wide": _randn((n, t, h + case["pad"]), dt, gen, n ** -0.5)}
    got["post"] = (1 + 0.1 * _randn((h,), torch.float32, gen)).to(wt)
    got["pre"] = (1 + 0.1 * _randn((h,), torch.float32, gen)).to(wt)
    got["gate"] = (0.5 + 0.2 * _randn((h,), torch.float32, gen)).to(wt) if case["gate"] else None
    stream = _randn((t, h), torch.float32, gen)
    stream[:, 1::61] *= 20                        # a few channels of large values
    if case["op"] == "norm":
        got["wide"][:, 3::97] = 0                 # tokens of padding
        stream[3::97] = 0
        got["residual"] = stream.to(dt)
        return got
    # what the forward pass kept
    got["hidden"], got["block"] = stream.to(dt), _randn((t, h), dt, gen)
    got["rstd"] = torch.stack([(x.float().square().mean(1) + EPS).rsqrt() for x in (got["block"], got["hidden"])])
    got["grad"] = _randn((t, h), dt, gen)
    return got


def _held(case, rank):
    """The experts that a rank holds: equal shares, the last ones smaller."""
    share = -(-case["experts"] // case["ranks"])
    return range(min(rank * share, case["experts"]), min((rank + 1) * share, case["experts"]))


def _experts_inputs(case, gen):
    t, h, f, dt = case["rows"], case["hidden"], case["ffn"], DTYPES[case["dtype"]]
    got = {"x": _randn((t, h), dt, gen)}
    score = torch.rand((t, case["experts"]), device="cuda", generator=gen)
    got["ids"] = score.topk(case["topk"], 1).indices.to(torch.int32)
    got["weights"] = torch.softmax(_randn((t, case["topk"]), torch.float32, gen), 1)
    # a rank's experts: the gate's rows, then the linear part's, and the way down
    got["up"] = [_randn((len(_held(case, r)), 2 * f, h), dt, gen, h ** -0.5) for r in range(case["ranks"])]
    got["down"] = [_randn((len(_held(case, r)), h, f), dt, gen, f ** -0.5) for r in range(case["ranks"])]
    return got


def _sample_inputs(case, gen):
    n, t, v, dt = case["ranks"], case["rows"], case["vocab"], DTYPES[case["dtype"]]
    part = -(-v // n)
    whole = _randn((t, n * part), torch.float32, gen, 2.0)
    # a few tokens stand out in every row, by different amounts; some are ruled out
    peaks = torch.randint(0, v, (t, 24), device="cuda", generator=gen)
    whole.scatter_add_(1, peaks, 4 + 6 * torch.rand((t, 24), device="cuda", generator=gen))
    whole[:, 7::1001] = -math.inf
    wide = torch.zeros((n, t, part + case["pad"]), dtype=dt, device="cuda")
    wide[:, :, :part] = whole.view(t, n, part).transpose(0, 1).to(dt)
    rows = torch.arange(t, device="cuda")
    got = {"wide": wide, "uniform": torch.rand(t, device="cuda", generator=gen)}
    got["temperature"] = 0.6 + 0.6 * torch.rand(t, device="cuda", generator=gen)
    got["temperature"][5::16] = 0                 # greedy rows
    got["topk"] = got["topp"] = got["minp"] = None
    if case["topk"]:
        got["topk"] = torch.tensor([50, 20, 0, 200], dtype=torch.int32, device="cuda")[rows % 4]
    if case["topp"]:
        got["topp"] = torch.tensor([0.9, 0.95, 0.8], device="cuda")[rows % 3]
    if case["minp"]:
        got["minp"] = torch.tensor([0.05, 0.0], device="cuda")[rows % 2]
    return got


def _inputs(case, seed):
    """The tensors that a case starts from, made from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("norm", "backward"):
        return _norm_inputs(case, gen)
    if case["op"] == "experts":
        return _experts_inputs(case, gen)
    if case["op"] == "sample":
        return _sample_inputs(case, gen)
    t, h, e = case["rows"], case["hidden"], case["experts"]
    return {"x": _randn((t, h), DTYPES[case["dtype"]], gen),
            "router": _randn((e, h), DTYPES[case["wtype"]], gen, h ** -0.5),
            "bias": _randn((e,), torch.float32, gen, 0.1) if case["bias"] else None}


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
    n, t, dt, op = case["ranks"], case["rows"], DTYPES[case["dtype"]], case["op"]
    comm = state["comm"] = _communicator(n)

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "sample":
        v, pad = case["vocab"], case["pad"]
        part = -(-v // n)
        state["desc"] = V.vSampleDesc(t, v, dt, stride=part + pad)
        state["logits"] = V.vBuffers(state["wide"][r] for r in range(n))
        state["tokens"], state["logprob"] = empty(n, t, dtype=torch.int32), empty(t, dtype=torch.float32)
        state["recv"] = V.vBuffers(state["tokens"][r] for r in range(n))
        return state
    h = case["hidden"]
    if op in ("norm", "backward"):
        state["desc"] = V.vBlockNormDesc(t, h, dt, DTYPES[case["wtype"]], eps=EPS, residual_scale=case["alpha"],
                                         send_stride=h + case["pad"])
        state["send"] = V.vBuffers(state["wide"][r] for r in range(n))
        state["out"] = empty(n, t, h)
        state["recv"] = V.vBuffers(state["out"][r] for r in range(n))
        state["stream"] = empty(t, h)
        if op == "norm":
            state["block"], state["rstd"] = empty(t, h), empty(2, t, dtype=torch.float32)
            return state
        state["grad_post"], state["grad_pre"] = torch.empty_like(state["post"]), torch.empty_like(state["pre"])
        state["grad_gate"] = torch.empty_like(state["gate"]) if case["gate"] else None
        state["workspace"] = empty(V.vBlockNormBackwardWorkspace(state["desc"], comm), dtype=torch.uint8)
        return state
    state["desc"] = V.vMoeDesc(t, h, case["ffn"], case["experts"], case["topk"], dt,
                               DTYPES[case["wtype"]] if op == "route" else None,
                               normalize=case["normalize"] if op == "route" else True)
    if op == "route":
        state["ids"], state["weights"] = empty(t, case["topk"], dtype=torch.int32), empty(t, case["topk"], dtype=torch.float32)
        return state
    state["out"] = empty(n, t, h)
    state["recv"] = V.vBuffers(state["out"][r] for r in range(n))
    state["up_bufs"], state["down_bufs"] = V.vBuffers(state["up"]), V.vBuffers(state["down"])
    state["workspace"] = empty(V.vMoeExpertsWorkspace(state["desc"], comm), dtype=torch.uint8)
    return state


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "backward": _plain_backward, "route": _plain_route, "experts": _plain_experts,
            "sample": _plain_sample}[state["case"]["op"]](state)


def _run_own(s):
    from collective_communication_virtual_gb300 import vcomm as V
    op, comm = s["case"]["op"], s["comm"]
    if op == "norm":
        V.vAllReduceBlockNorm(s["desc"], s["send"], s["residual"], s["post"], s["gate"], s["pre"], s["block"], s["stream"],
                              s["recv"], s["rstd"], comm)
        return {"normed": s["out"], "stream": s["stream"], "block": s["block"], "rstd": s["rstd"]}
    if op == "backward":
        V.vAllReduceBlockNormBackward(s["desc"], s["send"], s["hidden"], s["block"], s["rstd"], s["post"], s["gate"],
                                      s["pre"], s["grad"], s["stream"], s["recv"], s["grad_post"], s["grad_gate"],
                                      s["grad_pre"], s["workspace"], comm)
        return {"grad": s["out"], "residual": s["stream"], "post": s["grad_post"], "gate": s["grad_gate"],
                "pre": s["grad_pre"]}
    if op == "route":
        V.vMoeRoute(s["desc"], s["x"], s["router"], s["bias"], s["ids"], s["weights"], comm)
        return {"ids": s["ids"], "weights": s["weights"]}
    if op == "experts":
        V.vMoeExperts(s["desc"], s["x"], s["ids"], s["weights"], s["up_bufs"], s["down_bufs"], s["recv"], s["workspace"], comm)
        return {"partial": s["out"]}
    V.vSample(s["desc"], s["logits"], s["temperature"], s["topk"], s["topp"], s["minp"], s["uniform"], s["recv"],
              s["logprob"], comm)
    return {"tokens": s["tokens"], "logprob": s["logprob"]}


def _plain_norm(s):
    case = s["case"]
    n, h, dt = case["ranks"], case["hidden"], s["wide"].dtype
    block = s["wide"][:, :, :h].sum(0, dtype=torch.float32)
    r1 = 1.0 / (block.square().mean(1) + EPS).sqrt()
    x = block * r1[:, None] * s["post"].float()
    if s["gate"] is not None:
        x = x * s["gate"].float()
    x = x + case["alpha"] * s["residual"].float()
    r2 = 1.0 / (x.square().mean(1) + EPS).sqrt()
    normed = (x * r2[:, None] * s["pre"].float()).to(dt)
    return {"normed": normed.expand(n, -1, -1).contiguous(), "stream": x.to(dt), "block": block.to(dt),
            "rstd": torch.stack([r1, r2])}


def _plain_backward(s):
    case = s["case"]
    n, h, dt, wt = case["ranks"], case["hidden"], s["wide"].dtype, s["post"].dtype
    dy = s["wide"][:, :, :h].sum(0, dtype=torch.float32)
    r1, r2 = s["rstd"][0][:, None], s["rstd"][1][:, None]
    x1, x2 = s["block"].float() * r1, s["hidden"].float() * r2
    g2 = dy * s["pre"].float()
    dh = r2 * (g2 - x2 * (g2 * x2).mean(1, keepdim=True)) + s["grad"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    g1 = dh * (s["post"].float() * gate)
    db = r1 * (g1 - x1 * (g1 * x1).mean(1, keepdim=True))
    q = (dh * x1).sum(0)
    return {"grad": db.to(dt).expand(n, -1, -1).contiguous(), "residual": (case["alpha"] * dh).to(dt),
            "post": (q * gate).to(wt), "gate": None if s["gate"] is None else (q * s["post"].float()).to(wt),
            "pre": (dy * x2).sum(0).to(wt)}


def _plain_route(s):
    # 64 bits, as two experts' logits may be next to one another
    logits = s["x"].double() @ s["router"].double().t()
    score = logits if s["bias"] is None else logits + s["bias"].double()
    ids = score.sort(dim=1, descending=True, stable=True).indices[:, :s["case"]["topk"]]
    chosen = logits.gather(1, ids)
    e = (chosen - chosen.amax(1, keepdim=True)).exp()
    total = e.sum(1, keepdim=True)
    if not s["case"]["normalize"]:
        total = (logits - chosen.amax(1, keepdim=True)).exp().sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (e / total).float()}


def _plain_experts(s):
    case, dt = s["case"], s["x"].dtype
    f, x = case["ffn"], s["x"].float()
    out = torch.zeros((case["ranks"], *x.shape), device="cuda")
    for r in range(case["ranks"]):
        for i, expert in enumerate(_held(case, r)):
            share = (s["weights"] * (s["ids"] == expert)).sum(1)
            rows = share.nonzero()[:, 0]
            if rows.numel() == 0:
                continue
            wide = x[rows] @ s["up"][r][i].float().t()
            gated = wide[:, :f] / (1 + (-wide[:, :f]).exp()) * wide[:, f:]
            out[r, rows] += share[rows, None] * (gated @ s["down"][r][i].float().t())
    return {"partial": out.to(dt)}


def _plain_sample(s):
    case = s["case"]
    n, t, v = case["ranks"], case["rows"], case["vocab"]
    part = -(-v // n)
    # 64 bits, as the number drawn may be next to a token's border
    logits = s["wide"][:, :, :part].transpose(0, 1).reshape(t, n * part)[:, :v].double()
    greedy = s["temperature"] <= 0
    values, order = logits.sort(dim=1, descending=True, stable=True)
    heat = torch.where(greedy, 1.0, s["temperature"].double())[:, None]
    e = ((values - values[:, :1]) / heat).exp()
    place = torch.arange(v, device="cuda")
    keep = torch.ones_like(e, dtype=torch.bool)
    if s["topk"] is not None:
        keep &= place < torch.where(s["topk"] > 0, s["topk"], v)[:, None]
    if s["topp"] is not None:
        mass = torch.where(keep, e, 0.0).cumsum(1)
        keep[:, 1:] &= mass[:, :-1] < s["topp"].double()[:, None] * mass[:, -1:]
    if s["minp"] is not None:
        keep &= e >= s["minp"].double()[:, None]
    keep &= ~greedy[:, None] | (place == 0)
    # the draw goes through the vocabulary in its own order
    kept = torch.zeros_like(e).scatter_(1, order, torch.where(keep, e, 0.0))
    mass = kept.cumsum(1)
    token = (mass <= s["uniform"].double()[:, None] * mass[:, -1:]).sum(1)
    z = (logits.gather(1, token[:, None]) - values[:, :1]) / heat
    logprob = z[:, 0] - e.sum(1).log()
    return {"tokens": token.to(torch.int32).expand(n, -1).contiguous(), "logprob": logprob.float()}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "backward": _exact_backward, "route": _exact_route, "experts": _exact_experts,
            "sample": _exact_sample}[case["op"]](case, s)


def _sum_of_ranks(case, s):
    total = torch.zeros((case["rows"], case["hidden"]), dtype=torch.float64, device="cuda")
    for r in range(case["ranks"]):
        total += s["wide"][r, :, :case["hidden"]].double()
    return total


def _exact_norm(case, s):
    n, h = case["ranks"], case["hidden"]
    block = _sum_of_ranks(case, s)
    r1 = torch.pow(torch.einsum("th,th->t", block, block) / h + EPS, -0.5)
    scale = s["post"].double()
    if s["gate"] is not None:
        scale = scale * s["gate"].double()
    stream = torch.einsum("th,t,h->th", block, r1, scale).add_(s["residual"].double(), alpha=case["alpha"])
    r2 = torch.pow(torch.einsum("th,th->t", stream, stream) / h + EPS, -0.5)
    normed = torch.einsum("th,t,h->th", stream, r2, s["pre"].double())
    return {"normed": torch.stack([normed] * n), "stream": stream, "block": block, "rstd": torch.stack([r1, r2])}


def _exact_backward(case, s):
    n, h = case["ranks"], case["hidden"]
    dy, hidden, block = _sum_of_ranks(case, s), s["hidden"].double(), s["block"].double()
    r1, r2 = s["rstd"].double()
    pre, post = s["pre"].double(), s["post"].double()
    dh = torch.einsum("th,h,t->th", dy, pre, r2)
    dh -= hidden * (torch.einsum("th,h,th->t", dy, pre, hidden) * r2 ** 3 / h)[:, None]
    dh += s["grad"].double()
    scale = post if s["gate"] is None else post * s["gate"].double()
    db = torch.einsum("th,h,t->th", dh, scale, r1)
    db -= block * (torch.einsum("th,h,th->t", dh, scale, block) * r1 ** 3 / h)[:, None]
    q = torch.einsum("th,th,t->h", dh, block, r1)
    return {"grad": torch.stack([db] * n), "residual": torch.mul(dh, case["alpha"]),
            "post": q if s["gate"] is None else q * s["gate"].double(), "gate": None if s["gate"] is None else q * post,
            "pre": torch.einsum("th,th,t->h", dy, hidden, r2)}


def _exact_route(case, s):
    logits = torch.einsum("th,eh->te", s["x"].double(), s["router"].double()).cpu()
    bias = torch.zeros(case["experts"], dtype=torch.float64) if s["bias"] is None else s["bias"].double().cpu()
    ids, weights = [], []
    for row in logits:
        score = (row + bias).tolist()
        chosen = sorted(range(case["experts"]), key=lambda i: (-score[i], i))[:case["topk"]]
        over = chosen if case["normalize"] else list(range(case["experts"]))
        ids.append(chosen)
        weights.append(torch.exp(row[chosen] - torch.logsumexp(row[over], 0)))
    return {"ids": torch.tensor(ids, dtype=torch.int32).cuda(), "weights": torch.stack(weights).cuda()}


def _exact_experts(case, s):
    t, k = s["ids"].shape
    x, f = s["x"].double(), case["ffn"]
    out = torch.zeros((case["ranks"], *x.shape), dtype=torch.float64, device="cuda")
    flat = s["ids"].flatten().tolist()
    for r in range(case["ranks"]):
        for i, expert in enumerate(_held(case, r)):
            slots = [j for j, e in enumerate(flat) if e == expert]
            if not slots:
                continue
            rows = torch.tensor([j // k for j in slots], device="cuda")
            up = s["up"][r][i].double()
            left, right = torch.nn.functional.linear(x[rows], up[:f]), torch.nn.functional.linear(x[rows], up[f:])
            y = torch.nn.functional.linear(left * torch.sigmoid(left) * right, s["down"][r][i].double())
            share = s["weights"].flatten()[torch.tensor(slots, device="cuda")].double()
            out[r].index_add_(0, rows, y * share[:, None])
    return {"partial": out}


def _exact_sample(case, s):
    n, v = case["ranks"], case["vocab"]
    part = -(-v // n)
    tokens, logprobs = [], []
    for t in range(case["rows"]):
        z = torch.cat([s["wide"][r, t, :part] for r in range(n)])[:v].double()
        heat = float(s["temperature"][t])
        z = torch.log_softmax(z / heat if heat > 0 else z, 0)
        order = z.sort(descending=True, stable=True).indices
        p = z[order].exp()
        count = v
        if s["topk"] is not None and int(s["topk"][t]) > 0:
            count = min(v, int(s["topk"][t]))
        if s["topp"] is not None:
            mass = p[:count].cumsum(0)
            count = min(count, 1 + int(torch.searchsorted(mass, float(s["topp"][t]) * mass[-1], right=False)))
        if s["minp"] is not None:
            count = min(count, int((p >= float(s["minp"][t]) * p[0]).sum()))
        kept = order[:1 if heat <= 0 else count].sort().values
        mass = z[kept].exp().cumsum(0)
        token = kept[torch.searchsorted(mass, float(s["uniform"][t]) * mass[-1:], right=True).clamp(max=len(kept) - 1)]
        tokens.append(token)
        logprobs.append(z[token])
    tokens = torch.cat(tokens).to(torch.int32)
    return {"tokens": tokens.expand(n, -1).contiguous(), "logprob": torch.cat(logprobs)}
