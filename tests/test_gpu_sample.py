"""Sampling from logits split over the ranks, against the definition in 64 bits: every filter, ties,
masked and odd values, split and strided vocabularies of one token to the most."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from collective_communication_virtual_gb300 import vcomm as V
from tests import sample_ref as S
from tests.gpu_util import DEV
from tests.test_gpu_norm import BF16, F16, F32

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


def split(logits, ranks, part, stride, offset):
    """Device copies of each rank's columns; what lies between and behind them is a large value."""
    rows, vocab = logits.shape
    got = []
    for r in range(ranks):
        flat = torch.full((offset + rows * stride + 64,), 60000.0, dtype=logits.dtype, device=DEV)
        lo, hi = min(vocab, r * part), min(vocab, (r + 1) * part)
        flat[offset:offset + rows * stride].view(rows, stride)[:, :hi - lo].copy_(logits[:, lo:hi])
        got.append(flat[offset:])
    return got


def column(values, dtype):
    return None if values is None else torch.tensor(values, dtype=dtype, device=DEV)


def sample(comm, logits, uniform, ranks=1, temperature=None, top_k=None, top_p=None, min_p=None, part=0, pad=0, offset=0,
           skip=()):
    rows, vocab = logits.shape
    part = part or -(-vocab // ranks)
    bufs = split(logits, ranks, part, part + pad, offset)
    tokens = [None if r in skip else torch.full((rows + 3,), -9, dtype=torch.int32, device=DEV) for r in range(ranks)]
    logprob = torch.full((rows + 3,), 77.0, device=DEV)
    V.vSample(V.vSampleDesc(rows, vocab, logits.dtype, part, part + pad), bufs, column(temperature, F32), column(top_k, torch.int32),
              column(top_p, F32), column(min_p, F32), column(uniform, F32), tokens, logprob, comm)
    torch.cuda.synchronize()
    wanted = [t.cpu() for t in tokens if t is not None]
    assert all(torch.equal(t, wanted[0]) for t in wanted) and (wanted[0][rows:] == -9).all() and (logprob[rows:] == 77).all()
    return wanted[0][:rows].tolist(), logprob[:rows].cpu().double().tolist()


def check(tokens, logprobs, logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    host = logits.double().numpy()
    for row, token in enumerate(tokens):
        filters = dict(temperature=1.0 if temperature is None else temperature[row], top_k=0 if top_k is None else top_k[row],
                       top_p=1.0 if top_p is None else top_p[row], min_p=0.0 if min_p is None else min_p[row])
        u = float(np.float32(uniform[row]))
        assert S.matches(token, host[row], u, **filters), (row, token, u, filters)
        e, _ = S.kept(host[row], temperature=filters["temperature"])
        want = S.logprob(e, host[row], token, filters["temperature"])
        # the difference and its quotient, the rounded weights' sum (2^-20 of it: each is rounded as an
        # fp32 product of up to 64) and the logarithm.  The sum is taken in units of 2^-44, to which at
        # most every weight is rounded on its own: vocab of those units, which the logarithm of a sum
        # of at least 1 does not enlarge.  (At -3e-8 the first version of this bound, without that
        # term, allowed 6e-14, where one unit is 5.7e-14.)
        slack = 2.0 ** -19 * (1 - np.exp(-abs(want))) + 2.0 ** -22 * abs(want) + host.shape[1] * 2.0 ** -44
        assert abs(logprobs[row] - want) <= slack, (row, want)


def spread(rows, vocab, dtype, seed, peaks=8):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=gen) * 2
    at = torch.randint(0, vocab, (rows, peaks), generator=gen)
    x.scatter_add_(1, at, 3 + 5 * torch.rand(rows, peaks, generator=gen))
    if vocab > 8:
        x[:, 5::97] = -float("inf")
    return x.to(dtype), torch.rand(rows, generator=gen).tolist()


FILTERS = [dict(), dict(top_k=[1, 2, 50, 0, 700]), dict(top_p=[0.9, 0.5, 0.999, 0.0, 1.0]), dict(min_p=[0.1, 0.01, 0.0, 1.0, 2.0]),
           dict(top_k=[40, 0, 5, 300, 1000], top_p=[0.9, 0.95, 0.3, 0.8, 0.99]),
           dict(temperature=[0.7, 1.3, 0.0, 0.05, 5.0], top_k=[0, 20, 3, 10, 100], top_p=[0.8, 0.9, 0.1, 0.7, 0.95], min_p=[0.05, 0.0, 0.5, 0.02, 0.001])]


def cycle(filters, rows):
    return {k: [v[i % len(v)] for i in range(rows)] for k, v in filters.items()}


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("filters", FILTERS)
@pytest.mark.parametrize("ranks,rows,vocab", [(1, 5, 1), (1, 5, 2), (2, 10, 7), (3, 10, 100), (1, 40, 1000), (4, 10, 4096), (2, 10, 4097),
                                              (8, 5, 8192), (3, 10, 20000), (3, 5, 50001), (8, 5, 131072), (64, 5, 32001)])
def test_sample(comms, ranks, rows, vocab, filters, dtype):
    logits, uniform = spread(rows, vocab, dtype, vocab + ranks)
    f = cycle(filters, rows)
    check(*sample(comms(ranks), logits, uniform, ranks, **f), logits, uniform, **f)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_largest_vocabulary_and_many_rows(comms, dtype):
    logits, uniform = spread(10, 262144, dtype, 3)
    for filters in FILTERS[1:]:
        f = cycle(filters, 10)
        check(*sample(comms(8), logits, uniform, 8, **f), logits, uniform, **f)
    logits, uniform = spread(700, 9000, dtype, 4)
    f = cycle(FILTERS[4], 700)
    check(*sample(comms(2), logits, uniform, 2, **f), logits, uniform, **f)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("kw", [dict(pad=8), dict(pad=3), dict(offset=1), dict(part=3000), dict(part=9999, pad=1, offset=3),
                                dict(skip=(0, 2)), dict(part=1668)])
def test_parts_strides_and_offsets(comms, dtype, kw):
    logits, uniform = spread(10, 5003, dtype, 5)
    f = cycle(FILTERS[5], 10)
    check(*sample(comms(3), logits, uniform, 3, **f, **kw), logits, uniform, **f)


@pytest.mark.parametrize("filters", [dict(top_k=7), dict(top_p=0.8), dict(min_p=0.2), dict(top_k=60, top_p=0.9), dict()])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab,levels", [(64, 64), (64, 4), (300, 1), (5000, 40)])
def test_every_kept_token_is_drawn_and_no_other(comms, vocab, levels, dtype, filters):
    # one row drawn with 2048 numbers that cover [0, 1); few different values, so that ties are cut
    gen = torch.Generator().manual_seed(vocab + levels)
    values = torch.randn(levels, generator=gen) * 1.5
    row = values[torch.randint(0, levels, (vocab,), generator=gen)].to(dtype)
    n = 2048
    uniform = ((torch.arange(n) + 0.5) / n).tolist()
    f = {k: [v] * n for k, v in filters.items()}
    tokens, _ = sample(comms(2), row.expand(n, -1).contiguous(), uniform, 2, **f)
    host = row.double().numpy()
    e, mask = S.kept(host, **filters)
    want, lo, hi, _ = S.draw(e, mask, 0.5)
    for token, u in zip(tokens, uniform):
        assert mask[token] and lo[token] - S.NEAR <= u <= hi[token] + S.NEAR
    assert tokens == sorted(tokens)
    assert set(np.flatnonzero(mask & (hi - lo > 1.01 / n))) <= set(tokens)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("vocab", [100, 9000, 70000])
def test_values_at_the_ends(comms, vocab, dtype):
    inf, nan = float("inf"), float("nan")
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(12, vocab, generator=gen)
    x[0] = -inf                                       # nothing to draw
    x[1] = nan
    x[2, :] = -inf
    x[2, vocab - 1] = -3.0                            # one
    x[3, 4::7] = nan
    x[4, [3, vocab // 2, vocab - 1]] = inf            # infinite ones share the draw
    x[5] = 0.0
    x[5, ::2] = -0.0                                  # equal to 0
    x[6] = torch.finfo(dtype).min
    x[7] = torch.finfo(dtype).max
    x[7, ::3] = torch.finfo(dtype).min
    x[8] *= torch.finfo(dtype).tiny                   # all weights 1
    x[9] = torch.finfo(dtype).min
    x[9, 5] = 0
    logits = x.to(dtype)
    for u in (0.0, 0.37, 1 - 2.0 ** -24):
        for f in (dict(), dict(top_k=[30] * 12), dict(top_p=[0.9] * 12), dict(top_k=[30] * 12, top_p=[0.5] * 12, min_p=[0.01] * 12)):
            tokens, logprobs = sample(comms(2), logits, [u] * 12, 2, **f)
            assert tokens[:2] == [-1, -1] and all(np.isnan(logprobs[:2])) and tokens[2] == vocab - 1
            check(tokens[2:], logprobs[2:], logits[2:], [u] * 10, **{k: v[2:] for k, v in f.items()})


def test_parameters_at_the_ends(comms):
    logits, _ = spread(1, 3000, F32, 9)
    inf, nan = float("inf"), float("nan")
    rows = [(t, k, p, m, u) for t in (1.0, 1e-38, 1e-3, 1e30) for k, p, m, u in
            [(0, 1.0, 0.0, 0.3), (-5, nan, nan, 0.3), (1 << 30, 2.0, -1.0, 0.3), (2999, 0.999999, 1e-30, 0.9), (2, 1e-30, 0.0, 0.99),
             (10, 0.5, 1.0, -1.0), (10, 0.5, 0.0, 1.0), (10, 0.9, 0.0, inf), (10, 0.9, 0.0, nan), (10, -1.0, 0.0, 0.9)]]
    rows += [(t, 5, 0.9, 0.1, 0.99) for t in (0.0, -1.0, nan, -inf)]
    t, k, p, m, u = zip(*rows)
    many = logits.expand(len(rows), -1).contiguous()
    tokens, logprobs = sample(comms(1), many, u, 1, t, k, p, m)
    host = logits[0].double().numpy()
    for i, row in enumerate(rows):
        temperature = row[0] if row[0] == row[0] else 0.0
        assert S.matches(tokens[i], host, np.float32(row[4]), temperature=temperature, top_k=row[1],
                         top_p=1.0 if row[2] != row[2] else row[2], min_p=0.0 if row[3] != row[3] else row[3]), row
    # an infinite temperature makes all tokens alike
    alike, _ = sample(comms(1), torch.randn(1, 64).expand(64, -1).contiguous(), [(i + 0.5) / 64 for i in range(64)], 1, [inf] * 64)
    assert alike == list(range(64))


def test_flat_rows_where_topp_keeps_nearly_all(comms):
    # borders of a hundred thousand nearly equal weights
    gen = torch.Generator().manual_seed(21)
    x = torch.randn(16, 100000, generator=gen) * 0.01
    u = torch.rand(16, generator=gen).tolist()
    for dtype in (F32, BF16):
        for f in (dict(), dict(top_p=[0.9] * 16), dict(top_p=[0.999] * 16, top_k=[90000] * 16)):
            check(*sample(comms(4), x.to(dtype), u, 4, **f), x.to(dtype), u, **f)


def test_the_same_tokens_again_on_streams_in_a_group_and_in_a_graph(comms):
    comm = comms(4)
    rows, vocab = 20, 30000
    logits, uniform = spread(rows, vocab, BF16, 31)
    f = cycle(FILTERS[5], rows)
    want, _ = sample(comm, logits, uniform, 4, **f)
    bufs = split(logits, 4, vocab // 4, vocab // 4, 0)
    args = [column(f["temperature"], F32), column(f["top_k"], torch.int32), column(f["top_p"], F32), column(f["min_p"], F32)]
    u, desc = column(uniform, F32), V.vSampleDesc(rows, vocab, BF16)
    outs = [torch.full((4, rows), -9, dtype=torch.int32, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    for out, side in zip(outs[:2], (torch.cuda.Stream(), torch.cuda.Stream())):
        for _ in range(3):
            V.vSample(desc, bufs, *args, u, list(out), None, comm, stream=side)
    V.vcommGroupStart(comm)
    V.vSample(desc, list(bufs), *args, u, list(outs[2]), None, comm)
    torch.cuda.synchronize()
    assert (outs[2] == -9).all()
    V.vcommGroupEnd(comm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        V.vSample(desc, bufs, *args, u, list(outs[3]), None, comm)
    u.fill_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(o[r].tolist() == want for o in outs[:3] for r in range(4))
    half, logprobs = outs[3][0].tolist(), None
    host = logits.double().numpy()
    for row in range(rows):
        assert S.matches(half[row], host[row], 0.5, **{k: v[row] for k, v in f.items()})


def test_rows_past_two_to_the_31_elements(comms):
    vocab, stride = 64, 1 << 20
    rows = 2100
    x = torch.full((rows * stride,), -5.0, dtype=BF16, device=DEV).view(rows, stride)
    at = torch.arange(rows, device=DEV) % vocab
    x[torch.arange(rows, device=DEV), at] = 30.0
    tokens = torch.empty(rows, dtype=torch.int32, device=DEV)
    V.vSample(V.vSampleDesc(rows, vocab, BF16, stride=stride), [x], None, None, None, None,
              torch.full((rows,), 0.5, device=DEV), [tokens], None, comms(1))
    assert torch.equal(tokens.long(), at)


def test_refusals(comms):
    comm = comms(2)
    x = torch.zeros(4, 64, dtype=BF16, device=DEV)
    u, tokens = torch.zeros(4, device=DEV), torch.full((4,), -9, dtype=torch.int32, device=DEV)
    good = dict(rows=4, vocab=100, datatype=BF16, part=64)

    def refused(call, *args):
        with pytest.raises(V.VcommError) as e:
            call(*args)
        assert e.value.code == V.vInvalidArgument

    fine = [[x, x], None, None, None, None, u, [tokens, None], None]
    for change in (dict(vocab=0), dict(vocab=262145), dict(rows=(1 << 24) + 1), dict(part=49), dict(part=262145), dict(stride=63),
                   dict(stride=1 << 62), dict(datatype=torch.int32)):
        refused(V.vSample, V.vSampleDesc(**{**good, **change}), *fine, comm)
    d = V.vSampleDesc(**good)
    odd = x.data_ptr() + 1
    for i, value in [(0, [x, None]), (0, [odd, x]), (0, [x]), (1, odd), (2, odd), (3, odd), (4, odd), (5, None), (5, odd),
                     (6, [None, None]), (6, [odd, None]), (7, odd)]:
        refused(V.vSample, d, *fine[:i], value, *fine[i + 1:], comm)
    V.vSample(V.vSampleDesc(**{**good, "rows": 0}), [None, None], None, None, None, None, None, [None, None], None, comm)
    torch.cuda.synchronize()
    assert (tokens == -9).all() and V.vcommGetAsyncError(comm) == V.vSuccess
    V.vSample(V.vSampleDesc(4, 60, BF16, part=64), [x, None], None, None, None, None, u, [None, tokens], None, comm)
    assert tokens.tolist() == [0] * 4
    V.vcommGroupStart(comm)
    V.vSample(d, [x, None], None, None, None, None, u, [tokens, None], None, comm)
    refused(V.vcommGroupEnd, comm)
