"""The entry points of the block norm, the mixture of experts and the sampling without a GPU: refusals,
groups, workspaces and launch shapes on a host stand-in (decoder_host.cpp), and the structures' layout."""
from __future__ import annotations

import ctypes
import itertools
import os
import shutil
import subprocess

import pytest
import torch

from collective_communication_virtual_gb300 import build, vcomm as V

HERE = os.path.dirname(os.path.abspath(__file__))
COMM = ctypes.c_void_p(0x1000)
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
OK, BAD = V.vSuccess, V.vInvalidArgument


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("host") / "decoder_host.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")))
    sources = [os.path.join(build.CSRC, f) for f in ("operators.cpp", "block_norm.cpp", "moe.cpp", "sample.cpp")]
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-Wl,--no-undefined", "-I",
                    build.INCLUDE, "-I", build.CSRC, "-isystem", os.path.join(cuda, "include"),
                    os.path.join(HERE, "decoder_host.cpp"), *sources, "-o", so, "-ldl"], check=True)
    lib = ctypes.CDLL(so)
    for name, (args, res) in V._SIGNATURES.items():
        if hasattr(lib, name):
            getattr(lib, name).argtypes, getattr(lib, name).restype = args, res
    return lib


def pointers(*values):
    return (ctypes.c_void_p * len(values))(*values)


def at(x):
    return ctypes.addressof(x) if isinstance(x, (ctypes.Structure, ctypes.Array)) else x


class Call:
    """An entry point with arguments that it takes, one of which can be replaced."""

    def __init__(self, f, **args):
        self.f, self.args = f, args

    def __call__(self, **change):
        return self.f(*(at(v) for v in {**self.args, **change}.values()))


def calls(host, ranks=2):
    host.host_start(ranks)
    bufs, other = pointers(*range(0x10000, 0x10000 + ranks * 0x1000, 0x1000)), pointers(*range(0x80000, 0x80000 + ranks * 0x1000, 0x1000))
    block = dict(desc=V.vBlockNormDesc(4, 64, BF16), send=bufs)
    tail = dict(comm=COMM, stream=None)
    moe = V.vMoeDesc(4, 64, 32, 6, 2, BF16)
    return {
        "forward": Call(host.vAllReduceBlockNorm, **block, residual=0x100, post=0x200, gate=0x300, pre=0x400, blockOut=0x500,
                        residualOut=0x600, recv=other, rstd=0x700, **tail),
        "backward": Call(host.vAllReduceBlockNormBackward, **block, hidden=0x100, block=0x200, rstd=0x300, post=0x400, gate=0x500,
                         pre=0x600, gradStream=0x700, gradResidual=0x800, recv=other, gradPost=0x900, gradGate=0xA00,
                         gradPre=0xB00, workspace=0xC00, bytes=1 << 30, **tail),
        "route": Call(host.vMoeRoute, desc=moe, x=0x100, router=0x200, bias=0x300, ids=0x400, weights=0x500, **tail),
        "experts": Call(host.vMoeExperts, desc=moe, x=0x100, ids=0x200, weights=0x300, up=bufs, down=bufs, recv=other,
                        workspace=0x400, bytes=1 << 30, **tail),
        "sample": Call(host.vSample, desc=V.vSampleDesc(4, 100, BF16), logits=bufs, temperature=0x100, topK=0x200, topP=0x300,
                       minP=0x400, uniform=0x500, tokens=other, logprob=0x600, **tail),
    }


OPTIONAL = {"forward": ["residual", "gate", "blockOut", "residualOut", "rstd"], "backward": ["gradStream", "gradResidual"],
            "route": ["bias"], "experts": [], "sample": ["temperature", "topK", "topP", "minP", "logprob"]}


@pytest.mark.parametrize("name", list(OPTIONAL))
def test_what_may_be_null_and_what_not(host, name):
    call = calls(host)[name]
    assert call() == OK and host.host_launches() == 1
    for key in call.args:
        if key in ("stream", "bytes"):
            continue
        change = {key: None}
        if name == "backward" and key == "gate":
            assert call(gate=None) == BAD and call(gradGate=None) == BAD and call(gate=None, gradGate=None) == OK
            continue
        before = host.host_launches()
        want = OK if key in OPTIONAL[name] else BAD
        assert call(**change) == want, (key, want)
        assert host.host_launches() == before + (want == OK)


@pytest.mark.parametrize("name", list(OPTIONAL))
def test_addresses_off_their_elements_are_refused(host, name):
    call = calls(host)[name]
    for key, value in call.args.items():
        if isinstance(value, int) and key not in ("bytes", "comm"):
            assert call(**{key: value + 1}) == BAD, key
        if isinstance(value, ctypes.Array):
            for i in range(2):
                odd = type(value)(*value)
                odd[i] += 1
                assert call(**{key: odd}) == BAD, key
    assert host.host_launches() == 0


@pytest.mark.parametrize("name", list(OPTIONAL))
def test_a_group_keeps_its_own_copy(host, name):
    # the arrays and the descriptor may be reused as soon as the recorded call returns
    call = calls(host)[name]
    host.host_group(1)
    keep = {k: type(v)(*v) if isinstance(v, ctypes.Array) else v for k, v in call.args.items()}
    desc = type(keep["desc"]).from_buffer_copy(keep["desc"])
    assert Call(call.f, **{**keep, "desc": desc})() == OK and host.host_launches() == 0
    for v in keep.values():
        if isinstance(v, ctypes.Array):
            v[0] = v[1] = 1
    ctypes.memset(ctypes.addressof(desc), 0xFF, ctypes.sizeof(desc))
    assert host.host_group_end() == OK and host.host_launches() == 1
    # and a recorded call's error is the group's
    host.host_group(1)
    key = "x" if "x" in call.args else "pre" if "pre" in call.args else "uniform"
    assert call(**{key: None}) == OK
    assert host.host_group_end() == BAD


def test_ranks_without_experts_or_columns_need_no_buffer(host):
    c = calls(host, 4)["experts"]
    none = pointers(0x1000, 0x2000, 0x3000, None)
    assert c(desc=V.vMoeDesc(4, 64, 32, 3, 2, BF16), up=none, down=none) == OK
    assert c(desc=V.vMoeDesc(4, 64, 32, 4, 2, BF16), up=none, down=none) == BAD
    c = calls(host, 4)["sample"]
    assert c(desc=V.vSampleDesc(4, 96, BF16, 32), logits=none) == OK
    assert c(desc=V.vSampleDesc(4, 97, BF16, 32), logits=none) == BAD


def test_sizes_at_their_limits(host):
    c = calls(host)
    route, experts, sample = c["route"], c["experts"], c["sample"]
    assert route(desc=V.vMoeDesc(1024, 65536, 65536, 1024, 32, F32)) == OK
    assert experts(desc=V.vMoeDesc(1024, 64, 64, 1024, 32, F32), bytes=1 << 40) == OK
    for change in (dict(rows=1025), dict(hidden=65537), dict(ffn=65537), dict(experts=1025), dict(experts=0), dict(top_k=33, experts=64),
                   dict(top_k=0), dict(top_k=7), dict(row_stride=63), dict(recv_stride=63), dict(router_type=F16)):
        d = V.vMoeDesc(**{**dict(rows=4, hidden=64, ffn=32, experts=6, top_k=2, datatype=BF16), **change})
        assert route(desc=d) == BAD and experts(desc=d) == BAD, change
    assert sample(desc=V.vSampleDesc(1 << 24, 262144, F32)) == OK
    for change in (dict(rows=(1 << 24) + 1), dict(vocab=0), dict(vocab=262145), dict(part=49), dict(stride=49), dict(part=1 << 20)):
        assert sample(desc=V.vSampleDesc(**{**dict(rows=4, vocab=100, datatype=BF16), **change})) == BAD, change
    forward = c["forward"]
    for change in (dict(residual_scale=float("nan")), dict(residual_scale=float("-inf")), dict(eps=-1.0), dict(hidden=65537)):
        assert forward(desc=V.vBlockNormDesc(**{**dict(rows=4, hidden=64, datatype=BF16), **change})) == BAD, change


# ---- workspaces and launch shapes ---------------------------------------------------------------

SHAPE = ("vecs", "team", "per_cta", "cluster", "threads", "staged", "rounds", "ctas", "smem", "parts")
WIDTHS = [1, 7, 8, 31, 64, 100, 129, 512, 1000, 2048, 2731, 4096, 4099, 8192, 12296, 16384, 20480, 20481, 24001, 32768, 40961, 65535,
          65536]


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("backward", [False, True])
def test_block_norm_shapes_hold_every_row_within_the_hardware(host, dtype, wtype, backward):
    out = (ctypes.c_int * len(SHAPE))()
    per = 16 // dtype.itemsize
    need = ctypes.c_size_t()
    for ranks, hidden, rows, offset, extra in itertools.product((1, 2, 3, 8, 24, 64), WIDTHS, (1, 3, 77, 300, 2500, 9001, 1 << 20),
                                                                (0, dtype.itemsize), (None, 0x7000)):
        host.host_start(ranks)
        desc = V.vBlockNormDesc(rows, hidden, dtype, wtype)
        send = pointers(*[0x100000 + offset] * ranks)
        d = ctypes.addressof(desc)
        assert host.vBlockNormBackwardWorkspace(d, COMM, ctypes.addressof(need)) == OK
        if backward:
            assert host.vAllReduceBlockNormBackward(d, at(send), 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, extra, 0x8000, at(send),
                                                    0x9000, 0xA000, 0xB000, 0xC000, need.value, COMM, None) == OK, (ranks, hidden, rows)
            host.host_back(out)
        else:
            assert host.vAllReduceBlockNorm(d, at(send), extra, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, at(send), 0x8000, COMM, None) == OK
            host.host_block(out)
        s = dict(zip(SHAPE, out))
        where = (ranks, hidden, rows, offset, s)
        assert s["vecs"] in (1, 2, 4) and s["cluster"] in (1, 2, 4, 8), where
        assert s["cluster"] * s["team"] * s["vecs"] * per >= hidden, where
        assert s["threads"] == s["team"] * s["per_cta"] and s["threads"] % 32 == 0 and s["threads"] <= (512 if s["staged"] else 640), where
        assert s["smem"] <= 227 * 1024 - 768, where
        assert s["cluster"] == 1 or (s["per_cta"] == 1 and s["team"] > 32), where
        if backward:
            assert 1 <= s["parts"] <= 16 * 152 and need.value >= s["parts"] * 2 * hidden * 4, where
        elif s["staged"] and s["rounds"]:
            assert (s["ctas"] - 1) * s["rounds"] * s["per_cta"] < rows <= s["ctas"] * s["rounds"] * s["per_cta"], where


EXPERTS = ("tokens", "split_up", "split_down", "grid_up", "grid_down", "stages_up", "stages_down", "here", "smem_up", "smem_down",
           "aligned", "tile_up", "tile_down", "share")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_expert_shapes(host, dtype):
    out = (ctypes.c_int * len(EXPERTS))()
    need = ctypes.c_size_t()
    for ranks, rows, hidden, ffn, experts, k in itertools.product((1, 3, 8), (1, 4, 5, 16, 64, 300, 1024), (8, 100, 1001, 4096), (8, 333, 1536),
                                                                  (1, 10, 40, 128, 1024), (1, 4, 32)):
        if k > experts:
            continue
        host.host_start(ranks)
        desc = V.vMoeDesc(rows, hidden, ffn, experts, k, dtype)
        d, bufs = ctypes.addressof(desc), pointers(*[0x100000] * ranks)
        assert host.vMoeExpertsWorkspace(d, COMM, ctypes.addressof(need)) == OK
        args = (d, 0x1000, 0x2000, 0x3000, at(bufs), at(bufs), at(bufs), 0x4000)
        assert host.vMoeExperts(*args, need.value - 1, COMM, None) == BAD
        assert host.vMoeExperts(*args, need.value, COMM, None) == OK
        host.host_experts(out)
        s = dict(zip(EXPERTS, out))
        where = (ranks, rows, hidden, ffn, experts, k, s)
        assert s["share"] * ranks >= experts and need.value >= rows * k * 4 * (ffn + hidden), where
        assert (s["tokens"] > 0) == (dtype != F32), where
        # a kernel that may say that a wait ran out is one that the communicator waits for
        assert host.host_tracked() == (s["tokens"] > 0), where
        if s["tokens"]:
            assert s["tokens"] in (16, 32, 64), where
            for way, columns, tiles in (("up", hidden, -(-ffn // 64)), ("down", ffn, -(-hidden // 128))):
                split, grid = s["split_" + way], s["grid_" + way]
                assert split in (1, 2, 4) and split <= max(1, -(-columns // 128)) and (split == 1 or s["tokens"] == 16), where
                assert grid % split == 0 and split <= grid <= 152, where
                assert 2 <= s["stages_" + way] <= 8 and s["smem_" + way] <= 225 * 1024, where
        else:
            assert s["tile_up"] in (8, 16, 32) and s["tile_down"] in (16, 32), where
            # a counter for every tile of columns
            assert need.value >= rows * k * 4 * (ffn + hidden) + -(-hidden // s["tile_down"]) * 4, where


def test_few_tokens_get_all_stages_that_fit(host):
    # a stage holds 128 columns of 128 rows of the weights, 32 KiB, and of 16 tokens one or two values, 4 KiB each
    out = (ctypes.c_int * len(EXPERTS))()
    for rows, hidden, ffn, experts, k in ((1, 2048, 1024, 64, 4), (1, 4096, 1536, 128, 8), (13, 1001, 333, 10, 3), (4, 64, 32, 6, 2)):
        assert calls(host)["experts"](desc=V.vMoeDesc(rows, hidden, ffn, experts, k, BF16)) == OK
        host.host_experts(out)
        s = dict(zip(EXPERTS, out))
        for way, stage in (("up", 36 * 1024), ("down", 40 * 1024)):
            assert s["tokens"] == 16 and (s["stages_" + way] == 8 or s["smem_" + way] + stage > 225 * 1024), (rows, s)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_communicators_limit_and_hook_reach_the_experts(host, dtype):
    host.host_experts_limit.restype = ctypes.c_longlong
    assert calls(host)["experts"](desc=V.vMoeDesc(4, 64, 32, 6, 2, dtype)) == OK
    assert host.host_experts_limit() == 7654321 and host.host_experts_stall() == 5


def test_sample_shapes(host):
    out = (ctypes.c_int * 5)()
    for ranks, rows, vocab, dtype, offset in itertools.product((1, 3, 8, 64), (1, 10, 40, 300, 1 << 20), (1, 2, 7, 63, 64, 1000, 4097, 50001, 131072, 262144),
                                                               (BF16, F32), (0, 1)):
        host.host_start(ranks)
        desc = V.vSampleDesc(rows, vocab, dtype)
        bufs = pointers(*[0x100000 + offset * dtype.itemsize] * ranks)
        assert host.vSample(at(desc), at(bufs), None, None, None, None, 0x1000, at(pointers(*[0x2000] + [None] * (ranks - 1))), None, COMM,
                            None) == OK
        host.host_sample(out)
        cluster, each, parts, outs, part = out
        per = 16 // dtype.itemsize
        where = (ranks, rows, vocab, dtype, cluster, each)
        assert outs == 1 and part * ranks >= vocab and (parts - 1) * part < vocab <= parts * part, where
        # the blocks that the parts touch, wherever each starts within 16 bytes
        blocks = sum(-(-(per - 1 + min(part, vocab - r * part)) // per) for r in range(parts))
        most = -(-blocks // (16 * cluster))
        assert cluster in (1, 2, 4, 8) and most <= 32 * each, where
        assert 2560 * 8 + 512 * (each | 1) * 16 <= 192 * 1024, where


# ---- the library itself and the binding ------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    build.build()
    return V.lib()


def test_a_null_or_foreign_communicator_is_refused(lib):
    garbage = ctypes.create_string_buffer(4096)
    n = ctypes.c_size_t()
    for comm in (None, ctypes.addressof(garbage)):
        for f, args in ((lib.vAllReduceBlockNorm, 10), (lib.vMoeRoute, 6), (lib.vSample, 9)):
            assert f(*[ctypes.addressof(garbage)] * args, comm, None) == BAD
        assert lib.vAllReduceBlockNormBackward(*[ctypes.addressof(garbage)] * 15, 1 << 20, comm, None) == BAD
        assert lib.vMoeExperts(*[ctypes.addressof(garbage)] * 8, 1 << 20, comm, None) == BAD
        for f in (lib.vBlockNormBackwardWorkspace, lib.vMoeExpertsWorkspace):
            assert f(ctypes.addressof(garbage), comm, ctypes.addressof(n)) == BAD


@pytest.mark.parametrize("struct", [V.vBlockNormDesc_t, V.vMoeDesc_t, V.vSampleDesc_t])
def test_descriptors_have_the_headers_layout(tmp_path, struct):
    fields = [name for name, _ in struct._fields_]
    name = struct.__name__
    src = tmp_path / "t.c"
    src.write_text('#include "vcomm.h"\n#include <stdio.h>\nint main(void){printf("%zu", sizeof(' + name + '));'
                   + "".join(f'printf(" %zu", offsetof({name}, {f}));' for f in fields) + "return 0;}\n")
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c99", "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    want = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert want == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


def test_descriptor_defaults():
    d = V.vBlockNormDesc(3, 64, F16)
    assert (d.residualScale, d.datatype, d.weightType, d.sendStride) == (1.0, V.vFloat16, V.vFloat16, 0)
    m = V.vMoeDesc(3, 64, 32, 8, 2, BF16, F32, False)
    assert (m.datatype, m.routerType, m.normalize, m.rowStride, m.recvStride) == (V.vBFloat16, V.vFloat32, 0, 0, 0)
    s = V.vSampleDesc(3, 1000, F32)
    assert (s.part, s.stride, s.datatype) == (0, 0, V.vFloat32)
