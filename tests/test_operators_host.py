"""The operators' entry points without a GPU: refusals before CUDA is touched, the binding's
structures and its marshalling."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

from collective_communication_virtual_gb300 import build, vcomm as V

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "vcomm.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return V.lib()


def test_a_null_or_foreign_communicator_or_list_is_refused(lib):
    arr = (ctypes.c_void_p * 4)()
    desc = V.vRmsNormDesc(4, 64, torch.bfloat16)
    size = ctypes.c_size_t()
    garbage = ctypes.create_string_buffer(4096)
    d, a, n = ctypes.addressof(desc), ctypes.addressof(arr), ctypes.addressof(size)
    for comm in (None, ctypes.addressof(garbage)):
        assert lib.vAllReduceRmsNorm(d, a, None, a, None, a, None, comm, None) == V.vInvalidArgument
        assert lib.vAllReduceRmsNormQuant(d, a, None, a, None, a, a, None, comm, None) == V.vInvalidArgument
        assert lib.vAllReduceRmsNormBackward(d, a, a, a, a, None, a, a, a, 1 << 20, comm, None) == V.vInvalidArgument
        assert lib.vRmsNormBackwardWorkspace(d, comm, n) == V.vInvalidArgument
        assert lib.vGradNormWorkspace(None, comm, n) == V.vInvalidArgument
        assert lib.vGradNorm(None, a, a, 1 << 20, comm, None) == V.vInvalidArgument
        assert lib.vClipGradNorm(None, 1.0, a, a, 1 << 20, comm, None) == V.vInvalidArgument
    assert lib.vGradListDestroy(None) == V.vInvalidArgument
    assert lib.vGradListDestroy(ctypes.addressof(garbage)) == V.vInvalidArgument


def test_list_arguments_are_checked_before_cuda(lib):
    handle = ctypes.c_void_p(123)
    counts, types = (ctypes.c_size_t * 1)(8), (ctypes.c_int * 1)(V.vFloat32)
    grads = (ctypes.c_void_p * 1)(4096)
    at = ctypes.addressof
    for args in ((0, 1, at(counts), at(types), None, at(grads), None), (65, 1, at(counts), at(types), None, at(grads), None),
                 (1, -1, at(counts), at(types), None, at(grads), None), (1, 1, None, at(types), None, at(grads), None),
                 (1, 1, at(counts), None, None, at(grads), None), (1, 1, at(counts), at(types), None, None, None)):
        assert lib.vGradListCreate(at(handle), *args) == V.vInvalidArgument
        assert handle.value is None
    assert lib.vGradListCreate(None, 1, 1, at(counts), at(types), None, at(grads), None) == V.vInvalidArgument
    if not torch.cuda.is_available():
        assert lib.vGradListCreate(at(handle), 1, 1, at(counts), at(types), None, at(grads), None) == V.vUnhandledCudaError
        assert handle.value is None


def test_the_descriptor_has_the_headers_layout(tmp_path):
    fields = [name for name, _ in V.vRmsNormDesc_t._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include "vcomm.h"\n#include <stdio.h>\nint main(void){printf("%zu", sizeof(vRmsNormDesc_t));'
                   + "".join(f'printf(" %zu", offsetof(vRmsNormDesc_t, {f}));' for f in fields) + "return 0;}\n")
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    want = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert want == [ctypes.sizeof(V.vRmsNormDesc_t)] + [getattr(V.vRmsNormDesc_t, f).offset for f in fields]
    text = open(HEADER).read()
    assert "#define VCOMM_MAX_HIDDEN 65536" in text


def test_descriptor_defaults():
    d = V.vRmsNormDesc(3, 64, torch.float16)
    assert (d.rows, d.hidden, d.sendStride, d.residualStride, d.recvStride) == (3, 64, 0, 0, 0)
    assert (d.datatype, d.weightType, d.quantGroup) == (V.vFloat16, V.vFloat16, 0)
    assert V.vRmsNormDesc(3, 64, torch.float16, torch.float32).weightType == V.vFloat32


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return V.vSuccess
        return call


def test_made_buffers_stand_for_their_list(monkeypatch):
    fake = Recorder()
    monkeypatch.setattr(V, "lib", lambda: fake)
    monkeypatch.setitem(V._N_RANKS, 0x1234, 3)
    comm = ctypes.c_void_p(0x1234)
    desc = V.vRmsNormDesc(1, 8, torch.float32)
    made = V.vBuffers([16, None, 48])
    V.vAllReduceRmsNorm(desc, made, None, 64, None, [1, 2, None], None, comm, stream=0)
    _, args = fake.calls[-1]
    assert list((ctypes.c_void_p * 3).from_address(args[1])) == [16, None, 48]
    assert list(args[5]) == [1, 2, None] and args[3] == 64 and args[0] == ctypes.addressof(desc)
    for wrong in (V.vBuffers([1, 2]), [1, 2, 3, 4]):
        with pytest.raises(V.VcommError) as e:
            V.vAllReduceRmsNorm(desc, wrong, None, 64, None, made, None, comm, stream=0)
        assert e.value.code == V.vInvalidArgument
    # the collectives take them too
    V.vAllReduce(made, made, 4, V.vFloat32, "sum", comm, stream=0)
    assert fake.calls[-1][1][0] == made.address


def test_a_tensor_list_is_checked_and_marshalled(monkeypatch):
    seen = {}

    class Fake:
        def vGradListCreate(self, out, n_ranks, n, counts, types, replicated, grads, outs):
            seen.update(ranks=n_ranks, counts=list((ctypes.c_size_t * n).from_address(counts)),
                        types=list((ctypes.c_int * n).from_address(types)),
                        replicated=list((ctypes.c_ubyte * n).from_address(replicated)),
                        grads=list((ctypes.c_void_p * (n * n_ranks)).from_address(grads)), outs=outs)
            ctypes.c_void_p.from_address(out).value = 77
            return V.vSuccess

        def vGradListDestroy(self, handle):
            seen["destroyed"] = handle
            return V.vSuccess

    monkeypatch.setattr(V, "lib", lambda: Fake())
    grads = [[torch.zeros(5), torch.zeros(3, dtype=torch.bfloat16)] for _ in range(2)]
    tensors = V.vTensorList(grads, replicated=[False, True])
    assert tensors.handle == 77 and seen["ranks"] == 2 and seen["counts"] == [5, 3]
    assert seen["types"] == [V.vFloat32, V.vBFloat16] and seen["replicated"] == [0, 1] and seen["outs"] is None
    assert seen["grads"] == [t.data_ptr() for r in grads for t in r]
    tensors.close()
    tensors.close()
    assert seen["destroyed"] == 77 and tensors.handle is None
    wrong = [grads[0], [torch.zeros(5), torch.zeros(4, dtype=torch.bfloat16)]]
    for args in ((wrong,), (grads, wrong), (grads, grads[:1]), (grads, None, [True]), ([],),
                 ([[torch.zeros(4, 4).t()[:2]]],)):
        with pytest.raises(V.VcommError) as e:
            V.vTensorList(*args)
        assert e.value.code == V.vInvalidArgument
