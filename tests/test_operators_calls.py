"""The operators' entry points on a host stand-in for the device and the communicator
(operators_host.cpp)."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from collective_communication_virtual_gb300 import build, vcomm as V

HERE = os.path.dirname(os.path.abspath(__file__))
COMM = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """The entry points over host memory, with the binding's signatures."""
    so = str(tmp_path_factory.mktemp("host") / "operators_host.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")))
    subprocess.run(["g++", "-O3", "-std=c++17", "-Wall", "-fPIC", "-shared", "-pthread", "-Wl,-Bsymbolic", "-Wl,--no-undefined",
                    "-I", build.INCLUDE, "-I", build.CSRC, "-isystem", os.path.join(cuda, "include"),
                    os.path.join(HERE, "operators_host.cpp"), os.path.join(build.CSRC, "operators.cpp"), "-o", so, "-ldl"],
                   check=True)
    lib = ctypes.CDLL(so)
    for name, (args, res) in V._SIGNATURES.items():
        if hasattr(lib, name):
            getattr(lib, name).argtypes, getattr(lib, name).restype = args, res
    return lib


def ints(*values):
    """Addresses of nothing, as a pointer array."""
    return (ctypes.c_void_p * len(values))(*values)


@pytest.mark.parametrize("rows,hidden", [(1, 512), (12, 1024), (3, 4096), (331, 1001)])
def test_the_backward_pass_needs_nothing_of_the_communicator_but_its_launches(host, rows, hidden):
    # the variable all-to-all owns the communicator's counters; the stand-in has none, so a
    # reference to them does not link
    host.host_start(2)
    desc = V.vRmsNormDesc(rows, hidden, torch.bfloat16)
    need = ctypes.c_size_t()
    d = ctypes.addressof(desc)
    assert host.vRmsNormBackwardWorkspace(d, COMM, ctypes.addressof(need)) == V.vSuccess
    bufs = ints(0x10000, 0x20000)
    a = ctypes.addressof(bufs)
    assert host.vAllReduceRmsNormBackward(d, a, 0x30000, 0x40000, 0x50000, None, a, 0x60000, 0x70000, need.value, COMM,
                                          None) == V.vSuccess
    assert host.host_launches() == 1
