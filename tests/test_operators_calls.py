"""The operators' entry points on a host stand-in for the device and the communicator
(operators_host.cpp)."""
from __future__ import annotations

import ctypes
import gc
import os
import shutil
import subprocess
import threading
import weakref

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


class Lists:
    """Gradient lists of one fp32 tensor of 64 elements on each of two ranks."""

    def __init__(self, host):
        self.host = host
        host.host_start(2)
        self.counts, self.types, self.grads = (ctypes.c_size_t * 1)(64), (ctypes.c_int * 1)(V.vFloat32), ints(0x10000, 0x20000)

    def make(self):
        handle = ctypes.c_void_p()
        at = ctypes.addressof
        assert self.host.vGradListCreate(at(handle), 2, 1, at(self.counts), at(self.types), None, at(self.grads), None) == V.vSuccess
        return handle.value

    def uses(self, handle):
        """What each call answers: the workspace's, the norm's and the clipping's."""
        need = ctypes.c_size_t()
        return [self.host.vGradNormWorkspace(handle, COMM, ctypes.addressof(need)),
                self.host.vGradNorm(handle, 0x30000, 0x40000, 1 << 20, COMM, None),
                self.host.vClipGradNorm(handle, 1.0, 0x30000, 0x40000, 1 << 20, COMM, None)]


def test_a_destroyed_list_is_refused_everywhere(host):
    lists = Lists(host)
    before = host.host_allocated()
    first = lists.make()
    assert lists.uses(first) == [V.vSuccess] * 3
    assert host.vGradListDestroy(first) == V.vSuccess
    for _ in range(2):
        launches = host.host_launches()
        assert lists.uses(first) == [V.vInvalidArgument] * 3
        assert host.vGradListDestroy(first) == V.vInvalidArgument
        assert host.host_launches() == launches
        lists.make()                 # a later list does not answer to the old handle
    assert host.host_allocated() == before + 2


def test_a_list_destroyed_before_its_group_ends_is_refused_there(host):
    lists = Lists(host)
    handle = lists.make()
    host.host_group(1)
    assert host.vClipGradNorm(handle, 1.0, 0x30000, 0x40000, 1 << 20, COMM, None) == V.vSuccess
    assert host.vGradListDestroy(handle) == V.vSuccess
    assert host.host_group_end() == V.vInvalidArgument
    assert host.host_launches() == 0


def test_lists_of_several_threads(host):
    # created, used and destroyed on four threads at once, the last use after the destruction
    lists = Lists(host)
    wrong = []

    def work():
        for _ in range(500):
            handle = lists.make()
            if lists.uses(handle) != [V.vSuccess] * 3 or host.vGradListDestroy(handle) != V.vSuccess:
                wrong.append(handle)
            if lists.uses(handle) != [V.vInvalidArgument] * 3:
                wrong.append(handle)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---- the binding's tensor lists ----------------------------------------------------------------

class FakeLists:
    """The list calls of the library, on handles of its own."""

    def __init__(self):
        self.live, self.made, self.calls = set(), 0, []

    def vGradListCreate(self, out, *args):
        self.made += 1
        self.live.add(self.made)
        ctypes.c_void_p.from_address(out).value = self.made
        return V.vSuccess

    def vGradListDestroy(self, handle):
        self.live.remove(handle)
        return V.vSuccess

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return V.vSuccess
        return call


@pytest.fixture
def fake(monkeypatch):
    made = FakeLists()
    monkeypatch.setattr(V, "lib", lambda: made)
    monkeypatch.setitem(V._N_RANKS, COMM.value, 1)
    before = V._dropped_lists[:]     # handles of the library's own
    V._dropped_lists.clear()
    yield made
    V._dropped_lists[:] = before


def test_a_tensor_list_holds_its_tensors(fake):
    # memory that the list's calls scale must not become another tensor's while the list lives
    grad, out = torch.ones(5), torch.ones(5)
    seen = [weakref.ref(grad), weakref.ref(out)]
    tensors = V.vTensorList([[grad]], [[out]])
    del grad, out
    gc.collect()
    assert all(r() is not None for r in seen)
    tensors.close()
    gc.collect()
    assert all(r() is None for r in seen)


def test_a_list_without_references_is_destroyed_by_the_next_one(fake):
    # not where the reference is lost, which may be within a graph's capture
    tensors = V.vTensorList([[torch.ones(5)]])
    first = tensors.handle
    del tensors
    gc.collect()
    assert fake.live == {first}
    kept = V.vTensorList([[torch.ones(5)]])
    assert fake.live == {kept.handle} and kept.handle != first
    kept.close()
    assert not fake.live
    del kept
    gc.collect()
    V.vTensorList([[torch.ones(5)]]).close()
    assert not fake.live


def refused(call, *args, **kw):
    with pytest.raises(V.VcommError) as e:
        call(*args, **kw)
    assert e.value.code == V.vInvalidArgument


def test_a_list_of_host_tensors_is_taken_by_no_call(fake):
    tensors = V.vTensorList([[torch.ones(5)]])
    space = (0x10000, 1 << 20)
    refused(V.vGradNormWorkspace, tensors, COMM)
    refused(V.vGradNorm, tensors, 0x20000, space, COMM, stream=0)
    refused(V.vClipGradNorm, tensors, 1.0, 0x20000, space, COMM, stream=0)
    assert not fake.calls


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on a device."""
    device_index = 0

    def get_device(self):
        return self.device_index


def on_device(index):
    t = torch.ones(5).as_subclass(OnDevice)
    t.device_index = index
    return t


def test_entries_that_are_no_tensors_or_lie_elsewhere_are_refused(fake, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    here, there, host = on_device(0), on_device(1), torch.ones(5)
    V.vGradNormWorkspace(V.vTensorList([[here]], [[here]]), COMM)
    for grads in ([[None]], [[here, None]], [[here], [None]], [None], [[3]]):        # a frozen parameter's gradient
        refused(V.vTensorList, grads)
    refused(V.vTensorList, [[here]], [[None]])
    for grads in ([[here, there]], [[here], [there]], [[here, host]], [[there]]):
        refused(V.vTensorList, grads)
    for outs in ([[there]], [[host]]):
        refused(V.vTensorList, [[here]], outs)
    assert fake.made == 1


# ---- launch shapes of the norms ------------------------------------------------------------------

SHAPE = ("vecs", "team", "per_cta", "cluster", "threads", "staged", "rounds", "ctas", "smem", "parts")
MOST_SMEM = 227 * 1024 - 2 * 320         # of a CTA, less the kernels' static arrays
ROWS = [1, 2, 3, 31, 76, 77, 153, 300, 1500, 2433, 4096, 9001, 45000, 1 << 20, (1 << 31) - 1]
WIDTHS = [1, 2, 7, 8, 31, 64, 100, 128, 129, 255, 512, 1000, 1031, 2047, 2048, 2731, 4096, 4099, 5120, 8192, 9001, 10241, 12296,
          16384, 20480, 20481, 24001, 32768, 40961, 65535, 65536]


@pytest.mark.parametrize("elem,weight", [(2, 2), (2, 4), (4, 4)])
@pytest.mark.parametrize("mode", ["plain", "groups", "backward"])
def test_launch_shapes_hold_every_row_within_the_hardware(host, elem, weight, mode):
    out = (ctypes.c_int * len(SHAPE))()
    per = 16 // elem
    for hidden in WIDTHS:
        for segments in (1, 2, 3, 4, 5, 9, 17, 33, 64, 65, 66):
            for general in (0, 1) if hidden % per == 0 else (1,):
                for rows in ROWS:
                    host.host_norm_shape(ctypes.c_size_t(rows), hidden, elem, weight, segments, general, mode == "backward",
                                         mode == "groups", out)
                    s = dict(zip(SHAPE, out))
                    at = (hidden, segments, general, rows, s)
                    # a row's columns, by the team's threads
                    assert s["vecs"] in (1, 2, 4) and s["cluster"] in (1, 2, 4, 8), at
                    assert s["cluster"] * s["team"] * s["vecs"] * per >= hidden, at
                    assert s["threads"] == s["team"] * s["per_cta"] and s["threads"] % 32 == 0, at
                    assert s["threads"] <= (512 if s["staged"] else 640) and s["smem"] <= MOST_SMEM, at
                    assert s["team"] % 32 == 0 or s["team"] in (1, 2, 4, 8, 16), at
                    # the CTAs of a cluster meet at barriers that only teams of several warps reach
                    assert s["cluster"] == 1 or (s["per_cta"] == 1 and s["team"] > 32), at
                    # a group's maximum is found in neighbouring lanes of one warp
                    if mode == "groups":
                        assert s["vecs"] == 1 or s["team"] * per >= 128, at
                        assert s["cluster"] == 1 or s["team"] * s["vecs"] * per % 128 == 0, at
                    # every row, once
                    if mode == "backward":
                        assert 1 <= s["parts"] <= 16 * 152, at
                    elif s["staged"] and s["rounds"]:
                        assert 1 <= s["rounds"] <= 6, at
                        assert (s["ctas"] - 1) * s["rounds"] * s["per_cta"] < rows <= s["ctas"] * s["rounds"] * s["per_cta"], at
                    elif s["staged"]:
                        assert 1 <= s["ctas"] <= 16 * 152, at


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_backward_workspace_is_enough_whatever_the_buffers_alignment(host, dtype):
    esz = dtype.itemsize
    need = ctypes.c_size_t()
    for ranks in (1, 2, 8, 31):
        host.host_start(ranks)
        for hidden in (8, 100, 1001, 1024, 2048, 4096, 9001, 16384, 65536):
            for rows in (1, 40, 200, 1500, 20000):
                desc = V.vRmsNormDesc(rows, hidden, dtype)
                d = ctypes.addressof(desc)
                assert host.vRmsNormBackwardWorkspace(d, COMM, ctypes.addressof(need)) == V.vSuccess
                for offset in (0, esz):
                    for residual in (None, 0x50000):
                        bufs = ints(*[0x100000 + offset] * ranks)
                        a = ctypes.addressof(bufs)
                        assert host.vAllReduceRmsNormBackward(d, a, 0x30000, 0x40000, 0x60000, residual, a, 0x70000, 0x80000,
                                                              need.value, COMM, None) == V.vSuccess, (ranks, hidden, rows)
