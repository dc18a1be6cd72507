"""The sampling's integer weights, in the steps that the kernel takes, against exp in 64 bits."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from collective_communication_virtual_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
BOUND = 2.0 ** -28.8           # of a weight, and one unit


@pytest.fixture(scope="module")
def weights(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("weight") / "sample_weight.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-ffp-contract=off", "-fPIC", "-shared", "-I", build.CSRC,
                    os.path.join(HERE, "sample_weight_host.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).sample_weights
    f.argtypes, f.restype = [ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_void_p], None

    def get(top, temperature, x):
        x = np.ascontiguousarray(x, dtype=np.float32)
        out = np.empty(x.size, dtype=np.uint64)
        f(float(top), float(temperature), x.ctypes.data, x.size, out.ctypes.data)
        return out
    return get


def far_off(got, top, temperature, x):
    """How far beyond one unit, in shares of the weight."""
    want = np.exp((x.astype(np.float64) - float(top)) / float(temperature)) * 2.0 ** 44
    return ((np.abs(got.astype(np.float64) - want) - 1.0) / want)[want > 2.0 ** 8]


@pytest.mark.parametrize("decade", [0, -1, 1, -6, 6, -30, 30])
def test_weights_are_right_to_their_bound(weights, decade):
    rng = np.random.default_rng(100 + decade)
    worst = 0.0
    for _ in range(60):
        temperature = np.float32(rng.uniform(0.2, 2.0) * 10.0 ** decade)
        top = np.float32(rng.normal() * 20.0 * temperature)
        x = (top - temperature * rng.uniform(0, 28, 50000)).astype(np.float32)
        off = far_off(weights(top, temperature, x), top, temperature, x)
        worst = max(worst, off.max())
        assert worst <= BOUND, (temperature, top, x[off.argmax()])
    assert worst > 2.0 ** -31      # (the inputs reach the bound's order)


def test_weights_where_exponents_are_cut(weights):
    # next to the middle between two 32nds, where the series has its longest way to go
    rng = np.random.default_rng(5)
    for k in range(0, 1200, 7):
        z = np.float64((k + 0.5) / 32 * np.log(2.0))
        x = np.float32(-z) + np.arange(-500, 500, dtype=np.float32) * np.spacing(np.float32(z))
        for temperature in (1.0, np.float32(rng.uniform(0.5, 1.5))):
            scaled = (x.astype(np.float64) * float(temperature)).astype(np.float32)
            off = far_off(weights(0.0, temperature, scaled), 0.0, temperature, scaled)
            assert off.size == 0 or off.max() <= BOUND


def test_weights_at_the_ends(weights):
    inf, one = np.float32(np.inf), 1 << 44
    assert weights(3.0, 1.0, [3.0, -inf, -1e30]).tolist() == [one, 0, 0]
    assert weights(inf, 1.0, [inf, 5.0, -inf]).tolist() == [one, 0, 0]
    assert weights(0.0, inf, [0.0, -5.0]).tolist() == [one, one]
    assert weights(2.0, 1e-38, [2.0, 1.0]).tolist() == [one, 0]
    assert weights(2.0, 1e-45, [2.0, 1.0]).tolist() == [one, 0]
    assert weights(-1e38, 1e30, [-1e38, -3e38]).tolist() == [one, 0]
    x = -np.linspace(0, 31.2, 100001, dtype=np.float32)          # 2^-45: nothing is left
    got = weights(0.0, 1.0, x).astype(np.int64)
    assert got[-1] == 0 and (np.diff(got)[np.diff(x) < 0] <= np.maximum(got[:-1] * BOUND * 2, 1)).all()
