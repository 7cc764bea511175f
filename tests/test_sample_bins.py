"""The sampler's bins (csrc/sample_bins.h) on the host, over rows whose spread and temperature take every extreme."""
import ctypes
import itertools
import math
import os
import subprocess

import numpy as np
import pytest

from memory_bound_decode_gemv_amd import _build

SOURCE = """
#include "sample_bins.h"
extern "C" float scale_of(float m, float low, float reach) { return dg::bin_scale(m, low, reach); }
extern "C" float place_of(float m, float x, float scale) { return dg::bin_place(dg::bin_distance(m, x), scale); }
extern "C" int bins() { return dg::kBins; }
"""
BIG = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("bins")
    src, obj, lib = (str(tmp / n) for n in ("bins.hip", "bins.o", "bins.so"))
    open(src, "w").write(SOURCE)
    subprocess.run([_build.hipcc(), "--offload-host-only", "-O2", "-std=c++17", "-fPIC", "-I", _build.CSRC, "-c", src,
                    "-o", obj], check=True, capture_output=True)
    subprocess.run(["g++", "-shared", "-o", lib, obj], check=True, capture_output=True)
    m = ctypes.CDLL(lib)
    f = ctypes.c_float
    m.scale_of.argtypes, m.scale_of.restype = [f, f, f], f
    m.place_of.argtypes, m.place_of.restype = [f, f, f], f
    return m


def rows():
    """(maximum, smallest finite value, temperature, fraction bits)"""
    values = [0.0, 1.0, -3.0, 20.5, 1e-40, -1e-40, 1e30, -1e30, BIG, -BIG, BIG / 2]
    for m, low in itertools.product(values, values):
        if low <= m:
            for T, F in itertools.product((1e-45, 1e-30, 0.01, 1.0, 1e30, 1e36, 1.3e37, 1e38, math.inf), (31, 51)):
                yield np.float32(m), np.float32(low), np.float32(T), F


def reach(T, F):
    with np.errstate(over="ignore"):
        return np.float32(np.float32(F + 1) * np.float32(0.69314718)) * T


def test_masked_tokens_and_padding_are_in_the_last_bin(rule):
    """-infinity is behind every border, or in the last bin, whose elements are sifted by weight: it is also what stands
    for the places behind a row's end, which are never listed."""
    last = rule.bins() - 1
    for m, low, T, F in rows():
        scale = rule.scale_of(m, low, reach(T, F))
        assert rule.place_of(m, -math.inf, scale) == last, (m, low, T, F, scale)
    assert rule.place_of(math.inf, -math.inf, rule.scale_of(math.inf, 0.0, 1.0)) == last


def test_bins_follow_the_order_of_values(rule):
    """The maximum is in bin 0, places do not fall with falling values, and a value without weight (from the reach on) is
    in the last bin unless the steps are at their finest."""
    last = rule.bins() - 1
    for m, low, T, F in rows():
        far = reach(T, F)
        scale = rule.scale_of(m, low, far)
        xs = np.linspace(float(m), float(low), 17).astype(np.float32)   # falling
        places = [rule.place_of(m, x, scale) for x in xs]
        assert rule.place_of(m, m, scale) == 0.0
        assert all(a <= b for a, b in zip(places, places[1:])) and max(places) <= last
        with np.errstate(over="ignore"):
            beyond = np.float32(m - np.float32(1.001) * far)
        if np.isfinite(far) and low < beyond < m - far and scale < np.float32(1e30):
            assert rule.place_of(m, beyond, scale) == last


def test_rows_of_one_value_share_the_first_bin(rule):
    for v in (0.0, -7.25, BIG, -BIG, 1e-45):
        for T in (1e-45, 1.0, math.inf):
            assert rule.place_of(v, v, rule.scale_of(v, v, reach(np.float32(T), 51))) == 0.0
