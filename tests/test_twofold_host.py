"""The rotary angles of twofold.cuh, compiled for the host with the device's rounding functions written out:
(cos, sin) of a turn in two floats each, against 64 bits."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from decode_attention_gb300 import build

HOST = r"""
#include <cmath>
#include <cstdint>
#include <cstring>
#define __device__
#define __host__
#define __forceinline__ inline
static inline float __fadd_rn(float a, float b) { return a + b; }
static inline float __fsub_rn(float a, float b) { return a - b; }
static inline float __fmul_rn(float a, float b) { return a * b; }
static inline float __fmaf_rn(float a, float b, float c) { return std::fma(a, b, c); }
static inline int __float_as_int(float x) { int i; std::memcpy(&i, &x, 4); return i; }
static inline float __int_as_float(int i) { float x; std::memcpy(&x, &i, 4); return x; }
#include "kernels/twofold.cuh"
extern "C" void angles(const uint64_t *f, int n, float *out) {
    for (int i = 0; i < n; ++i) {
        gqa::Twofold c, s;
        gqa::cos_sin_nearest(f[i], &c, &s);
        out[4 * i] = c.h, out[4 * i + 1] = c.l, out[4 * i + 2] = s.h, out[4 * i + 3] = s.l;
    }
}
"""


@pytest.fixture(scope="module")
def angles(tmp_path_factory):
    d = tmp_path_factory.mktemp("twofold")
    (d / "host.cpp").write_text(HOST)
    so = str(d / "host.so")
    # (no contraction: the order of the roundings is the source's)
    subprocess.run(["g++", "-shared", "-fPIC", "-O2", "-ffp-contract=off", "-std=c++17", "-I", build.CSRC,
                    str(d / "host.cpp"), "-o", so], check=True)
    fn = ctypes.CDLL(so, mode=os.RTLD_LOCAL).angles

    def run(f):
        f = np.ascontiguousarray(f, dtype=np.uint64)
        out = np.empty((f.size, 4), dtype=np.float32)
        fn(f.ctypes.data_as(ctypes.c_void_p), f.size, out.ctypes.data_as(ctypes.c_void_p))
        return out.astype(np.float64)
    return run


def turns():
    rng = np.random.default_rng(11)
    some = rng.integers(0, 1 << 64, 1 << 20, dtype=np.uint64, endpoint=False)
    small = some[:1 << 16] >> rng.integers(0, 60, 1 << 16).astype(np.uint64)
    eighths = np.arange(8, dtype=np.uint64) << np.uint64(61)
    near = (eighths[:, None] + np.arange(-200, 201).astype(np.int64).astype(np.uint64) * np.uint64(1 << 30)).ravel()
    # positions up to the longest cache's, pairs of both geometries
    freq = np.concatenate([1e4 ** (-2.0 * np.arange(128) / 256), 1e6 ** (-2.0 * np.arange(64) / 512)]) / (2 * np.pi)
    pos = np.concatenate([np.arange(64), 262143 - np.arange(64)]).astype(np.uint64)
    real = ((freq * 2.0 ** 64).astype(np.uint64)[None] * pos[:, None]).ravel()
    return np.concatenate([some, small, near, real])


def test_angles(angles):
    """Both floats: 2^-30.  The high one alone: half its spacing and that, 2^-24 of itself at most but for
    the smallest."""
    f = turns()
    got = angles(f)
    a = 2 * np.pi * (f.astype(np.float64) * 2.0 ** -64)
    for k, want in ((0, np.cos(a)), (2, np.sin(a))):
        high, low = got[:, k], got[:, k + 1]
        assert np.abs(high + low - want).max() <= 2.0 ** -30
        half = np.spacing(np.abs(high).astype(np.float32)).astype(np.float64) / 2
        assert np.all(np.abs(high - want) <= half + 2.0 ** -30)
        assert np.all(np.abs(low) <= half)
