"""The angles of linear attention's rotation (no GPU): the device functions of la.cuh that form them, compiled for the host with
a trap on signed overflow, which the language leaves undefined, against 64-bit and whole-number arithmetic.  Integers hold the
angle modulo a turn to 2^-32 of it, and its conversion to fp32 to 2^-24 of a half turn: 2 pi 2^-32 + pi 2^-24 = 1.9e-7."""
import ctypes
import math
import os
import re
import subprocess
from fractions import Fraction

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "recurrent_state_update_gb300", "csrc")
HOST = """
#include <cmath>
#include <cstdint>
#include <cstring>
struct float2 { float x, y; };
static uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
static uint64_t __umul64hi(uint64_t a, uint64_t b) { return (uint64_t)(((unsigned __int128)a * b) >> 64); }
static void sincospif(float x, float *s, float *c) { *s = (float)std::sin(M_PI * x); *c = (float)std::cos(M_PI * x); }
%s
extern "C" void angles(const float *freq, const int32_t *pos, int n, float *out) {
    for (int i = 0; i < n; ++i) {
        const float2 r = turned(turns(freq[i]), pos[i]);
        out[2 * i] = r.x, out[2 * i + 1] = r.y;
    }
}
int main() {
    const float freq[4] = {1.0f, 0.5f, 1e-4f, 0.0f};
    const int32_t pos[8] = {0, 1, 3, 4, 131072, INT32_MAX, -1, INT32_MIN};
    volatile float used;  // (or the compiler leaves the calls out)
    for (volatile float f : freq)
        for (volatile int32_t p : pos) used = turned(turns(f), p).x;
    return 0;
}
"""


@pytest.fixture(scope="module")
def source(tmp_path_factory):
    text = open(os.path.join(CSRC, "la.cuh")).read()
    parts = [re.search(r"__device__ __forceinline__ (%s \(?%s\(.*?\n}\n)" % (kind, name), text, re.S).group(1)
             for kind, name in (("uint64_t", "turns"), ("float2", "turned"))]
    at = tmp_path_factory.mktemp("angles") / "angles.cpp"
    at.write_text(HOST % "".join("static " + p for p in parts))
    return at


def test_no_angle_overflows_a_signed_number(source):
    exe = source.with_suffix(".exe")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", str(source), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], timeout=60)
    assert r.returncode == 0, "a signed product overflowed"


def test_angles_at_every_position(source):
    lib = source.with_suffix(".so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(source), "-o", str(lib)], check=True)
    g = np.random.default_rng(5)
    freq = np.concatenate([[1.0, 1.0, 0.5, 0.0, 1e-30], 10000.0 ** -g.random(2000)]).astype(np.float32)
    pos = np.concatenate([[2 ** 31 - 1, -2 ** 31, 4, 7, 2 ** 31 - 1], g.integers(-2 ** 31, 2 ** 31, 2000)]).astype(np.int32)
    out = np.empty((len(freq), 2), np.float32)
    as_p = lambda a, t: a.ctypes.data_as(ctypes.POINTER(t))  # noqa: E731
    ctypes.CDLL(str(lib)).angles(as_p(freq, ctypes.c_float), as_p(pos, ctypes.c_int32), len(freq), as_p(out, ctypes.c_float))
    turn = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)  # 2 pi
    for f, p, (c, s) in zip(freq, pos, out):
        a = float(Fraction(float(f)) * int(p) % turn)
        assert abs(c - math.cos(a)) <= 2.6e-7 and abs(s - math.sin(a)) <= 2.6e-7, (f, p)  # 1.9e-7, and the results' 2^-24
