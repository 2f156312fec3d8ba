"""The exponents of the chunked delta rule's units (gdr_units.h, compiled here
for the host): every factor that the kernels form of them is a finite, normal
fp32 number, and nothing they scale overflows, whatever the state and values."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_depthwise_short_conv1d_amd", "csrc")
SHIM = r"""
#define __host__
#define __device__
#include "gdr_units.h"
extern "C" {
int plain_unit() { return sconv::kPlainUnit; }
int x_scale() { return sconv::kXExp; }
int z_unit() { return sconv::kZExp; }
int x_exp(int e) { return sconv::x_exp(e); }
int held(int e) { return sconv::held_exp(e); }
int first(int e) { return sconv::first_unit(e); }
int for_values(int un, int e) { return sconv::unit_for_values(un, e); }
void step(int un, int zero, int e, int xe, int *out) {
    const sconv::UnitStep s = sconv::next_unit(un, zero != 0, e, xe);
    out[0] = s.up;
    out[1] = s.zu;
}
}
"""
f32 = np.float32


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    src, lib = d / "units.cpp", d / "units.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def step(u, un, zero, e, xe):
    out = (ctypes.c_int * 2)()
    u.step(un, int(zero), e, xe, out)
    return out[0], out[1]


def pow2(e):
    assert -126 <= e <= 127, e
    return f32(2.0) ** f32(e)


def exp_of(u, m):
    m = f32(m)
    if m == 0:
        return u.held(-1000)
    return u.held(0 if not np.isfinite(m) else int(np.frexp(m)[1]))


def test_every_step_has_factors_within_fp32(units):
    """From any unit, by any bound and X: 2^-un, 2^up, 2^zu and the identity's element exist, and the unit stays held."""
    for un in range(-126, 127):
        for e in range(-150, 129, 3):
            for zero in (False, True):
                for xe in (-112, -109, -60, 0, 40, 113, 127):
                    xe = units.x_exp(xe)
                    up, zu = step(units, un, zero, units.held(e), xe)
                    for x in (up, zu, un + up, -(un + up), units.x_scale() - xe, xe - units.z_unit()):
                        assert -126 <= x <= 126, (un, e, zero, xe, up, zu)


def test_first_unit(units):
    for e in range(-149, 129):
        un = units.first(e)
        assert -126 <= un <= 126
        if e > -112:                                   # the state's largest element, below 2^e, comes below 2^14
            assert un + e <= 15


def test_a_state_of_zero_has_the_unit_one(units):
    """... two chunks after the last value at the latest, and it never grows from there."""
    for un in range(-126, 127):
        up, _ = step(units, un, True, units.held(-1000), units.held(-1000))
        un += up
        up, _ = step(units, un, True, units.held(-1000), units.held(-1000))
        assert un + up == 0


def test_lowered_unit_fits_the_values(units):
    top = 90
    for un in range(units.plain_unit() + 1, 127):
        for e in range(-149, 129):
            to = units.for_values(un, units.held(e))
            assert to <= un and to + min(e, 127) <= top
            assert to == un or to + e >= top - 1       # no further than needed


def column(u, chunks, s0, kb):
    """One column of the kernels' scaling in fp32: a chunk is (decay of the whole chunk, largest |v| of it).  z and the next
    state are as large as a rule that contracts can make them: 64 values' sum, each times kb = kf beta, and the state once more."""
    s = f32(s0)
    un = 0 if s == 0 else u.first(exp_of(u, s))
    s = s * pow2(un)
    with np.errstate(under="ignore", over="raise", invalid="raise"):
        for last, v in chunks:
            last, v = f32(last), f32(v)
            if un > u.plain_unit():
                to = u.for_values(un, exp_of(u, v))
                s = f32(np.ldexp(s, to - un))
                un = to
            assert abs(s) < 2 ** 15
            xv = f32(kb) * f32(v * pow2(un))
            xe = u.x_exp(exp_of(u, xv + s))
            to_x, t = pow2(u.x_scale() - xe), f32(2.0 ** (u.z_unit() - u.x_scale()))
            z = t * (f32(64) * (xv * to_x) + s * to_x)
            bound = f32(z * pow2(xe - u.z_unit())) * f32(128) + s * last
            up, zu = step(u, un, bound == 0, exp_of(u, bound), xe)
            un += up
            y = z * pow2(zu)
            assert abs(y) < 65504
            s = s * (last * pow2(up)) + y
            assert np.isfinite(s) and np.isfinite(pow2(-un))
    return s * pow2(-un)


@pytest.mark.parametrize("zeros", range(1, 6))
@pytest.mark.parametrize("decay", [1.0, 0.5, 1e-10, 1e-30, 0.0])
@pytest.mark.parametrize("s0", [0.0, 1e-38, 1e-30, 1.0, 1e30])
def test_values_after_chunks_that_write_nothing(units, zeros, decay, s0):
    for v in (1e-30, 1e-4, 1.0, 200.0, 1e6, 2.0 ** 79):
        if s0 > 1 and v > 1e6:
            continue
        for kb in (1.0, 2.0 ** 20 if v < 2.0 ** 59 else 1.0):
            got = column(units, [(decay, 0.0)] * zeros + [(0.5, v)] * 3, s0, kb)
            assert np.isfinite(got) and got != 0
