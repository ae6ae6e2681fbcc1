"""Host side of a layer's row operators at the ends of what they take (no GPU)."""
import copy
import ctypes
import os
import pickle
import subprocess

import numpy as np
import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from _parity import ensure_built

OK, INVALID = 0, 1


@pytest.fixture(scope="module")
def L():
    ensure_built()
    return bs.lib()


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("base,rot,s", [
    (1e4, 64, dict(kind=1, factor=1e-310)),                                          # f / factor
    (1e4, 16, dict(kind=2, factor=1e-308)),                                          # 1e-308^(16 / 14) underflows: 0^-x
    (1e4, 64, dict(kind=2, factor=1e308)),                                           # the base overflows
    (1e4, 64, dict(kind=3, factor=1e-310, original=100.0, low=1.0, high=4.0)),
    (1e4, 64, dict(kind=4, factor=1e-310, original=100.0, low=1.0, high=4.0)),
    (1e4, 64, dict(kind=5, divisors=[1.0] * 31 + [1e-320])),
    (1e4, 64, dict(kind=1, factor=2.0, amplitude=3.5e38)),                           # finite, but not as a float
    (1e4, 64, dict(kind=5, divisors=[1.0] * 32, amplitude=1e300))])
def test_turns_that_are_not_finite_are_refused(L, base, rot, s):
    s = dict(s)
    div = (ctypes.c_double * 32)(*s.pop("divisors")) if "divisors" in s else None
    scaling = bs.RopeScaling(**s, divisors=None if div is None else ctypes.addressof(div))
    turns, amp = (ctypes.c_uint64 * 64)(*[77] * 64), ctypes.c_float(-3.0)
    assert L.scout_rope_turns(base, rot, ctypes.byref(scaling), turns, ctypes.byref(amp)) == INVALID
    assert list(turns) == [77] * 64 and amp.value == -3.0


@pytest.mark.parametrize("base,rot,s,first,last", [
    (1e308, 64, {}, None, 0.0),                                                      # the last pairs stand still
    (1e4, 64, dict(kind=1, factor=1e300), 0.0, 0.0),
    (1e4, 64, dict(kind=2, factor=1e-308), 0.15915494309189535, None),               # 1e4 1e-308^(64 / 62) is 1e-314, its pairs below 1e305
    (1e4, 64, dict(kind=1, factor=2.0, amplitude=3.4e38), None, None)])
def test_turns_at_the_ends_of_what_is_finite(L, base, rot, s, first, last):
    turns, amp = (ctypes.c_uint64 * 32)(*[77] * 32), ctypes.c_float(-3.0)
    scaling = ctypes.byref(bs.RopeScaling(**s)) if s else None
    assert L.scout_rope_turns(base, rot, scaling, turns, ctypes.byref(amp)) == OK
    got = [t / 2.0 ** 64 for t in turns]
    assert all(0.0 <= t < 1.0 for t in got) and amp.value == pytest.approx(s.get("amplitude", 1.0))
    assert first is None or got[0] == pytest.approx(first, abs=2.0 ** -60)
    assert last is None or got[-1] == pytest.approx(last, abs=2.0 ** -60)


# ---------------------------------------------------------------------------
# Rope
# ---------------------------------------------------------------------------
def test_a_rope_is_read_only(L):
    # calls use the arguments that were put together when it was made: a field that could be set would not reach them
    r = bs.rope(1e4, 64, layout="interleaved", scaling={"kind": "linear", "factor": 2.0, "amplitude": 1.5}, device="cpu")
    for name, value in (("amplitude", 2.0), ("layout", "half"), ("rot_dim", 32), ("turns", r.turns.clone()), ("other", 1)):
        with pytest.raises(AttributeError):
            setattr(r, name, value)
        if name != "other":
            with pytest.raises(AttributeError):
                delattr(r, name)
    assert (r.rot_dim, r.layout, r.amplitude) == (64, "interleaved", 1.5) and r.turns.numel() == 32


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))], ids=["copy", "deepcopy", "pickle"])
def test_a_rope_is_copied_whole(L, how):
    r = bs.rope(1e4, 64, layout="interleaved", scaling={"kind": "linear", "factor": 2.0, "amplitude": 1.5}, device="cpu")
    c = how(r)
    assert (c.rot_dim, c.layout, c.amplitude) == (64, "interleaved", 1.5) and torch.equal(c.turns, r.turns)
    assert c._args[0] is c.turns and c._args[1:] == r._args[1:]


@pytest.mark.parametrize("rot", [2 ** 32 + 64, 2 ** 31 + 64, -2 ** 32 + 64, 2 ** 70])
def test_a_rope_of_more_channels_than_32_bits_hold_is_refused(L, rot):
    # not cut to its low 32 bits, which name 64 channels here
    x, p = torch.zeros((2, 3, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(bs.ScoutError, match="rot_dim"):
        bs.rotate(x, p, bs.Rope(torch.zeros(32, dtype=torch.int64), rot, "half", 1.0))
    with pytest.raises(bs.ScoutError):
        bs.rope(1e4, rot, device="cpu")


# ---------------------------------------------------------------------------
# cosine and sine of a turn
# ---------------------------------------------------------------------------
# csrc/rotate.cuh's sincos_turn itself, its intrinsics written as the host's (each a single rounding).  With u = 2^-24 and
# z = x^2 at most 1/64, errors to first order:
#   x is off by u of itself (the integer's conversion), z by 3 u of itself.
#   sine: the inner steps leave 46.5 u; the last one z 46.5 u + 3 u 0.65 + its rounding 4 u (half a step in [4, 8)) + the
#   constant's rounding 2.9 u + the fit 0.1 u = 9.7 u of at least 5.65, 1.7 u; times x and rounded: 3.7 u of the sine.
#   cosine: the inner steps leave 36 u; the last one z 36 u + 3 u 0.3 + its rounding u / 2 = 2 u of at least 0.7: 2.8 u.
# Odd quarters exchange the two.
SIN, COS = 4 * 2.0 ** -24, 3 * 2.0 ** -24


@pytest.fixture(scope="module")
def sincos(tmp_path_factory):
    csrc = os.path.join(os.path.dirname(bs.__file__), "csrc")
    with open(os.path.join(csrc, "rotate.cuh")) as f:
        text = f.read()
    at = text.index("__device__ __forceinline__ void sincos_turn")
    body = text[at:text.index("\n}\n", at) + 3]
    d = tmp_path_factory.mktemp("sincos")
    (d / "s.cpp").write_text("""#include <cmath>
#include <cstdint>
#include <cstring>
#define __device__
#define __forceinline__ inline
static float __fmul_rn(float a, float b) { return a * b; }
static float __fmaf_rn(float a, float b, float c) { return std::fma(a, b, c); }
static float __uint_as_float(uint32_t v) { float f; std::memcpy(&f, &v, 4); return f; }
static uint32_t __float_as_uint(float f) { uint32_t v; std::memcpy(&v, &f, 4); return v; }
""" + body + """extern "C" void run(const uint32_t* t, long n, float* s, float* c) {
  for (long i = 0; i < n; ++i) sincos_turn(t[i], s[i], c[i]);
}
""")
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-o", d / "s.so", d / "s.cpp"], check=True)
    run = ctypes.CDLL(str(d / "s.so")).run

    def call(t):
        s, c = np.empty(len(t), np.float32), np.empty(len(t), np.float32)
        run(*(ctypes.c_void_p(a.ctypes.data) if i != 1 else ctypes.c_long(a) for i, a in enumerate((t, len(t), s, c))))
        return s, c
    return call


def test_cosine_and_sine_of_a_turn_are_within_their_bounds(sincos):
    rng = np.random.default_rng(0)
    near = np.concatenate([np.arange(-3000, 3001), [2 ** k for k in range(12, 29)], [-2 ** k for k in range(12, 29)]])
    t = np.concatenate([(np.arange(8)[:, None] * 2 ** 29 + near).ravel(), rng.integers(0, 2 ** 32, 1 << 20),
                        rng.integers(0, 2 ** 26, 1 << 16) - 2 ** 25]) % 2 ** 32
    s, c = sincos(np.ascontiguousarray(t.astype(np.uint32)))
    quarter = (t + 2 ** 29) // 2 ** 30 % 4
    rest = (t + 2 ** 29) % 2 ** 30 - 2 ** 29  # exact
    a = rest * (2 * np.pi / 2 ** 32)
    sin, cos = np.sin(a), np.cos(a)
    want_s, want_c = np.choose(quarter, [sin, cos, -sin, -cos]), np.choose(quarter, [cos, -sin, -cos, sin])
    odd = quarter % 2 == 1
    for got, want, bound in ((s, want_s, np.where(odd, COS, SIN)), (c, want_c, np.where(odd, SIN, COS))):
        assert np.all(np.abs(got - want) <= bound * np.abs(want))
