"""Host side of a layer's row operators at the ends of what they take (no GPU)."""
import copy
import ctypes
import pickle

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
