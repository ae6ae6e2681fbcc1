"""Host side of a layer's row operators: the frequencies of rotary positions, refusals before any launch, and
the oracle's own pins (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from oracle import rows_oracle as R
from _parity import ensure_built

OK, INVALID, UNSUPPORTED = 0, 1, 2
F = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)  # 8 bytes past a 16-byte boundary
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    ensure_built()
    return bs.lib()


def call(fn, args, **change):
    assert set(change) <= set(args)
    return fn(*dict(args, **change).values())


def rope(turns=4096, rot=128, layout=0, amp=1.0):
    return ctypes.pointer(bs.RopeArgs(turns, rot, layout, amp))


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
SCALINGS = [None, {"kind": "linear", "factor": 4.0}, {"kind": "linear", "factor": 0.5}, {"kind": "ntk", "factor": 8.0},
            {"kind": "rotations", "factor": 8.0, "original": 8192.0}, {"kind": "index", "factor": 4.0, "original": 32768.0},
            {"kind": "rotations", "factor": 2.0, "original": 500.0, "low": 0.5, "high": 30.0, "amplitude": 1.5},
            {"kind": "index", "factor": 0.5, "original": 100.0, "low": 2.0, "high": 3.0}]


@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: "none" if s is None else s["kind"])
@pytest.mark.parametrize("base,rot", [(1e4, 128), (1e6, 128), (5e5, 64), (1e4, 16), (1.5, 48)])
def test_turns_are_the_frequencies_in_fractions_of_a_turn(L, base, rot, scaling):
    r = bs.rope(base, rot, scaling=scaling, device="cpu")
    f, amp = R.frequencies(base, rot, scaling)
    turns = r.turns.numpy().view(np.uint64)
    assert turns.shape == (rot // 2,) and r.rot_dim == rot and r.amplitude == np.float32(amp)
    got = turns.astype(np.float64) / 2.0 ** 64  # the library keeps 53 bits
    # a dozen roundings of 2^-53 on either side (a power's error included), and the integer's, below 2^-64
    want = f / (2 * math.pi) % 1.0
    assert np.all(np.abs(got - want) <= 32 * 2.0 ** -53 * np.maximum(want, f / (2 * math.pi)) + 2.0 ** -64)


def test_divisors_scale_each_pair(L):
    div = np.linspace(0.25, 9.0, 32)
    f, _ = R.frequencies(1e4, 64, {"kind": "divisors", "divisors": div, "factor": 1.0})
    r = bs.rope(1e4, 64, scaling={"kind": "divisors", "divisors": div, "amplitude": 1.25}, device="cpu")
    want = f / (2 * math.pi) % 1.0
    assert np.allclose(r.turns.numpy().view(np.uint64) / 2.0 ** 64, want, rtol=1e-14, atol=2.0 ** -64) and r.amplitude == 1.25


@pytest.mark.parametrize("base,rot,s,rc", [
    (1.0, 64, {}, INVALID), (NAN, 64, {}, INVALID), (INF, 64, {}, INVALID), (1e4, 0, {}, UNSUPPORTED),
    (1e4, 24, {}, UNSUPPORTED), (1e4, 144, {}, UNSUPPORTED), (1e4, -16, {}, UNSUPPORTED),
    (1e4, 64, dict(kind=0), INVALID), (1e4, 64, dict(kind=6), INVALID), (1e4, 64, dict(kind=1, factor=0.0), INVALID),
    (1e4, 64, dict(kind=2, factor=-1.0), INVALID), (1e4, 64, dict(kind=1, factor=NAN), INVALID),
    (1e4, 64, dict(kind=3, factor=2.0, low=1.0, high=4.0), INVALID),
    (1e4, 64, dict(kind=3, factor=2.0, original=9.0, low=4.0, high=4.0), INVALID),
    (1e4, 64, dict(kind=4, factor=2.0, original=9.0, low=0.0, high=4.0), INVALID),
    (1e4, 64, dict(kind=4, factor=2.0, original=9.0, low=1.0, high=INF), INVALID),
    (1e4, 64, dict(kind=5), INVALID), (1e4, 64, dict(kind=1, factor=2.0, amplitude=-1.0), INVALID),
    (1e4, 64, dict(kind=1, factor=2.0, amplitude=NAN), INVALID), (1e4, 64, dict(kind=1, factor=2.0), OK)])
def test_turns_refusals(L, base, rot, s, rc):
    turns, amp = (ctypes.c_uint64 * 64)(*[77] * 64), ctypes.c_float(-3.0)
    assert L.scout_rope_turns(base, rot, ctypes.byref(bs.RopeScaling(**s)) if s else None, turns, ctypes.byref(amp)) == rc
    assert rc == OK or (list(turns) == [77] * 64 and amp.value == -3.0)


def test_turns_null_pointers_and_a_bad_divisor(L):
    turns, amp = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    assert L.scout_rope_turns(1e4, 64, None, None, ctypes.byref(amp)) == INVALID
    assert L.scout_rope_turns(1e4, 64, None, turns, None) == INVALID
    for bad in (0.0, -1.0, NAN):
        with pytest.raises(bs.ScoutError, match="INVALID"):
            bs.rope(1e4, 16, scaling={"kind": "divisors", "divisors": [1.0] * 7 + [bad]}, device="cpu")


def test_rope_refuses_names_it_does_not_know(L):
    for kw in (dict(layout="pairs"), dict(scaling={"kind": "log"}), dict(scaling={"kind": "linear"}),
               dict(scaling={"kind": "linear", "factor": 2.0, "original": 5.0}), dict(scaling={"kind": "index", "factor": 2.0}),
               dict(scaling={"kind": "divisors", "divisors": [1.0] * 3})):
        with pytest.raises(bs.ScoutError):
            bs.rope(1e4, 64, device="cpu", **kw)
    with pytest.raises(bs.ScoutError, match="layout"):
        bs.Rope(None, 64, "both", 1.0)


# ---------------------------------------------------------------------------
# refusals of the C ABI (every call is turned away on the host)
# ---------------------------------------------------------------------------
NORM = dict(kind=0, Y=F, ld_y=64, w_post=None, b_post=None, gate=None, ld_gate=0, alpha=1.0, h_type=0, H=F, ld_h=64, H_out=F,
            ld_ho=64, w=F, b=None, X=F, w_ahead=None, b_ahead=None, X_ahead=None, M=0, N=64, eps=1e-6, stream=None)


@pytest.mark.parametrize("change,rc", [
    ({}, OK), (dict(kind=2), INVALID), (dict(h_type=2), INVALID), (dict(H=None), INVALID), (dict(w=None), INVALID),
    (dict(X=None), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(ld_h=56), INVALID), (dict(ld_y=0), INVALID),
    (dict(ld_ho=8), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(alpha=NAN), INVALID), (dict(alpha=INF), INVALID), (dict(H_out=None), INVALID), (dict(Y=None), INVALID),
    (dict(Y=None, H_out=None), OK), (dict(Y=None, H_out=None, gate=F), INVALID), (dict(Y=None, H_out=None, w_post=F), INVALID),
    (dict(gate=F, ld_gate=32), INVALID), (dict(gate=F, ld_gate=64), OK), (dict(gate=F, ld_gate=68), UNSUPPORTED),
    (dict(w_ahead=F), INVALID), (dict(X_ahead=F), INVALID), (dict(w_ahead=F, X_ahead=F), OK), (dict(b=F), INVALID),
    (dict(b=F, kind=1), OK), (dict(b_post=F, kind=1), INVALID), (dict(b_ahead=F, kind=1), INVALID),
    (dict(b_post=F, w_post=F), INVALID), (dict(N=60), UNSUPPORTED),
    (dict(N=32776, ld_y=32776, ld_h=32776, ld_ho=32776), UNSUPPORTED),
    (dict(N=32768, ld_y=32768, ld_h=32768, ld_ho=32768), OK), (dict(ld_h=68), UNSUPPORTED), (dict(ld_y=68), UNSUPPORTED),
    (dict(ld_ho=68), UNSUPPORTED), (dict(Y=ODD), UNSUPPORTED), (dict(X=ODD), UNSUPPORTED), (dict(w=ODD), UNSUPPORTED),
    (dict(H=ODD), UNSUPPORTED), (dict(w_ahead=ODD, X_ahead=F), UNSUPPORTED)])
def test_add_norm_refusals(L, change, rc):
    assert call(L.scout_add_norm, NORM, **change) == rc


ROTATE = dict(x=F, ld_x=256, out=F, ld_o=256, pos=F, n=0, heads=2, D=128, rope=rope(), norm=None, eps=0.0, stream=None)
ROPES = [(dict(rope=None), INVALID), (dict(rope=rope(0)), INVALID), (dict(rope=rope(layout=2)), INVALID),
         (dict(rope=rope(amp=NAN)), INVALID), (dict(rope=rope(amp=INF)), INVALID), (dict(rope=rope(4104)), UNSUPPORTED),
         (dict(rope=rope(rot=8)), UNSUPPORTED), (dict(rope=rope(rot=136)), UNSUPPORTED), (dict(rope=rope(rot=0)), UNSUPPORTED),
         (dict(rope=rope(rot=144)), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID)]


@pytest.mark.parametrize("change,rc", ROPES + [
    ({}, OK), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(pos=None), INVALID), (dict(n=-1), INVALID),
    (dict(heads=0), INVALID), (dict(ld_x=248), INVALID), (dict(ld_o=128), INVALID), (dict(ld_x=260), UNSUPPORTED),
    (dict(ld_o=260), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(x=ODD), UNSUPPORTED), (dict(out=ODD), UNSUPPORTED),
    (dict(norm=ODD), UNSUPPORTED), (dict(pos=ctypes.c_void_p(4098)), UNSUPPORTED),
    (dict(heads=(1 << 20) + 1, ld_x=1 << 28, ld_o=1 << 28), UNSUPPORTED)])
def test_rotate_refusals(L, change, rc):
    assert call(L.scout_rotate, ROTATE, **change) == rc


APPEND = dict(K=F, ld_k=256, V=F, ld_v=256, pos=F, rope=rope(), k_norm=None, eps=0.0, map=F, n=0, Hkv=2, D=128, P=32, Kp=F,
              Vp=F, n_slots=10, q=F, ld_q=512, Hq=4, q_norm=None, q_out=F, ld_qo=512, status=None, stream=None)
QUERIES = [(dict(Hq=-1), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(ld_q=256), INVALID),
           (dict(ld_qo=504), INVALID), (dict(ld_q=516), UNSUPPORTED), (dict(q=ODD), UNSUPPORTED), (dict(q_out=ODD), UNSUPPORTED),
           (dict(q_norm=ODD), UNSUPPORTED)]


@pytest.mark.parametrize("change,rc", ROPES + QUERIES + [
    ({}, OK), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(pos=None), INVALID), (dict(map=None), INVALID),
    (dict(Kp=None), INVALID), (dict(Vp=None), INVALID), (dict(n=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(n_slots=0), INVALID), (dict(ld_k=128), INVALID), (dict(ld_v=248), INVALID), (dict(ld_v=260), UNSUPPORTED),
    (dict(ld_k=260), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(P=8), UNSUPPORTED), (dict(K=ODD), UNSUPPORTED),
    (dict(V=ODD), UNSUPPORTED), (dict(Kp=ODD), UNSUPPORTED), (dict(Vp=ODD), UNSUPPORTED), (dict(k_norm=ODD), UNSUPPORTED),
    (dict(map=ctypes.c_void_p(4100)), UNSUPPORTED), (dict(n_slots=1 << 31), UNSUPPORTED),
    (dict(Hq=0, q=None, q_out=None, ld_q=0, ld_qo=0), OK)])
def test_append_rotated_refusals(L, change, rc):
    assert call(L.scout_append_rotated_kv, APPEND, **change) == rc


APPEND8 = dict(fmt=0, K=F, ld_k=256, V=F, ld_v=256, n=4, pos=None, rope=rope(), k_norm=None, eps=0.0, prev=None, seq=F, table=F,
               B=2, Hkv=2, D=128, P=32, cap=8, Kp=F, Vp=F, Ks=F, Vs=F, n_slots=10, q=F, ld_q=512, Hq=4, q_norm=None, q_out=F,
               ld_qo=512, status=None, stream=None)


@pytest.mark.parametrize("change,rc", ROPES + QUERIES + [
    (dict(fmt=2), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(seq=None), INVALID),
    (dict(table=None), INVALID), (dict(Kp=None), INVALID), (dict(Vp=None), INVALID), (dict(Ks=None), INVALID),
    (dict(Vs=None), INVALID), (dict(n=-1), INVALID), (dict(B=0), INVALID), (dict(cap=0), INVALID), (dict(n_slots=0), INVALID),
    (dict(ld_k=128), INVALID), (dict(ld_v=128), INVALID), (dict(ld_v=257), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(P=0), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(cap=8193), UNSUPPORTED),
    (dict(B=4096, cap=8192, P=64), UNSUPPORTED), (dict(Kp=ODD), UNSUPPORTED), (dict(V=ODD), UNSUPPORTED),
    (dict(Vp=ODD), UNSUPPORTED), (dict(n_slots=1 << 31), UNSUPPORTED), (dict(pos=ctypes.c_void_p(4098)), UNSUPPORTED),
    (dict(n=0, K=None, V=None, q=None, q_out=None), OK)])
def test_append_rotated8_refusals(L, change, rc):
    assert call(L.scout_append_rotated_kv8, APPEND8, **change) == rc


PREDICT = dict(X=F, W=F, Q=F, M=8, N=128, K=64, pos=F, rope=rope(), norm=None, eps=0.0, status=None, launch=None, stream=None)


@pytest.mark.parametrize("change,rc", ROPES + [
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(Q=None), INVALID), (dict(M=0), INVALID), (dict(pos=None), INVALID),
    (dict(M=257), UNSUPPORTED), (dict(N=100), UNSUPPORTED), (dict(K=65), UNSUPPORTED), (dict(X=ODD), UNSUPPORTED),
    (dict(norm=ODD), UNSUPPORTED), (dict(launch=ctypes.pointer(bs.Launch(-1))), INVALID)])
def test_predict_rotated_refusals(L, change, rc):
    assert call(L.scout_predict_q_rotated, PREDICT, **change) == rc


READ = dict(Kp=F, Vp=F, n_slots=10, table=F, seq=F, B=2, Hkv=2, D=128, P=32, cap=8, list=F, n_list=0, Ko=F, Vo=F, sb=8192,
            sh=4096, st=128, T=32, host=0, status=None, stream=None)
READ8 = dict(dict(fmt=0, Kp=F, Vp=F, Ks=F, Vs=F), **{k: v for k, v in READ.items() if k not in ("Kp", "Vp")})
READS = [({}, OK), (dict(Kp=None), INVALID), (dict(Vp=None), INVALID), (dict(table=None), INVALID), (dict(seq=None), INVALID),
         (dict(Ko=None), INVALID), (dict(Vo=None), INVALID), (dict(n_slots=0), INVALID), (dict(B=0), INVALID),
         (dict(Hkv=0), INVALID), (dict(cap=0), INVALID), (dict(T=0), INVALID), (dict(sb=-8), INVALID), (dict(sh=-8), INVALID),
         (dict(st=-8), INVALID), (dict(n_list=-1), INVALID), (dict(host=2), INVALID), (dict(D=64), UNSUPPORTED),
         (dict(P=24), UNSUPPORTED), (dict(cap=8193), UNSUPPORTED), (dict(B=1 << 20, cap=1 << 12), UNSUPPORTED),
         (dict(n_slots=1 << 31), UNSUPPORTED), (dict(st=132), UNSUPPORTED), (dict(sh=8), UNSUPPORTED), (dict(sb=24), UNSUPPORTED), (dict(Ko=ctypes.c_void_p(4112)), UNSUPPORTED),
         (dict(Kp=ODD), UNSUPPORTED), (dict(Vo=ODD), UNSUPPORTED), (dict(list=ctypes.c_void_p(4100)), UNSUPPORTED)]


@pytest.mark.parametrize("change,rc", READS)
def test_read_refusals(L, change, rc):
    assert call(L.scout_read_kv, READ, **change) == rc


@pytest.mark.parametrize("change,rc", READS + [(dict(fmt=2), INVALID), (dict(Ks=None), INVALID), (dict(Vs=None), INVALID)])
def test_read8_refusals(L, change, rc):
    assert call(L.scout_read_kv8, READ8, **change) == rc


def test_binding_refuses_host_tensors(L):
    x, p = torch.zeros((2, 3, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    r = bs.rope(1e4, 64, device="cpu")
    with pytest.raises(bs.ScoutError, match="CUDA tensor"):
        bs.rotate(x, p, r)
    with pytest.raises(bs.ScoutError, match=r"\[n_tokens\]"):
        bs.rotate(x[0], p, r)
    with pytest.raises(bs.ScoutError, match="heads of a token"):
        bs.rotate(torch.zeros((2, 128, 3), dtype=torch.bfloat16).transpose(1, 2), p, r)
    with pytest.raises(bs.ScoutError, match="positions must be"):
        bs.rotate(x, p.long(), r)
    with pytest.raises(bs.ScoutError, match="norm must be"):
        bs.rotate(x, p, r, norm=torch.zeros(128))
    with pytest.raises(bs.ScoutError, match="shape of x"):
        bs.rotate(x, p, r, out=x[:1])
    with pytest.raises(bs.ScoutError, match="kind must be"):
        bs.add_norm("max", x[0], x[0], x[0, 0])
    h, w = torch.zeros((3, 128)), torch.zeros(128, dtype=torch.bfloat16)
    for bad, what in ((dict(Y=h), "Y must be"), (dict(H=h.half()), "bf16 or fp32"), (dict(w=w[:8]), "w must be"),
                      (dict(gate=x[:, 0]), "gate must be"), (dict(b_ahead=w), "need w_ahead"), (dict(H_out=h[:2]), "H_out must be"),
                      (dict(X=h), "X must be"), (dict(Y=x[0].t()), "Y must be"), (dict(Y=None, H_out=h), "needs Y")):
        with pytest.raises(bs.ScoutError, match=what):
            bs.add_norm("rms", **dict(dict(Y=x[0], H=h, w=w), **bad))
    with pytest.raises(bs.ScoutError, match="CUDA tensor on"):
        bs.add_norm("rms", x[0], h, w)
    pool, t, n = torch.zeros((4, 32, 128), dtype=torch.bfloat16), torch.zeros((1, 2, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    out = torch.zeros((1, 2, 64, 128), dtype=torch.bfloat16)
    for bad, what in ((dict(K_out=out[0]), "alike"), (dict(V_out=out[:, :, :8]), "alike"), (dict(K_out=out.float()), "alike"),
                      (dict(V_out=out.transpose(1, 2).contiguous().transpose(1, 2)), "same strides"),
                      (dict(K_out=out[:, :, :1].expand(1, 2, 64, 128), V_out=out[:, :, :1].expand(1, 2, 64, 128)), "overlap")):
        with pytest.raises(bs.ScoutError, match=what):
            bs.read_kv(**dict(dict(K_pool=pool, V_pool=pool, page_table=t, seq_len=n, B=1, Hkv=2, P=32, K_out=out, V_out=out), **bad))
    with pytest.raises(bs.ScoutError, match="CUDA tensor on"):
        bs.read_kv(pool, pool, t, n, 1, 2, 32, out, out)
    with pytest.raises(bs.ScoutError, match="K_scale and V_scale"):
        bs.read_kv8(pool, pool, None, None, t, n, 1, 2, 32, out, out)
    with pytest.raises(bs.ScoutError, match="need q"):
        bs.append_rotated_kv(x, x, p, r, torch.zeros((2, 3), dtype=torch.int64), 3, 32, pool, pool, q_norm=w)
    with pytest.raises(bs.ScoutError, match="tokens of K_new"):
        bs.append_rotated_kv(x, x, p, r, torch.zeros((2, 3), dtype=torch.int64), 3, 32, pool, pool, q=x[:1])


# ---------------------------------------------------------------------------
# the oracle's pins
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_oracle_scores_depend_on_the_distance_alone(layout):
    rng = np.random.default_rng(3)
    f, amp = R.frequencies(1e4, 64, None)
    q, k = rng.standard_normal((2, 1, 1, 128))
    turn = lambda x, p: R.rotate(x, np.array([[p]]) * f, 64, layout, amp)[0].ravel()  # noqa: E731
    assert np.isclose(turn(q, 105) @ turn(k, 100), turn(q, 7) @ turn(k, 2), rtol=1e-12)
    assert not np.isclose(turn(q, 105) @ turn(k, 100), turn(q, 7) @ turn(k, 3))
    assert np.isclose(turn(q, 9) @ turn(q, 9), q.ravel() @ q.ravel())
    assert np.array_equal(turn(q, 9)[64:], q.ravel()[64:])


def test_oracle_pair_and_direction():
    x = np.zeros((1, 1, 128))
    x[..., 0] = 1.0
    y = R.rotate(x, np.full((1, 64), np.pi / 2), 128, "half", 2.0)[0].ravel()
    assert np.allclose(y[[0, 64]], [0.0, 2.0]) and np.count_nonzero(np.abs(y) > 1e-9) == 1
    y = R.rotate(x, np.full((1, 64), np.pi / 2), 128, "interleaved", 1.0)[0].ravel()
    assert np.allclose(y[[0, 1]], [0.0, 1.0])


def test_oracle_norms():
    x = np.random.default_rng(0).standard_normal((4, 96)) * 3 + 5
    one = np.ones(96)
    y = R.norm(x, "layer", one, None, 0.0)[0]
    assert np.allclose(y.mean(1), 0) and np.allclose((y * y).mean(1), 1)
    y = R.norm(x, "rms", one, None, 0.0)[0]
    assert np.allclose((y * y).mean(1), 1) and np.allclose(y / x, (y / x)[:, :1])
    assert np.allclose(R.norm(x, "layer", 2 * one, 3 * one, 1e9)[0], 3.0, atol=1e-3)


def test_oracle_angles_of_far_positions():
    turns = [1 << 62, (1 << 64) - 1, 3]
    a = R.angles([0, 1, 2, 2 ** 31 - 1], turns)
    assert np.allclose(a[:, 0], [0, np.pi / 2, -np.pi, -np.pi / 2])
    assert np.allclose(a[:, 1], -2 * np.pi * np.array([0, 1, 2, 2 ** 31 - 1]) / 2.0 ** 64, rtol=1e-12, atol=0)
