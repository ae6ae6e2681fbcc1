"""GPU parity of a layer's row operators against the fp64 oracle (oracle/rows_oracle.py).

Tolerances, u = 2^-24 the unit of an fp32 rounding.  A result rounded to bf16 is off by 2^-8 of itself beside
its fp32 error.

Turned heads, with s the length of a channel's pair (amplitude and norm included): the angle is off by 2^-33 of a turn,
0.02 u s; sine and cosine by 4 u of themselves (tests/test_rows_limits_host.py), the amplitude's product by u, one of the
two products by u and their sum by u: 7.1 u s, as the products' magnitudes add up to s at most.  The norm: its sum has 4
roundings of positive terms in a lane and 5 where lanes are joined, and the eps, which count half in the root, rsqrtf 2 ulp =
4 u, two products: 11 u.  Together below 32 u s.

Predicted queries: K products summed in fp32, each partial sum off by at most 2 u (the tensor core cuts) of sum_k |x_k w_k|:
e = (2 K + 16) u sum |x w| for each entry before norm and turn.  A norm multiplies an entry's error by its factor and adds the
relative error of the row's length, |e| / |q|.

Norms over N: a sum has at most 64 sequential terms of a thread and 10 joins, 74 u of a sum of magnitudes, half of it in the
root; the mean of "layer" 74 u of the mean magnitude."""
import threading

import numpy as np
import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from oracle import cache8_oracle as C8
from oracle import rows_oracle as R
from _parity import ensure_built

pytestmark = pytest.mark.gpu
D = 128
U = 2.0 ** -24
DT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def bf16(rng, *shape, gain=True):
    x = rng.standard_normal(shape).astype(np.float32)
    if gain:
        x[..., rng.integers(0, shape[-1], 3)] *= 7.0
    return torch.from_numpy(x).to(torch.bfloat16).cuda()


def weight(rng, n):
    return torch.from_numpy((1 + 0.3 * rng.standard_normal(n)).astype(np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def same(a, b):
    """Bit for bit, NaN included."""
    return a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def turns_of(rope):
    return rope.turns.cpu().numpy().view(np.uint64)


def expected(x, pos, rope, norm=None, eps=0.0):
    """(turned heads, tolerance) of bf16 x [n][heads][D]."""
    y, size = R.rotate(f64(x), R.angles(np.maximum(pos, 0), turns_of(rope)), rope.rot_dim, rope.layout, rope.amplitude,
                       None if norm is None else f64(norm), eps)
    return y, 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * 32 * U * size


def strided(rng, n, heads, pad):
    """Rows inside a wider buffer -> (view [n][heads][D], the buffer)."""
    whole = bf16(rng, n, heads * D + pad)
    return whole[:, :heads * D].unflatten(1, (heads, D)), whole


# ---------------------------------------------------------------------------
# rotate
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,rot,normed,pad", [
    (1, 1, 128, False, 0), (1, 40, 128, True, 0), (2, 3, 16, True, 8), (3, 7, 48, False, 24), (4, 8, 112, True, 128),
    (5, 9, 64, False, 0), (7, 64, 96, True, 8), (33, 5, 32, True, 16), (130, 17, 80, False, 8)])
def test_rotate(layout, n, heads, rot, normed, pad):
    rng = np.random.default_rng(n * 100 + rot)
    rope = bs.rope(1e4, rot, layout=layout, scaling={"kind": "linear", "factor": 1.5, "amplitude": 1.25})
    x, whole = strided(rng, n, heads, pad)
    pos = rng.integers(0, 5000, n)
    pos[0] = 0
    if n > 3:
        pos[1], pos[3] = -1, 1 << 20
    norm = weight(rng, D) if normed else None
    before = whole.clone()
    out = torch.full((n, heads * D + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, :heads * D].unflatten(1, (heads, D))
    assert bs.rotate(x, i32(pos), rope, norm=norm, eps=1e-5, out=view) is not None
    y, tol = expected(x, pos, rope, norm, 1e-5)
    got = f64(view)
    live = pos >= 0
    assert np.all(np.abs(got - y)[live] <= tol[live])
    assert np.all(got[~live] == 9.0) and torch.all(out[:, heads * D:] == 9.0) and same(whole, before)
    if not normed:  # channels past the turned ones come through as they are
        assert same(view[i32(live).bool()][..., rot:], x[i32(live).bool()][..., rot:])
    # in place, and an output made by the call
    made = bs.rotate(x, i32(np.abs(pos)), rope, norm=norm, eps=1e-5)
    assert made.is_contiguous() and made.shape == x.shape and made.dtype == torch.bfloat16
    assert bs.rotate(x, i32(np.abs(pos)), rope, norm=norm, eps=1e-5, out=x).data_ptr() == x.data_ptr()
    assert same(made, x) and same(whole[:, heads * D:], before[:, heads * D:])


@pytest.mark.parametrize("scaling", [None, {"kind": "ntk", "factor": 8.0}, {"kind": "index", "factor": 4.0, "original": 32768.0},
                                     {"kind": "rotations", "factor": 8.0, "original": 8192.0}])
def test_rotate_far_positions(scaling):
    rng = np.random.default_rng(5)
    rope = bs.rope(1e6, 128, scaling=scaling)
    x = bf16(rng, 6, 2, D)
    pos = np.array([1, 32767, 131071, (1 << 24) + 1, (1 << 30) + 7, 2 ** 31 - 1])
    y, tol = expected(x, pos, rope)
    assert np.all(np.abs(f64(bs.rotate(x, i32(pos), rope)) - y) <= tol)
    # the frequencies themselves, where fp64 angles are good to 2^-30
    f, amp = R.frequencies(1e6, 128, scaling)
    y, size = R.rotate(f64(x[:3]), pos[:3, None] * f, 128, "half", amp)
    assert np.all(np.abs(f64(bs.rotate(x[:3], i32(pos[:3]), rope)) - y) <= 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * 33 * U * size)


def test_rotate_values_that_are_not_finite_spoil_their_heads_alone():
    rng = np.random.default_rng(6)
    rope = bs.rope(1e4, 64)
    x = bf16(rng, 8, 5, D)
    clean = bs.rotate(x, i32(np.arange(8)), rope)
    bad = x.clone()
    bad[2, 1, 3], bad[4, 4, 100], bad[7, 0, 40] = float("nan"), float("inf"), -float("inf")
    got = bs.rotate(bad, i32(np.arange(8)), rope)
    changed = (got.view(torch.int16) != clean.view(torch.int16)).nonzero().tolist()
    assert sorted(changed) == [[2, 1, 3], [2, 1, 35], [4, 4, 100], [7, 0, 8], [7, 0, 40]]
    assert torch.isnan(got[2, 1, 3]) and torch.isnan(got[2, 1, 35]) and got[4, 4, 100] == float("inf")
    norm = weight(rng, D)
    clean, got = (bs.rotate(v, i32(np.arange(8)), rope, norm=norm) for v in (x, bad))
    heads = sorted({tuple(e[:2]) for e in (got.view(torch.int16) != clean.view(torch.int16)).nonzero().tolist()})
    assert heads == [(2, 1), (4, 4), (7, 0)]


def test_rotate_a_head_of_zeros_stays_zero_and_large_values_stay_finite():
    rope = bs.rope(1e4, 128)
    x = torch.zeros((2, 1, D), dtype=torch.bfloat16, device="cuda")
    x[1] = 3e15  # squares of 1e31, their sum within fp32
    norm = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    got = bs.rotate(x, i32([3, 0]), rope, norm=norm, eps=1e-6)
    assert torch.all(got[0] == 0) and torch.all(got[1] == 1)


def test_rotate_rows_past_32_bit_offsets():
    rng = np.random.default_rng(8)
    rope = bs.rope(1e4, 128)
    ld = (1 << 31) + 64
    buf = torch.empty(2 * ld + 2 * D, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 2, D), (ld, D, 1))
    x.copy_(bf16(rng, 3, 2, D))
    y, tol = expected(x, np.array([5, 6, 7]), rope)
    assert np.all(np.abs(f64(bs.rotate(x, i32([5, 6, 7]), rope)) - y) <= tol)
    bs.rotate(x, i32([5, 6, 7]), rope, out=x)
    assert np.all(np.abs(f64(x) - y) <= tol)


@pytest.mark.parametrize("n,heads", [(20000, 3), (3, 3000), (4097, 33)])
def test_rotate_many_rows_and_many_heads(n, heads):
    """Every head of every row is turned once: against torch in 64 bits on the device."""
    rope = bs.rope(1e6, 128)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((n, heads, D), generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    f = torch.tensor(R.frequencies(1e6, 128)[0], device="cuda")
    a = (pos.double()[:, None] * f)[:, None]
    lo, hi = x[..., :64].double(), x[..., 64:].double()
    y = torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)
    size = torch.hypot(lo, hi).repeat(1, 1, 2)
    got = bs.rotate(x, pos, rope).double()
    assert torch.all((got - y).abs() <= 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * 33 * U * size)


def test_rotate_without_rows():
    rope = bs.rope(1e4, 64)
    x = torch.empty((0, 3, D), dtype=torch.bfloat16, device="cuda")
    assert bs.rotate(x, i32([]), rope).shape == (0, 3, D)


# ---------------------------------------------------------------------------
# append_rotated_kv
# ---------------------------------------------------------------------------
class Write:
    """New rows of a batch and its tables."""

    def __init__(self, rng, prev, seq, Hkv, Hq, P, pad=0, extra=0):
        self.prev, self.seq, self.Hkv, self.Hq, self.P = prev, seq, Hkv, Hq, P
        B = len(seq)
        self.B, self.cap = B, max(1, -(-max(max(seq), 1) // P)) + 1
        self.n = sum(seq) - sum(prev)
        rows = self.n + extra  # a padded batch's rows at the end
        self.n_slots = B * Hkv * self.cap + 3
        t = -np.ones((B, Hkv, self.cap), int)
        free = iter(rng.permutation(self.n_slots))
        for b in range(B):
            for h in range(Hkv):
                for j in range(-(-seq[b] // P)):
                    t[b, h, j] = next(free)
        self.table_np, self.table = t, i32(t)
        self.q = strided(rng, rows, Hq, pad)[0] if Hq else None
        self.K, self.V = strided(rng, rows, Hkv, pad)[0], strided(rng, rows, Hkv, pad)[0]
        at = np.concatenate([np.arange(p, s) for p, s in zip(prev, seq)] + [np.zeros(0, int)])
        self.pos = np.concatenate([at, -np.ones(extra, int)]).astype(int)
        owner = np.repeat(np.arange(B), np.array(seq) - np.array(prev))
        m = -np.ones((rows, Hkv), np.int64)
        m[:self.n] = t[owner, :, at // P] * P + (at % P)[:, None]
        self.slot_map = torch.from_numpy(m).cuda()
        self.seq_t, self.prev_t = i32(seq), i32(prev)
        self.kw, self.qw = weight(rng, D), weight(rng, D)

    def turned(self, rope, x, w, eps=1e-6):
        """Rows by the operator alone, padding rows as they were."""
        return bs.rotate(x, i32(self.pos), rope, norm=w, eps=eps, out=x.clone())


@pytest.mark.parametrize("layout,rot,normed", [("half", 128, True), ("interleaved", 64, False), ("half", 32, True)])
@pytest.mark.parametrize("lens,Hkv,Hq,P,pad,extra", [
    (([0], [1]), 1, 0, 16, 0, 0), (([31, 0, 7], [32, 5, 7]), 2, 6, 32, 128, 3), (([0, 100], [300, 101]), 8, 40, 64, 0, 0),
    (([5] * 70, [6] * 70), 3, 3, 16, 64, 9)])
def test_append_is_rotate_and_append_kv(layout, rot, normed, lens, Hkv, Hq, P, pad, extra):
    rng = np.random.default_rng(Hkv * 10 + P)
    w = Write(rng, *lens, Hkv, Hq, P, pad, extra)
    rope = bs.rope(1e4, rot, layout=layout)
    kw, qw = (w.kw, w.qw if Hq else None) if normed else (None, None)
    pools = [bf16(rng, w.n_slots, P, D) for _ in "KV"]
    one, two = [p.clone() for p in pools], [p.clone() for p in pools]
    st = word()
    q_out = None if not Hq else torch.full((w.n + extra, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    out = bs.append_rotated_kv(w.K, w.V, i32(w.pos), rope, w.slot_map, Hkv, P, *one, k_norm=kw, q=w.q, q_norm=qw, q_out=q_out,
                               status=st)
    bs.append_kv(w.turned(rope, w.K, kw), w.V.contiguous(), w.slot_map, Hkv, P, *two)
    assert same(one[0], two[0]) and same(one[1], two[1]) and int(st) == 0
    if Hq:
        assert out is q_out and same(out[:w.n], w.turned(rope, w.q, qw)[:w.n]) and torch.all(out[w.n:] == 3.0)
        y, tol = expected(w.q[:w.n], w.pos[:w.n], rope, qw, 1e-6)
        assert np.all(np.abs(f64(out[:w.n]) - y) <= tol)
        again = bs.append_rotated_kv(w.K, w.V, i32(w.pos), rope, w.slot_map, Hkv, P, *one, k_norm=kw, q=w.q, q_norm=qw, q_out=w.q)
        assert same(again[:w.n], out[:w.n])
    else:
        assert out is None


def test_append_skips_and_reports_slots():
    rng = np.random.default_rng(1)
    w = Write(rng, [0], [9], 2, 2, 16)
    rope = bs.rope(1e4, 128)
    m = w.slot_map.clone()
    m[3, 0], m[4, 1], m[6, 0] = -1, -(1 << 60), w.n_slots * 16
    pools = [torch.full((w.n_slots, 16, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "KV"]
    st = word()
    pos = i32([0, 1, -1, 3, 4, 5, 6, 7, 8])
    q = bs.append_rotated_kv(w.K, w.V, pos, rope, m, 2, 16, *pools, q=w.q, status=st, q_out=torch.full_like(w.q, 2.0))
    assert int(st) == 1
    want = bs.rotate(w.K, pos, rope)
    for i in range(9):
        for h in range(2):
            skipped = i == 2 or (i, h) in ((3, 0), (4, 1), (6, 0))
            row = int(w.slot_map[i, h])
            for pool, x in zip(pools, (want, w.V)):
                r = pool.view(-1, D)[row]
                assert torch.all(r == 5.0) if skipped else same(r, x[i, h])
    assert torch.all(q[2] == 2.0) and same(q[3], bs.rotate(w.q, pos, rope)[3])  # a query does not need a slot


def test_append_pool_rows_past_32_bit_offsets():
    rng = np.random.default_rng(2)
    w = Write(rng, [0], [4], 1, 1, 64)
    slots = (1 << 31) // (64 * D) + 70  # the last rows' elements lie past 2^31
    pools = [torch.empty((slots, 64, D), dtype=torch.bfloat16, device="cuda") for _ in "KV"]
    rows = torch.tensor([[slots * 64 - 1], [0], [(1 << 31) // D], [(1 << 31) // D + 4097]], device="cuda")
    rope = bs.rope(1e4, 128)
    bs.append_rotated_kv(w.K, w.V, i32(w.pos), rope, rows, 1, 64, *pools)
    for pool, x in zip(pools, (w.turned(rope, w.K, None), w.V)):
        assert same(pool.view(-1, D)[rows[:, 0]], x[:, 0])


# ---------------------------------------------------------------------------
# append_rotated_kv8
# ---------------------------------------------------------------------------
def pools8(rng, w, fmt):
    """Pools with finite codes, scales powers of two."""
    codes = rng.integers(0, 0x78, (w.n_slots, w.P, D)).astype(np.uint8) | (rng.integers(0, 2, (w.n_slots, w.P, D)) << 7).astype(np.uint8)
    scale = 2.0 ** rng.integers(-9, 2, w.n_slots)
    return [torch.from_numpy(codes).cuda().view(DT[fmt]), torch.from_numpy(scale.astype(np.float32)).cuda()]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("layout,rot,normed", [("half", 128, True), ("interleaved", 48, False), ("half", 64, False)])
@pytest.mark.parametrize("lens,Hkv,Hq,P,pad,extra", [
    (([0], [1]), 1, 1, 16, 0, 0), (([31, 0, 7, 3], [32, 5, 7, 90]), 3, 9, 32, 128, 3), (([0, 100], [300, 101]), 8, 40, 64, 0, 0),
    (([5] * 70, [6] * 70), 2, 0, 16, 64, 9), (([0, 0, 17], [200, 1, 400]), 5, 5, 32, 0, 0)])
def test_append8_is_rotate_and_append_kv8(fmt, layout, rot, normed, lens, Hkv, Hq, P, pad, extra):
    rng = np.random.default_rng(Hkv * 10 + P)
    w = Write(rng, *lens, Hkv, Hq, P, pad, extra)
    rope = bs.rope(1e4, rot, layout=layout)
    kw, qw = (w.kw, w.qw if Hq else None) if normed else (None, None)
    K, V = pools8(rng, w, fmt), pools8(rng, w, fmt)
    one = [t.clone() for t in (K[0], V[0], K[1], V[1])]
    two = [t.clone() for t in one]
    st = [word(), word()]
    q_out = None if not Hq else torch.full((w.n + extra, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    out = bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, w.B, Hkv, P, *one, prev_len=w.prev_t, k_norm=kw, q=w.q,
                                q_norm=qw, q_out=q_out, status=st[0])
    k = w.turned(rope, w.K, kw)
    bs.append_kv8(k, w.V.contiguous(), w.table, w.seq_t, w.B, Hkv, P, *two, prev_len=w.prev_t, status=st[1])
    for a, b in zip(one, two):
        assert same(a, b)
    assert int(st[0]) == int(st[1]) == 0
    # and the oracle's codes of those rows
    for x, pool, scale, start in ((k, one[0], one[2], K), (w.V, one[1], one[3], V)):
        codes, s = C8.append8(f64(x[:w.n]), lens[0], lens[1], w.table_np, start[0].view(torch.uint8).cpu().numpy(),
                              start[1].double().cpu().numpy(), fmt, P)[:2]
        assert np.array_equal(pool.view(torch.uint8).cpu().numpy(), codes) and np.array_equal(scale.double().cpu().numpy(), s)
    if Hq:
        assert same(out[:w.n], w.turned(rope, w.q, qw)[:w.n]) and torch.all(out[w.n:] == 3.0)
    # positions given: the same places, and others
    three = [t.clone() for t in (K[0], V[0], K[1], V[1])]
    bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, w.B, Hkv, P, *three, prev_len=w.prev_t, k_norm=kw, positions=i32(w.pos))
    for a, b in zip(three, two):
        assert same(a, b)
    w.pos = np.where(w.pos >= 0, w.pos * 3 + 1000, -1)
    four = [t.clone() for t in (K[0], V[0], K[1], V[1])]
    five = [t.clone() for t in four]
    bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, w.B, Hkv, P, *four, prev_len=w.prev_t, k_norm=kw, positions=i32(w.pos))
    bs.append_kv8(w.turned(rope, w.K, kw), w.V.contiguous(), w.table, w.seq_t, w.B, Hkv, P, *five, prev_len=w.prev_t)
    for a, b in zip(four, five):
        assert same(a, b)


@pytest.mark.parametrize("P", [16, 32, 64])
def test_append8_token_by_token_is_append8_at_once_where_scales_agree(P):
    """A sequence written one token a call: the same q, and the codes of append_kv8's own steps."""
    rng = np.random.default_rng(P)
    w = Write(rng, [0, 0], [2 * P + 3, 5], 2, 2, P)
    rope = bs.rope(1e4, 128)
    K, V = pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    one = [t.clone() for t in (K[0], V[0], K[1], V[1])]
    two = [t.clone() for t in one]
    k = w.turned(rope, w.K, w.kw)
    first = {0: 0, 1: 2 * P + 3}
    for t in range(2 * P + 3):
        live = [b for b in range(2) if t < w.seq[b]]
        rows = torch.tensor([first[b] + t for b in live], device="cuda")
        seq, prev = i32([min(t + 1, n) for n in w.seq]), i32([min(t, n) for n in w.seq])
        q = bs.append_rotated_kv8(w.K[rows], w.V[rows], rope, w.table, seq, 2, 2, P, *one, prev_len=prev, k_norm=w.kw, q=w.q[rows])
        bs.append_kv8(k[rows], w.V[rows], w.table, seq, 2, 2, P, *two, prev_len=prev)
        assert same(q, bs.rotate(w.q[rows], i32([t] * len(live)), rope))
    for a, b in zip(one, two):
        assert same(a, b)


def check_write8(rng, w, fmt, rope, **kw):
    """append_rotated_kv8 against rotate and append_kv8, bit for bit."""
    K, V = pools8(rng, w, fmt), pools8(rng, w, fmt)
    one = [K[0], V[0], K[1], V[1]]
    two = [t.clone() for t in one]
    st = word()
    q = bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, w.B, w.Hkv, w.P, *one, prev_len=w.prev_t, k_norm=w.kw, q=w.q,
                              q_norm=w.qw if w.Hq else None, status=st, **kw)
    bs.append_kv8(w.turned(rope, w.K, w.kw), w.V.contiguous(), w.table, w.seq_t, w.B, w.Hkv, w.P, *two, prev_len=w.prev_t)
    for a, b in zip(one, two):
        assert same(a, b)
    assert int(st) == 0 and (q is None or same(q, w.turned(rope, w.q, w.qw)))


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("new", [1, 3, 4, 5, 15, 16, 17, 31, 40])
def test_append8_around_the_number_of_tokens_that_chooses_the_kernel(P, new):
    rng = np.random.default_rng(P + new)
    prev = [0, P - 1, 2 * P + 3, 7]
    check_write8(rng, Write(rng, prev, [p + new for p in prev], 3, 5, P), "e4m3", bs.rope(1e4, 96))


@pytest.mark.parametrize("P,Hkv,Hq,seq", [
    (16, 2, 1, [30011, 9, 20000]), (32, 1, 0, [70000]), (64, 3, 17, [9000, 1, 63, 64, 65]), (16, 40, 40, [700, 100]),
    (64, 1, 33, [40000, 3]), (32, 11, 2, [1000] * 3)])
def test_append8_prompts_over_the_whole_grid(P, Hkv, Hq, seq):
    rng = np.random.default_rng(P + Hkv)
    check_write8(rng, Write(rng, [0] * len(seq), seq, Hkv, Hq, P), "e5m2", bs.rope(1e6, 128))


@pytest.mark.parametrize("B,P", [(1500, 64), (4096, 32)])
def test_append8_prompts_of_many_sequences(B, P):
    """More shared memory than needs no request: the prefixes of a large batch beside a block's cosines."""
    rng = np.random.default_rng(B)
    seq = rng.integers(0, 40, B)
    prev = np.minimum(seq, rng.integers(0, 3, B))
    w = Write(rng, prev.tolist(), seq.tolist(), 1, 1, P)
    assert w.n > 16 * B
    check_write8(rng, w, "e4m3", bs.rope(1e4, 128, layout="interleaved"))


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("prev,seq", [([3, 0], [60, 20]), ([3, 0, 50], [9, 20, 51])])
def test_append8_values_that_are_not_finite(P, prev, seq):
    rng = np.random.default_rng(4 + P)
    w = Write(rng, prev, seq, 3, 0, P)
    rope = bs.rope(1e4, 64)
    last = w.n - 1
    w.K[2, 1, 7], w.K[20, 0, 100], w.K[last, 2, 33] = float("inf"), -float("inf"), float("nan")
    w.V[1, 0, 0], w.V[last, 1, 127] = float("inf"), float("nan")
    K, V = pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    for kw in (None, w.kw):
        one = [t.clone() for t in (K[0], V[0], K[1], V[1])]
        two = [t.clone() for t in one]
        bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, w.B, 3, P, *one, prev_len=w.prev_t, k_norm=kw)
        bs.append_kv8(w.turned(rope, w.K, kw), w.V, w.table, w.seq_t, w.B, 3, P, *two, prev_len=w.prev_t)
        for a, b in zip(one, two):
            assert same(a, b)


def test_writes_without_rows():
    rng = np.random.default_rng(3)
    w = Write(rng, [5], [5], 2, 4, 16)
    rope = bs.rope(1e4, 64)
    pool, K, V = bf16(rng, w.n_slots, 16, D), pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    before = [pool.clone(), K[0].clone(), V[1].clone()]
    q = bs.append_rotated_kv(w.K, w.V, i32([]), rope, w.slot_map, 2, 16, pool, pool, q=w.q)
    q8 = bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, 1, 2, 16, K[0], V[0], K[1], V[1], prev_len=w.prev_t, q=w.q)
    assert q.shape == q8.shape == (0, 4, D)
    assert same(before[0], pool) and same(before[1], K[0]) and same(before[2], V[1])


def test_append8_zero_rows_and_no_eps():
    rng = np.random.default_rng(14)
    w = Write(rng, [0], [20], 2, 0, 32)
    rope = bs.rope(1e4, 128)
    w.K[3] = 0
    K, V = pools8(rng, w, "e5m2"), pools8(rng, w, "e5m2")
    one = [t.clone() for t in (K[0], V[0], K[1], V[1])]
    two = [t.clone() for t in one]
    bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, 1, 2, 32, *one, k_norm=w.kw, eps=0.0)
    bs.append_kv8(w.turned(rope, w.K, w.kw, eps=0.0), w.V, w.table, w.seq_t, 1, 2, 32, *two)
    for a, b in zip(one, two):
        assert same(a, b)


def test_append8_bad_blocks_are_skipped_and_reported():
    rng = np.random.default_rng(5)
    w = Write(rng, [0, 0], [50, 40], 2, 2, 32)
    rope = bs.rope(1e4, 128)
    t = w.table.clone()
    t[0, 1, 1], t[1, 0, 0] = w.n_slots, -1
    K, V = pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    one = [x.clone() for x in (K[0], V[0], K[1], V[1])]
    two = [x.clone() for x in one]
    st = [word(), word()]
    q = bs.append_rotated_kv8(w.K, w.V, rope, t, w.seq_t, 2, 2, 32, *one, q=w.q, status=st[0])
    bs.append_kv8(w.turned(rope, w.K, None), w.V, t, w.seq_t, 2, 2, 32, *two, status=st[1])
    for a, b in zip(one, two):
        assert same(a, b)
    assert int(st[0]) == int(st[1]) == 1 and same(q, w.turned(rope, w.q, None))
    # rows that end early: the blocks before are written, the others not, and the queries of the rows there are
    st = word()
    q_out = torch.full((60, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    one, two = ([x.clone() for x in (K[0], V[0], K[1], V[1])] for _ in range(2))
    bs.append_rotated_kv8(w.K[:60], w.V[:60], rope, w.table, w.seq_t, 2, 2, 32, *one, q=w.q[:60], q_out=q_out, status=st)
    bs.append_kv8(w.turned(rope, w.K, None)[:60], w.V[:60], w.table, w.seq_t, 2, 2, 32, *two)
    for a, b in zip(one, two):
        assert same(a, b)
    assert int(st) == 1 and same(q_out, w.turned(rope, w.q, None)[:60])
    # a negative position counts as 0
    st = word()
    pos = w.pos.copy()
    pos[7] = -5
    q = bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, 2, 2, 32, *one, q=w.q, positions=i32(pos), status=st)
    assert int(st) == 1 and same(q, bs.rotate(w.q, i32(np.maximum(pos, 0)), rope))
    # lengths that do not fit, and no rows at all
    for prev, seq, n, want in ((None, [-1, 40], 40, 1), ([9, 9], [5, 9], 0, 1), (None, [9999, 40], 0, 5), ([5, 5], [5, 5], 0, 0)):
        st = word()
        bs.append_rotated_kv8(w.K[:n], w.V[:n], rope, w.table, i32(seq), 2, 2, 32, *one, prev_len=None if prev is None else i32(prev),
                              status=st)
        assert int(st) == want


def test_append8_of_the_largest_batch():
    rng = np.random.default_rng(6)
    seq = rng.integers(0, 4, 4096)
    prev = np.minimum(seq, rng.integers(0, 3, 4096))
    w = Write(rng, prev.tolist(), seq.tolist(), 1, 2, 16, extra=5)
    rope = bs.rope(1e4, 128)
    K, V = pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    one = [t.clone() for t in (K[0], V[0], K[1], V[1])]
    two = [t.clone() for t in one]
    q_out = torch.full_like(w.q, 3.0)
    bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, 4096, 1, 16, *one, prev_len=w.prev_t, q=w.q, q_out=q_out)
    bs.append_kv8(w.turned(rope, w.K, None), w.V, w.table, w.seq_t, 4096, 1, 16, *two, prev_len=w.prev_t)
    for a, b in zip(one, two):
        assert same(a, b)
    assert same(q_out[:w.n], w.turned(rope, w.q, None)[:w.n]) and torch.all(q_out[w.n:] == 3.0)


def at_16(t):
    """The same values at an address that is a multiple of 16, but not of 32."""
    buf = torch.empty(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
    start = 16 - buf.data_ptr() % 32
    view = buf[start + (32 if start < 0 else 0):][: t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    assert view.data_ptr() % 32 == 16
    return view.copy_(t)


@pytest.mark.parametrize("new", [1, 40])
def test_rows_and_pools_at_16_byte_boundaries(new):
    rng = np.random.default_rng(new)
    w = Write(rng, [5, 33], [5 + new, 33 + new], 3, 5, 32, pad=8)
    rope = bs.rope(1e4, 128)
    for n in ("K", "V", "q"):
        x = getattr(w, n)
        row = at_16(torch.zeros((x.shape[0], x.shape[1] * D + 8), dtype=torch.bfloat16, device="cuda"))
        view = row[:, :x.shape[1] * D].unflatten(1, (x.shape[1], D))
        setattr(w, n, view.copy_(x))
    kw, qw = at_16(w.kw), at_16(w.qw)
    want_k, want_q = w.turned(rope, w.K, w.kw), w.turned(rope, w.q, w.qw)
    one = [at_16(bf16(rng, w.n_slots, 32, D)) for _ in "KV"]
    two = [t.clone() for t in one]
    q = bs.append_rotated_kv(w.K, w.V, i32(w.pos), rope, w.slot_map, 3, 32, *one, k_norm=kw, q=w.q, q_norm=qw)
    bs.append_kv(want_k, w.V, w.slot_map, 3, 32, *two)
    assert same(one[0], two[0]) and same(one[1], two[1]) and same(q, want_q)
    K, V = pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    one = [at_16(K[0].view(torch.uint8)).view(DT["e4m3"]), at_16(V[0].view(torch.uint8)).view(DT["e4m3"]), K[1], V[1]]
    two = [t.clone() for t in one]
    q = bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, 2, 3, 32, *one, prev_len=w.prev_t, k_norm=kw, q=w.q, q_norm=qw)
    bs.append_kv8(want_k, w.V, w.table, w.seq_t, 2, 3, 32, *two, prev_len=w.prev_t)
    assert all(same(a, b) for a, b in zip(one, two)) and same(q, want_q)
    out = [[torch.zeros((2, 3, w.cap * 32, D), dtype=torch.bfloat16, device="cuda") for _ in "KV"] for _ in range(2)]
    for pools, o in zip((one, two), out):  # an 8-bit pool at 16 bytes is read; a bf16 one, or an output, is not
        bs.read_kv8(*pools, w.table, w.seq_t, 2, 3, 32, *o)
    assert same(out[0][0], out[1][0]) and same(out[0][1], out[1][1])
    with pytest.raises(bs.ScoutError, match="UNSUPPORTED"):
        bs.read_kv8(*one, w.table, w.seq_t, 2, 3, 32, at_16(out[0][0]), at_16(out[0][1]))
    pool = at_16(bf16(rng, w.n_slots, 32, D))
    with pytest.raises(bs.ScoutError, match="UNSUPPORTED"):
        bs.read_kv(pool, pool, w.table, w.seq_t, 2, 3, 32, *out[0])


# ---------------------------------------------------------------------------
# predict_q_rotated
# ---------------------------------------------------------------------------
def predicted(X, W, pos, rope, norm, eps):
    """(Q, tolerance) [M][heads][D]."""
    x, w = f64(X), f64(W)
    M, K = x.shape
    q, e = x @ w.T, (2 * K + 16) * U * (np.abs(x) @ np.abs(w).T)
    q, e = q.reshape(M, -1, D), e.reshape(M, -1, D)
    ang = R.angles(np.maximum(pos, 0), turns_of(rope))
    nw = None if norm is None else f64(norm)
    y, size = R.rotate(q, ang, rope.rot_dim, rope.layout, rope.amplitude, nw, eps)
    if norm is not None:
        length = np.sqrt((q * q).sum(-1, keepdims=True))
        factor = 1 / np.sqrt((q * q).mean(-1, keepdims=True) + eps)
        e = factor * np.abs(nw) * (e + np.abs(q) * np.sqrt((e * e).sum(-1, keepdims=True)) / length)
    a, b = R.pairs(e, rope.rot_dim, rope.layout)  # both errors of a pair reach each of its channels
    both = e.copy()
    for view in R.pairs(both, rope.rot_dim, rope.layout):
        view[...] = rope.amplitude * np.hypot(a, b)
    e = both * 1.01 + 32 * U * size  # second-order terms: both are small
    return y, 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * e


@pytest.mark.parametrize("M,heads,K,rot,layout,normed,max_ctas", [
    (1, 1, 64, 128, "half", True, None), (1, 8, 4096, 128, "half", True, None), (8, 32, 4096, 128, "half", True, None),
    (7, 3, 192, 64, "interleaved", False, None), (17, 5, 1088, 16, "half", True, 1), (40, 40, 5120, 128, "half", True, 80),
    (100, 2, 640, 96, "interleaved", True, None), (256, 4, 512, 128, "half", False, None), (255, 19, 320, 128, "interleaved", True, 7),
    (33, 152, 128, 48, "half", True, None)])
def test_predict(M, heads, K, rot, layout, normed, max_ctas):
    rng = np.random.default_rng(M + K)
    rope = bs.rope(1e6, rot, layout=layout, scaling={"kind": "index", "factor": 4.0, "original": 32768.0})
    X, W = bf16(rng, M, K), (bf16(rng, heads * D, K, gain=False).float() * 0.02).to(torch.bfloat16)
    pos = rng.integers(0, 1 << 18, M)
    if M > 2:
        pos[1] = -1
    norm = weight(rng, D) if normed else None
    Q = torch.full((M, heads * D), 3.0, dtype=torch.bfloat16, device="cuda")
    st = word()
    got = bs.predict_q_rotated(X, W, i32(pos), rope, norm=norm, eps=1e-6, Q=Q, status=st, max_ctas=max_ctas)
    assert got is Q and int(st) == 0
    y, tol = predicted(X, W, pos, rope, norm, 1e-6)
    out, live = f64(Q).reshape(M, heads, D), pos >= 0
    assert np.all(np.abs(out - y)[live] <= tol[live]) and np.all(out[~live] == 3.0)
    assert same(bs.predict_q_rotated(X, W, i32(pos), rope, norm=norm, Q=Q.clone(), max_ctas=max_ctas), Q)


def test_predict_in_a_graph_and_after_another_kernel():
    rng = np.random.default_rng(3)
    rope = bs.rope(1e6, 128)
    X, W, norm = bf16(rng, 8, 512), bf16(rng, 512, 512), weight(rng, D)
    pos = i32(np.arange(8))
    Q = torch.empty((8, 512), dtype=torch.bfloat16, device="cuda")
    bs.predict_q_rotated(X, W, pos, rope, norm=norm, Q=Q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bs.predict_q_rotated(X, W, pos, rope, norm=norm, Q=Q)
    X.copy_(bf16(rng, 8, 512))
    pos.add_(1000)
    g.replay()
    y, tol = predicted(X, W, np.arange(8) + 1000, rope, norm, 1e-6)
    assert np.all(np.abs(f64(Q).reshape(8, 4, D) - y) <= tol)


def test_predict_started_early_waits_for_its_input_and_positions():
    """A programmatic dependent of the kernel that writes X and the positions (its own predecessor)."""
    import ctypes

    rng = np.random.default_rng(4)
    rope = bs.rope(1e6, 128)
    W1, W2, x = bf16(rng, 2048, 2048), bf16(rng, 512, 2048), bf16(rng, 8, 2048)
    X = torch.zeros((8, 2048), dtype=torch.bfloat16, device="cuda")
    Q = torch.empty((8, 512), dtype=torch.bfloat16, device="cuda")
    pos = i32(np.arange(8))
    want = bs.predict_q_rotated(bs.predict_q(x, W1), W2, pos, rope)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = bs.RopeArgs(rope.turns.data_ptr(), 128, 0, 1.0)
    L = bs.lib()
    for _ in range(20):
        X.zero_()
        torch.cuda.synchronize()
        assert L.scout_predict_q(x.data_ptr(), W1.data_ptr(), X.data_ptr(), 8, 2048, 2048, None, None, st.cuda_stream) == 0
        assert L.scout_predict_q_rotated(X.data_ptr(), W2.data_ptr(), Q.data_ptr(), 8, 512, 2048, pos.data_ptr(), ctypes.byref(args),
                                         None, 1e-6, None, bs._launch(0, pdl=True), st.cuda_stream) == 0
        torch.cuda.synchronize()
        assert same(Q, want)


# ---------------------------------------------------------------------------
# read_kv
# ---------------------------------------------------------------------------
def read_case(rng, seq, Hkv, P, fmt, T=None, order="blocks", host=False, resident=1.0):
    B, cap = len(seq), max(1, -(-max(seq) // P)) + 1
    n_slots = B * Hkv * cap + 2
    table = rng.permutation(n_slots)[:B * Hkv * cap].reshape(B, Hkv, cap).copy()
    table[rng.random(table.shape) > resident] = -1
    T = cap * P if T is None else T
    shape = (B, Hkv, T, D) if order == "blocks" else (B, T, Hkv, D)
    out = []
    for _ in "KV":
        o = torch.full(shape, 9.0, dtype=torch.bfloat16)
        o = o.pin_memory() if host else o.cuda()
        out.append(o if order == "blocks" else o.transpose(1, 2))
    if fmt == "bf16":
        pools, scales = [bf16(rng, n_slots, P, D) for _ in "KV"], []
        values = [f64(p) for p in pools]
    else:
        pools, scales, values = [], [], []
        for _ in "KV":
            c = rng.integers(0, 0x7B, (n_slots, P, D)).astype(np.uint8)
            s = rng.uniform(0.01, 3.0, n_slots).astype(np.float32)
            s[::2] = 2.0 ** rng.integers(-20, 20, len(s[::2]))
            pools.append(torch.from_numpy(c).cuda().view(DT[fmt]))
            scales.append(torch.from_numpy(s).cuda())
            values.append(C8.decode(c, fmt) * s.astype(np.float64)[:, None, None])
    return table, pools, scales, values, out


def run_read(table, pools, scales, seq, P, out, blocks=None, **kw):
    B, Hkv, _ = table.shape
    lst = None if blocks is None else i32(np.array(blocks).reshape(-1, 2))
    if scales:
        return bs.read_kv8(*pools, *scales, i32(table), i32(seq), B, Hkv, P, *out, block_list=lst, **kw)
    return bs.read_kv(*pools, i32(table), i32(seq), B, Hkv, P, *out, block_list=lst, **kw)


def check_read(values, table, seq, P, out, blocks=None):
    torch.cuda.synchronize()
    for v, o in zip(values, out):
        shape = tuple(o.shape)
        written = R.read(np.ones(v.shape), table, seq, P, np.zeros(shape), blocks) == 1
        want, got = R.read(v, table, seq, P, np.zeros(shape), blocks), f64(o)
        assert np.all(np.abs(got - want)[written] <= 2.0 ** -8 * np.abs(want[written])) and np.all(got[~written] == 9.0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("order", ["blocks", "tokens"])
@pytest.mark.parametrize("seq,Hkv,P,host", [([1], 1, 16, False), ([0, 33, 64], 2, 32, False), ([100, 5], 8, 64, True), ([31] * 9, 3, 16, True)])
def test_read_all_blocks(fmt, order, seq, Hkv, P, host):
    rng = np.random.default_rng(P + len(seq))
    table, pools, scales, values, out = read_case(rng, seq, Hkv, P, fmt, order=order, host=host, resident=0.7)
    st = word()
    got = run_read(table, pools, scales, seq, P, out, status=st)
    assert got[0] is out[0] and got[1] is out[1]
    check_read(values, table, seq, P, out)
    assert int(st) == 0  # blocks that are not on the GPU are no fault
    if fmt != "bf16":  # powers of two: exact
        for v, o in zip(values, out):
            want = R.read(v, table, seq, P, np.full(tuple(o.shape), 9.0))
            even = R.read(np.broadcast_to((np.arange(len(v)) % 2 == 0)[:, None, None], v.shape).astype(float), table, seq, P,
                          np.zeros(tuple(o.shape))) == 1
            assert np.array_equal(f64(o)[even], want[even])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_read_a_list_of_blocks(fmt):
    rng = np.random.default_rng(2)
    seq = [70, 1, 0, 200]
    table, pools, scales, values, out = read_case(rng, seq, 2, 32, fmt)
    blocks = [(0, 0), (1, 2), (-1, -1), (3, 0), (6, 6), (6, 1), (7, 3), (-1, -1), (4, 0)]
    st = word()
    run_read(table, pools, scales, seq, 32, out, blocks, status=st)
    check_read(values, table, seq, 32, out, [b for b in blocks if b[0] >= 0])
    assert int(st) == 0
    for bad in ([(8, 0)], [(0, table.shape[2])], [(-1, 0)], [(0, -1)], [(-2, 5)]):
        st, now = word(), [o.clone() for o in out]
        run_read(table, pools, scales, seq, 32, now, [(0, 1)] + bad, status=st)
        assert int(st) == 1
        check_read(values, table, seq, 32, now, [b for b in blocks if b[0] >= 0] + [(0, 1)])
    for slot in (-1, len(pools[0])):
        st, t = word(), table.copy()
        t[0, 1, 1] = slot
        run_read(t, pools, scales, seq, 32, [o.clone() for o in out], [(1, 1), (1, 0)], status=st)
        assert int(st) == 1
    st = word()
    run_read(np.where(table == table[3, 0, 2], len(pools[0]) + 7, table), pools, scales, seq, 32, [o.clone() for o in out], status=st)
    assert int(st) == 1
    assert run_read(table, pools, scales, seq, 32, out, np.zeros((0, 2)))[0] is out[0]


def test_read_rows_that_do_not_fit_are_left_out():
    rng = np.random.default_rng(3)
    seq = [70, 40]
    table, pools, scales, values, out = read_case(rng, seq, 2, 32, "bf16", T=45)
    st = word()
    run_read(table, pools, scales, seq, 32, out, status=st)
    check_read(values, table, seq, 32, out)
    assert int(st) == 4


def test_read_slots_and_rows_past_32_bit_offsets():
    rng = np.random.default_rng(4)
    slots = (1 << 31) // (64 * D) + 9
    pools = [torch.empty((slots, 64, D), dtype=torch.bfloat16, device="cuda") for _ in "KV"]
    for p in pools:
        p[-1].copy_(bf16(rng, 64, D))
        p[3].copy_(bf16(rng, 64, D))
    out = [torch.empty((1 << 31) + 4 * 64 * D, dtype=torch.bfloat16, device="cuda").as_strided((2, 1, 128, D), (1 << 31, 0, D, 1)) for _ in "KV"]
    bs.read_kv(*pools, i32([[[slots - 1, -1]], [[3, slots - 1]]]), i32([64, 128]), 2, 1, 64, *out)
    for p, o in zip(pools, out):
        assert same(o[0, 0, :64], p[-1]) and same(o[1, 0, :64], p[3]) and same(o[1, 0, 64:], p[-1])


def test_read_needs_pinned_host_memory():
    rng = np.random.default_rng(5)
    table, pools, scales, values, out = read_case(rng, [40], 1, 32, "bf16", host=True)
    with pytest.raises(bs.ScoutError, match="UNSUPPORTED"):
        run_read(table, pools, scales, [40], 32, [o.clone() for o in out])
    with pytest.raises(bs.ScoutError, match="alike"):
        run_read(table, pools, scales, [40], 32, [out[0], out[1].cuda()])


def test_read_is_the_inverse_of_the_write():
    """What append_kv8 wrote comes back as rows that append_kv8 writes to the same codes."""
    rng = np.random.default_rng(6)
    w = Write(rng, [0, 0], [75, 20], 2, 0, 32)
    K, V = pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    one = [K[0], V[0], K[1], V[1]]
    bs.append_kv8(w.K, w.V, w.table, w.seq_t, 2, 2, 32, *one)
    k, v = (torch.zeros((2, 96, 2, D), dtype=torch.bfloat16, device="cuda") for _ in "KV")
    bs.read_kv8(*one, w.table, w.seq_t, 2, 2, 32, k.transpose(1, 2), v.transpose(1, 2))
    two = [t.clone() for t in one]
    rows = [torch.cat([x[0, :75], x[1, :20]]) for x in (k, v)]
    bs.append_kv8(*rows, w.table, w.seq_t, 2, 2, 32, *two)
    for a, b in zip(one, two):
        assert same(a, b)


# ---------------------------------------------------------------------------
# add_norm
# ---------------------------------------------------------------------------
def run_norm(rng, kind, M, N, wide, post, gate, ahead, alpha, pad, eps=1e-6, scale=1.0, bias=True):
    wt = torch.float32 if wide else torch.bfloat16
    Y = bf16(rng, M, N + pad)[:, :N]
    H = (bf16(rng, M, N + pad).to(wt) * scale)[:, :N] + (0.37 if wide else 0)
    v = {n: weight(rng, N) for n in ("w", "w_post", "w_ahead")}
    b = {n: bf16(rng, N) if kind == "layer" and bias else None for n in ("b", "b_post", "b_ahead")}
    g = None if gate == "none" else bf16(rng, N) if gate == "vector" else bf16(rng, M, N)
    kw = dict(b=b["b"], gate=g, alpha=alpha)
    if post:
        kw |= dict(w_post=v["w_post"], b_post=b["b_post"])
    if ahead:
        kw |= dict(w_ahead=v["w_ahead"], b_ahead=b["b_ahead"])
    out = bs.add_norm(kind, Y, H, v["w"], eps, **kw)
    # the same in fp64, with a bound on the fp32 errors
    opt = lambda t: None if t is None else f64(t)  # noqa: E731
    sums = 74 * U

    def normed(x, e, w, bb):
        y, z = R.norm(x, kind, f64(w), opt(bb), eps)
        dev = x - (x.mean(-1, keepdims=True) if kind == "layer" else 0.0)
        f = 1 / np.sqrt((dev * dev).mean(-1, keepdims=True) + eps)
        if kind == "layer":
            e = e + e.mean(-1, keepdims=True) + (sums + U) * np.abs(x).mean(-1, keepdims=True) + U * np.abs(dev)
        rel = f * np.sqrt((e * e).mean(-1, keepdims=True)) + (sums / 2 + 8 * U)  # of the factor
        err = np.abs(f64(w)) * (f * e + np.abs(z) * rel) * 1.01 + 3 * U * (np.abs(y) + np.abs(0.0 if bb is None else f64(bb)))
        return y, err

    p, e = f64(Y), np.zeros((M, N))
    if post:
        p, e = normed(p, e, v["w_post"], b["b_post"])
    if g is not None:
        p, e = p * f64(g), e * np.abs(f64(g)) + U * np.abs(p * f64(g))
    a = float(np.float32(alpha))
    h = f64(H) + a * p
    e = abs(a) * e + U * (np.abs(a * p) + np.abs(h))
    rounded = U if wide else 2.0 ** -8
    assert np.all(np.abs(f64(out[0]) - h) <= rounded * np.abs(h) + (1 + rounded) * e)
    for got, w, bb in [(out[1], v["w"], b["b"])] + ([(out[2], v["w_ahead"], b["b_ahead"])] if ahead else []):
        y, err = normed(h, e, w, bb)
        assert np.all(np.abs(f64(got) - y) <= 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * err)
    assert len(out) == 2 + ahead and out[0].dtype == wt and out[1].is_contiguous()
    return Y, H, v["w"], kw, out


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("M,N,wide,post,gate,ahead,alpha,pad", [
    (1, 8, False, False, "none", False, 1.0, 0), (5, 8, True, True, "rows", True, -0.7, 8), (3, 248, True, False, "vector", False, 0.5, 0),
    (9, 256, False, True, "none", True, 1.0, 16), (2, 512, False, False, "none", True, 1.0, 8), (3, 520, True, True, "none", False, 2.0, 0),
    (40, 5120, False, False, "none", True, 1.0, 0), (7, 4096, True, True, "vector", True, 0.125, 64), (2, 8192, False, True, "rows", True, 1.0, 0),
    (2, 8200, True, False, "none", True, 1.0, 0), (3, 16384, False, True, "vector", False, 1.0, 8), (2, 16392, False, True, "none", True, 1.0, 0),
    (2, 32768, True, True, "rows", True, 1.0, 0), (1000, 64, False, True, "rows", False, 1.0, 0), (257, 1000, True, False, "none", False, 1.0, 0)])
def test_add_norm(kind, M, N, wide, post, gate, ahead, alpha, pad):
    rng = np.random.default_rng(M + N)
    Y, H, w, kw, out = run_norm(rng, kind, M, N, wide, post, gate, ahead, alpha, pad)
    # the same bits in place, into given outputs, over Y, and again
    other = bs.add_norm(kind, Y, H, w, H_out=torch.empty((M, N + 24), dtype=H.dtype, device="cuda")[:, :N], **kw)
    assert all(same(a, b) for a, b in zip(out, other))
    y, h = Y.contiguous(), H.clone()
    x = bs.add_norm(kind, y, h, w, H_out=h, X=y, **kw)
    assert x[0] is h and x[1] is y and all(same(a, b) for a, b in zip(out, x))


def test_add_norm_gates_of_any_stride_and_a_stream_inside_a_wider_one():
    rng = np.random.default_rng(7)
    Y, w = bf16(rng, 6, 640), weight(rng, 640)
    H = bf16(rng, 6, 1920)[:, 640:1280]
    wide = bf16(rng, 6, 1280)
    want = bs.add_norm("rms", Y, H.contiguous(), w, gate=wide[:, 640:].contiguous())
    got = bs.add_norm("rms", Y, H, w, gate=wide[:, 640:])
    assert got[0].is_contiguous() and all(same(a, b) for a, b in zip(want, got))
    one = bs.add_norm("rms", Y, H, w, gate=wide[0, 640:].clone())
    for gate in (wide[:1, 640:].expand(6, 640), wide[:1, 640:].repeat(6, 1)):
        assert all(same(a, b) for a, b in zip(one, bs.add_norm("rms", Y, H, w, gate=gate)))
    with pytest.raises(bs.ScoutError, match="INVALID"):  # rows that overlap
        bs.add_norm("rms", Y, H[:1].expand(6, 640), w)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_add_norm_without_an_output_is_the_norms_alone(kind):
    rng = np.random.default_rng(1)
    H, w, wa = bf16(rng, 6, 640), weight(rng, 640), weight(rng, 640)
    h, x, xa = bs.add_norm(kind, None, H, w, w_ahead=wa)
    assert h is H
    zero = bs.add_norm(kind, torch.zeros_like(H), H, w, w_ahead=wa)
    assert same(zero[0], H) and same(zero[1], x) and same(zero[2], xa)
    assert same(bs.add_norm(kind, None, H, wa)[1], xa)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_add_norm_rows_of_one_value_and_of_none(kind):
    H = torch.full((3, 512), 4.0, device="cuda")
    H[1] = 0.0
    H[2, 7] = float("nan")
    one = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    x = bs.add_norm(kind, None, H, one)[1]
    assert torch.all(x[0] == (0.0 if kind == "layer" else 1.0)) and torch.all(x[1] == 0.0) and torch.all(torch.isnan(x[2]))
    e = torch.empty((0, 512), device="cuda")
    assert bs.add_norm(kind, e.bfloat16(), e, one)[1].shape == (0, 512)


def test_add_norm_a_large_mean_does_not_spoil_the_variance():
    rng = np.random.default_rng(2)
    run_norm(rng, "layer", 4, 4096, True, False, "none", True, 1.0, 0, scale=0.01)
    run_norm(rng, "layer", 4, 4096, True, False, "none", False, 1e-3, 0, scale=1e-3, bias=False)


def test_add_norm_rows_past_32_bit_offsets():
    rng = np.random.default_rng(3)
    ld = (1 << 31) + 64
    H = torch.empty(ld + 512, dtype=torch.bfloat16, device="cuda").as_strided((2, 512), (ld, 1))
    H.copy_(bf16(rng, 2, 512))
    w, Y = weight(rng, 512), bf16(rng, 2, 512)
    want = bs.add_norm("rms", Y, H.contiguous(), w)
    got = bs.add_norm("rms", Y, H, w, H_out=H)
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_add_norm_many_rows():
    g = torch.Generator(device="cuda").manual_seed(2)
    Y, H = (torch.randn((70001, 256), generator=g, device="cuda", dtype=torch.bfloat16) for _ in "YH")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    h, x = bs.add_norm("rms", Y, H, w)
    e = H.double() + Y.double()
    y = e * (e.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    assert torch.all((h.double() - e).abs() <= 2.0 ** -8 * e.abs() + 2 * U * e.abs())
    assert torch.all((x.double() - y).abs() <= (2.0 ** -8 + 64 * U) * y.abs())


# ---------------------------------------------------------------------------
# all of them
# ---------------------------------------------------------------------------
def calls(rng):
    """One call of each kind -> a list of functions that return output tensors."""
    w = Write(rng, [40, 0, 7], [41, 33, 7], 4, 8, 32)
    rope, norm = bs.rope(1e4, 128), w.qw
    kp, vp = (bf16(rng, w.n_slots, 32, D) for _ in "KV")
    K, V = pools8(rng, w, "e4m3"), pools8(rng, w, "e4m3")
    X, W = bf16(rng, 8, 256), bf16(rng, 1024, 256)
    Y, H, nw = bf16(rng, 5, 2048), bf16(rng, 5, 2048), weight(rng, 2048)
    pos = i32(w.pos)
    shape = (3, 4, w.cap * 32, D)

    def append(stream):
        a, b = kp.clone(), vp.clone()
        q = bs.append_rotated_kv(w.K, w.V, pos, rope, w.slot_map, 4, 32, a, b, k_norm=w.kw, q=w.q, stream=stream)
        return [a, b, q]

    def append8(stream):
        t = [x.clone() for x in (K[0], V[0], K[1], V[1])]
        q = bs.append_rotated_kv8(w.K, w.V, rope, w.table, w.seq_t, 3, 4, 32, *t, prev_len=w.prev_t, q=w.q, stream=stream)
        return t + [q]

    def read(stream):
        out = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in "KV"]
        return list(bs.read_kv8(K[0], V[0], K[1], V[1], w.table, w.seq_t, 3, 4, 32, *out, stream=stream))

    return [lambda s: [bs.rotate(w.q, pos, rope, norm=norm, stream=s)], append, append8, read,
            lambda s: [bs.predict_q_rotated(X, W, i32(np.arange(8)), rope, norm=norm, stream=s)],
            lambda s: list(bs.add_norm("rms", Y, H, nw, w_ahead=nw, stream=s))]


@pytest.mark.parametrize("which", range(6))
def test_calls_on_other_streams_in_graphs_and_from_threads(which):
    fn = calls(np.random.default_rng(which))[which]
    want = fn(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one = fn(None)
        two = fn(side)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(want, one)) and all(same(a, b) for a, b in zip(want, two))
    if which not in (4,):  # (its positions are copied from the host within the call)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = fn(None)
        for t in held:
            t.view(torch.uint8).fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, held))
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = fn(None)
                    torch.cuda.current_stream().synchronize()
                    if not all(same(a, b) for a, b in zip(want, got)):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_a_layer_from_its_stream_to_its_attention_and_its_host_copy():
    """Prompt, then decode steps, as a layer's program calls the operators: the stream normalised for this layer and for
    the prediction, heads turned into the cache, digests, the predicted query's selection, attention, the host copy.
    Each result against fp64 from the operands that the step before left."""
    rng = np.random.default_rng(11)
    B, Hq, Hkv, P, N, cap, k = 3, 8, 2, 32, 512, 12, 4
    G, scale, eps = Hq // Hkv, D ** -0.5, 1e-6
    rope = bs.rope(1e6, 128)
    wn, wn_next, qw, kw = weight(rng, N), weight(rng, N), weight(rng, D), weight(rng, D)
    Wqkv = (bf16(rng, (Hq + 2 * Hkv) * D, N, gain=False).float() * 0.05).to(torch.bfloat16)
    Wq_next = (bf16(rng, Hq * D, N, gain=False).float() * 0.05).to(torch.bfloat16)
    n_slots = B * Hkv * cap
    table = torch.full((B, Hkv, cap), -1, dtype=torch.int32, device="cuda")
    bits = torch.zeros((B, Hkv, 1), dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros((n_slots, P, D), dtype=torch.bfloat16, device="cuda") for _ in "KV")
    host = [torch.zeros((B, Hkv, cap, P, D), dtype=torch.bfloat16).pin_memory() for _ in "KV"]
    digest = torch.zeros((B, Hkv, cap, 2, D), dtype=torch.bfloat16, device="cuda")
    free = torch.arange(n_slots, dtype=torch.int32, device="cuda").flip(0).contiguous()
    ws_t, ws_a = bs.score_topk_workspace(B, Hkv, cap), bs.sparse_attn_workspace(B, Hq, Hkv, P)
    seqs = [[0, 0, 0], [200, 63, 1], [201, 64, 2], [202, 65, 3]]
    keys = [np.zeros((Hkv, 0, D)) for _ in range(B)]
    vals = [np.zeros((Hkv, 0, D)) for _ in range(B)]
    used = 0
    for prev, seq in zip(seqs, seqs[1:]):
        n = sum(seq) - sum(prev)
        pos = np.concatenate([np.arange(p, s) for p, s in zip(prev, seq)])
        st = word()
        seq_t, prev_t = i32(seq), i32(prev)
        slot_map = torch.zeros((n, Hkv), dtype=torch.int64, device="cuda")
        lst = torch.zeros((64, 2), dtype=torch.int32, device="cuda")
        counts = torch.zeros(3, dtype=torch.int32, device="cuda")
        bs.build_tables(seq_t, free[used:].contiguous(), n_slots, B, Hkv, P, table, bits, prev_len=prev_t, slot_map=slot_map,
                        block_list=lst, counts=counts, status=st)
        used += int(counts[2])
        Y, H = bf16(rng, n, N), bf16(rng, n, N)
        H1, X, Xa = bs.add_norm("rms", Y, H, wn, eps, w_ahead=wn_next)
        qkv = (X.float() @ Wqkv.float().T).to(torch.bfloat16).view(n, Hq + 2 * Hkv, D)
        q = bs.append_rotated_kv(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], i32(pos), rope, slot_map, Hkv, P, kp, vp, k_norm=kw,
                                 q=qkv[:, :Hq], q_norm=qw, eps=eps, status=st)
        bs.build_digest("minmax", kp, table, seq_t, B, Hkv, P, digest, block_list=lst[:int(counts[1])].contiguous(), status=st)
        bs.read_kv(kp, vp, table, seq_t, B, Hkv, P, *[h.view(B, Hkv, cap * P, D) for h in host], block_list=lst, status=st)
        last = torch.tensor(np.cumsum(np.array(seq) - np.array(prev)) - 1, device="cuda")  # each sequence's last token
        Qp = bs.predict_q_rotated(Xa[last].contiguous(), Wq_next, i32(pos)[last].contiguous(), rope, norm=qw, eps=eps, status=st)
        sel = bs.score_topk("minmax", Qp.view(B, Hq, D), digest, seq_t, bits, B, Hq, Hkv, P, cap, k, ws_t, status=st)
        O, lse = bs.sparse_attn(q[last].contiguous(), kp, vp, table, seq_t, sel["res"], sel["res_count"], B, Hq, Hkv, P, k, scale,
                                ws_a, status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        # stream and norms
        h = f64(H) + f64(Y)
        for got, w in ((X, wn), (Xa, wn_next)):
            y = R.norm(h, "rms", f64(w), None, eps)[0]
            assert np.all(np.abs(f64(got) - y) <= (2.0 ** -8 + 80 * U) * np.abs(y) + 8 * U * np.abs(f64(w)))
        # heads
        yq, tq = expected(qkv[:, :Hq], pos, rope, qw, eps)
        yk, tk = expected(qkv[:, Hq:Hq + Hkv], pos, rope, kw, eps)
        assert np.all(np.abs(f64(q) - yq) <= tq)
        yp, tp = predicted(Xa[last], Wq_next, pos[last.cpu().numpy()], rope, qw, eps)
        assert np.all(np.abs(f64(Qp).reshape(B, Hq, D) - yp) <= tp)
        # the cache, by way of its host copy
        row = 0
        for b in range(B):
            new = seq[b] - prev[b]
            for store, x, tol in ((keys, yk, tk), (vals, f64(qkv[:, Hq + Hkv:]), None)):
                got = f64(host[0] if store is keys else host[1])[b].reshape(Hkv, cap * P, D)
                want = x[row:row + new].transpose(1, 0, 2)
                diff = np.abs(got[:, prev[b]:seq[b]] - want)
                assert np.all(diff <= (0.0 if tol is None else tol[row:row + new].transpose(1, 0, 2)))
                assert np.array_equal(got[:, :prev[b]], store[b]) and not got[:, seq[b]:].any()
                store[b] = got[:, :seq[b]].copy()
            row += new
        # selection by the digests of those keys, attention over it
        for b in range(B):
            for hk in range(Hkv):
                nb = -(-seq[b] // P)
                lo = np.array([keys[b][hk, j * P:(j + 1) * P].min(0) for j in range(nb)])
                hi = np.array([keys[b][hk, j * P:(j + 1) * P].max(0) for j in range(nb)])
                qp = f64(Qp).reshape(B, Hq, D)[b, hk * G:(hk + 1) * G]
                score = np.maximum(qp[:, None] * lo, qp[:, None] * hi).sum(-1).max(0)
                chosen = sel["topk"][b, hk].tolist()[:min(k, nb)]
                left = [j for j in range(nb) if j not in chosen]
                assert int(sel["topk_count"][b, hk]) == min(k, nb)
                if left:
                    assert score[left].max() <= score[chosen].min() + 1e-4 * np.abs(score).max()
                t = np.concatenate([np.arange(j * P, min((j + 1) * P, seq[b])) for j in sel["res"][b, hk].tolist()[:int(sel["res_count"][b, hk])]])
                s = f64(q)[last[b], hk * G:(hk + 1) * G] @ keys[b][hk, t].T * scale
                e = np.exp(s - s.max(1, keepdims=True))
                want = e @ vals[b][hk, t] / e.sum(1, keepdims=True)
                got = f64(O)[b, hk * G:(hk + 1) * G]
                assert np.all(np.abs(got - want) <= 2e-3 + 1e-2 * np.abs(want))
    # the host copy is what the CPU side reads: every block on the host against every block on the GPU
    seq = seqs[-1]
    every = torch.full((B, Hkv, cap), -1, dtype=torch.int32)
    cnt = torch.zeros((B, Hkv), dtype=torch.int32)
    for b in range(B):
        nb = -(-seq[b] // P)
        every[b, :, :nb] = torch.arange(nb, dtype=torch.int32)
        cnt[b] = nb
    ql = q[last].contiguous()
    Og, _ = bs.sparse_attn(ql, kp, vp, table, i32(seq), every.cuda(), cnt.cuda(), B, Hq, Hkv, P, cap, scale, ws_a)
    Oc, _ = bs.cpu_attend(ql.cpu(), host[0], host[1], torch.tensor(seq, dtype=torch.int32), every, cnt, B, Hq, Hkv, P, cap, scale)
    assert np.all(np.abs(f64(Og) - np.asarray(Oc)) <= 2e-3 + 1e-2 * np.abs(f64(Og)))


def test_a_step_captured_once_and_replayed_as_sequences_grow():
    """One graph of a layer's row operators over an 8-bit cache, replayed while lengths, rows and residual stream change."""
    rng = np.random.default_rng(21)
    B, Hq, Hkv, P, N, cap = 4, 8, 2, 16, 256, 6
    rope, kw, qw, wn = bs.rope(1e4, 96, layout="interleaved"), weight(rng, D), weight(rng, D), weight(rng, N)
    Wqkv, Wp = bf16(rng, (Hq + 2 * Hkv) * D, N, gain=False), bf16(rng, Hq * D, N, gain=False)
    table = i32(rng.permutation(B * Hkv * cap).reshape(B, Hkv, cap))
    start = np.array([30, 0, 15, 7])
    st = {"prev": i32(start - (start > 0)), "seq": i32(start), "status": word()}
    Y, H = bf16(rng, B, N), bf16(rng, B, N)
    H1, X, Xa = torch.empty_like(H), torch.empty_like(H), torch.empty_like(H)
    qkv, q_out = torch.empty((B, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")
    Q = torch.empty((B, Hq * D), dtype=torch.bfloat16, device="cuda")
    w = Write(rng, [0], [1], 1, 0, P)
    w.n_slots, w.P = B * Hkv * cap, P

    def state():
        K, V = pools8(np.random.default_rng(5), w, "e4m3"), pools8(np.random.default_rng(6), w, "e4m3")
        return [K[0], V[0], K[1], V[1]], [torch.zeros((B, Hkv, cap * P, D), dtype=torch.bfloat16, device="cuda") for _ in "KV"]

    def step(pools, copy):
        rows = qkv.view(B, Hq + 2 * Hkv, D)
        st["prev"].copy_(st["seq"])
        st["seq"].add_(1)
        bs.add_norm("rms", Y, H, wn, w_ahead=kw.repeat(2), H_out=H1, X=X, X_ahead=Xa)
        torch.matmul(X, Wqkv.t(), out=qkv)
        bs.append_rotated_kv8(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], rope, table, st["seq"], B, Hkv, P, *pools, prev_len=st["prev"],
                              k_norm=kw, q=rows[:, :Hq], q_norm=qw, q_out=q_out, status=st["status"])
        bs.read_kv8(*pools, table, st["seq"], B, Hkv, P, *copy, status=st["status"])
        bs.predict_q_rotated(Xa, Wp, st["prev"], rope, norm=qw, Q=Q, status=st["status"])
        H.copy_(H1)
        return [H1, X, Xa, q_out, Q]

    one, two = state(), state()
    inputs = [bf16(rng, B, N) for _ in range(20)]
    seq0, H0 = st["seq"].clone(), H.clone()
    want = []
    for y in inputs:
        Y.copy_(y)
        want.append([t.clone() for t in step(*one)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st["seq"].copy_(seq0), H.copy_(H0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = step(*two)
    torch.cuda.synchronize()
    st["seq"].copy_(seq0), H.copy_(H0)
    for y, expect in zip(inputs, want):
        Y.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(expect, out))
    assert all(same(a, b) for a, b in zip(one[0] + one[1], two[0] + two[1])) and int(st["status"]) == 0
