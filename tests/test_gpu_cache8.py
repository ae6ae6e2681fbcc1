"""GPU parity of the block tables, the cache writes and the 8-bit paged cache against the fp64
oracle (oracle/cache8_oracle.py).

Tolerances.  Tables, bf16 writes, codes and scales are bit-exact; min/max digests are the exact
value rounded down and up; a mean passes each value through at most seven roundings of its sum and
two more (scale / count, and the product), so it is off by at most 9 * 2^-24 of the mean magnitude
(10 are allowed, for the products of the roundings).  Attention, per head, with A = scale *
max_t sum_c |q_c k_tc| and n tokens: a score is 16 accumulations (two of them joined) of exact
products, each off by at most 2^-23 A, and two fp32 products, so it is off by at most
es = 17 * 2^-23 A + 2^-22 A; the weights are off by 2 es (numerator and sum), 2^-20 (exp2, the split
and the scales) and n 2^-24 (the running sums), all relative, against sum_t p_t |v_t|.  The bf16 result
adds half a step of bf16, 2^-9 .. 2^-8 of the value."""
import sys
import threading

import numpy as np
import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from oracle import cache8_oracle as C8
from _parity import ensure_built

pytestmark = pytest.mark.gpu
D = 128
DT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return dev(np.asarray(a, dtype=np.int32))


def pool8(codes, fmt):
    return dev(codes).view(DT[fmt])


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def words_of(bits):
    B, H, n = bits.shape
    w = np.zeros((B, H, -(-n // 32) * 32), np.uint64)
    w[..., :n] = bits
    w = (w.reshape(B, H, -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def bf16_values(rng, shape, outliers=True):
    x = rng.standard_normal(shape).astype(np.float32)
    if outliers:
        x[..., rng.integers(0, shape[-1], 3)] *= 7.0
    return torch.from_numpy(x).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# build_tables
# ---------------------------------------------------------------------------
def run_tables(prev, seq, free, n_slots, Hkv, P, cap, table=None, bits=None, max_tokens=None, max_list=None,
               use_free=True, stream=None):
    B = len(seq)
    exp = C8.build_tables(prev, seq, free, n_slots, Hkv, P, cap, table, bits, max_tokens, max_list)
    t = torch.full((B, Hkv, cap), -77, dtype=torch.int32, device="cuda") if prev is None else i32(table)
    w = torch.full((B, Hkv, -(-cap // 32)), -77, dtype=torch.int32, device="cuda") if prev is None else dev(words_of(bits))
    out = {"cu": torch.full((B + 1,), -7, dtype=torch.int32, device="cuda"),
           "slot_map": torch.full(exp["slot_map"].shape, -7, dtype=torch.int64, device="cuda"),
           "block_list": torch.full(exp["block_list"].shape, -7, dtype=torch.int32, device="cuda"),
           "counts": torch.full((3,), -7, dtype=torch.int32, device="cuda"),
           "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    seq_t, prev_t = i32(seq), None if prev is None else i32(prev)
    free_t = i32(free) if use_free else None
    torch.cuda.synchronize()
    bs.build_tables(seq_t, free_t, n_slots, B, Hkv, P, t, w, prev_len=prev_t, cu_tokens=out["cu"],
                    slot_map=out["slot_map"], block_list=out["block_list"], counts=out["counts"], status=out["status"],
                    stream=stream)
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), exp["table"])
    assert np.array_equal(w.cpu().numpy(), words_of(exp["bits"]))
    for n in ("cu", "slot_map", "block_list", "counts"):
        assert np.array_equal(out[n].cpu().numpy(), exp[n]), n
    assert int(out["status"]) == exp["status"]
    return exp


@pytest.mark.parametrize("B,Hkv,P,cap,top", [
    (1, 1, 32, 1, 1), (1, 2, 16, 3, 47), (3, 3, 32, 40, 1250), (5, 8, 64, 33, 2100), (2, 40, 16, 65, 1030),
    (40, 8, 32, 64, 2048), (300, 1, 16, 9, 140), (2, 1, 32, 300, 9600)])
def test_tables_fresh_then_grown(B, Hkv, P, cap, top):
    rng = np.random.default_rng(B * 1000 + P)
    seq = rng.integers(0, top + 1, B)
    seq[rng.integers(0, B)] = top
    n_slots = B * Hkv * cap + 3
    free = rng.permutation(n_slots)
    one = run_tables(None, seq, free, n_slots, Hkv, P, cap, max_tokens=int(seq.sum()) + 5)
    used = one["counts"][2]
    grown = np.minimum(seq + rng.choice([0, 1, 2, P, 3 * P + 1], B), cap * P)
    run_tables(seq, grown, free[used:], n_slots, Hkv, P, cap, one["table"], one["bits"],
               max_list=one["block_list"].shape[0] + 300)
    run_tables(seq, seq, free[used:], n_slots, Hkv, P, cap, one["table"], one["bits"], max_tokens=2, max_list=3)


def test_tables_of_the_largest_batch_and_a_map_at_an_odd_address():
    rng = np.random.default_rng(9)
    seq = rng.integers(0, 60, 4096)
    n_slots = 4096 * 4 * 2
    run_tables(None, seq, rng.permutation(n_slots), n_slots, 2, 16, 4)
    exp = C8.build_tables(None, [33, 70], np.arange(20), 20, 4, 32, 3)
    m = torch.full((1 + 103 * 4,), -7, dtype=torch.int64, device="cuda")[1:].view(103, 4)  # 8 bytes past a 16-byte boundary
    t, w = (torch.zeros((2, 4, n), dtype=torch.int32, device="cuda") for n in (3, 1))
    bs.build_tables(i32([33, 70]), None, 20, 2, 4, 32, t, w, slot_map=m)
    assert np.array_equal(m.cpu().numpy(), exp["slot_map"])


def test_tables_stale_bits_of_new_blocks_are_replaced():
    # a row that an earlier, longer sequence has left bits in; two of the new blocks get no slot
    table, bits = -np.ones((1, 1, 40), int), np.ones((1, 1, 40), bool)
    table[0, 0, 0] = 7
    exp = run_tables([20], [5 * 32], [3, 4], 10, 1, 32, 40, table, bits)
    assert exp["bits"][0, 0, :6].tolist() == [True, True, True, False, False, True] and exp["status"] == 4


def test_tables_identity_slots_and_optional_outputs():
    run_tables(None, [70, 5], np.arange(100), 100, 2, 32, 4, use_free=False)
    seq, t = i32([33]), torch.zeros((1, 1, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((1, 1, 1), dtype=torch.int32, device="cuda")
    bs.build_tables(seq, None, 9, 1, 1, 32, t, w)
    assert t.flatten().tolist() == [0, 1] and w.item() == 3


@pytest.mark.parametrize("what", ["few_slots", "bad_slots", "too_long", "negative", "shrunk", "short_map", "no_tail"])
def test_tables_report_what_did_not_fit(what):
    rng = np.random.default_rng(3)
    seq, prev = [100, 33, 64], [90, 0, 31]
    table = -np.ones((3, 2, 5), int)
    bits = np.zeros((3, 2, 5), bool)
    table[0, :, :3], table[2, :, :1] = [[1, 2, 3], [4, 5, 6]], [[7], [8]]
    bits[0, :, :3] = bits[2, :, :1] = True
    free, kw = rng.permutation(np.arange(9, 40)), {}
    if what == "few_slots":
        free = free[:5]
    elif what == "bad_slots":
        free[[0, 3]] = -4, 40
    elif what == "too_long":
        seq[1] = 161
    elif what == "negative":
        seq[1], prev[2] = -3, -1
    elif what == "shrunk":
        prev[0] = 101
    elif what == "short_map":
        kw = {"max_tokens": 20, "max_list": 4}
    else:
        table[0, 1, 2] = -1
    exp = run_tables(prev, seq, free, 40, 2, 32, 5, table, bits, **kw)
    assert exp["status"] == (4 if what in ("few_slots", "too_long", "short_map") else 1)


# ---------------------------------------------------------------------------
# append_kv
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,Hkv,P,pad", [(1, 1, 16, 0), (7, 3, 32, 64), (130, 8, 64, 512), (1000, 2, 32, 8)])
def test_append_rows_land_where_the_map_says(n, Hkv, P, pad):
    rng = np.random.default_rng(n)
    n_slots = -(-n * Hkv // P) + 4
    rows = rng.permutation(n_slots * P)[: n * Hkv].reshape(n, Hkv).astype(np.int64)
    rows[rng.random((n, Hkv)) < 0.2] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = [bf16_values(rng, (n, Hkv * D + pad)).cuda()[:, pad:].view(n, Hkv, D) for _ in range(2)]
    new[1] = new[1].contiguous()  # one strided, one packed
    pools = [torch.full((n_slots, P, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    exp = [p.clone() for p in pools]
    for e, x in zip(exp, new):
        live = rows >= 0
        e.view(-1, D)[dev(rows[live])] = x[dev(live)]
    bs.append_kv(new[0], new[1], dev(rows), Hkv, P, *pools, status=status)
    assert all(torch.equal(a, b) for a, b in zip(pools, exp)) and int(status) == 0
    if n > 1:
        rows[1, 0] = n_slots * P  # outside: skipped and reported
        before = [p.clone() for p in pools]
        bs.append_kv(new[0], new[1], dev(rows), Hkv, P, *pools, status=status)
        assert int(status) == 1 and all(torch.equal(a, b) for a, b in zip(pools, before))


# ---------------------------------------------------------------------------
# append_kv8
# ---------------------------------------------------------------------------
def make_tables(rng, seq, Hkv, P, cap, spare=3):
    """Slots for every valid block of each unit; -> (table, n_slots)."""
    B = len(seq)
    n = sum(-(-int(s) // P) for s in seq) * Hkv
    perm, table, at = rng.permutation(n + spare), -np.ones((B, Hkv, cap), int), 0
    for b, s in enumerate(seq):
        for h in range(Hkv):
            m = -(-int(s) // P)
            table[b, h, :m] = perm[at:at + m]
            at += m
    return table, n + spare


def run_append8(rng, x, v, prev, seq, table, n_slots, codes, scales, fmt, P, **kw):
    Hkv = x.shape[1]
    pools = [pool8(c, fmt) for c in codes]
    sc = [dev(s.astype(np.float32)) for s in scales]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bs.append_kv8(x.cuda() if not x.is_cuda else x, v.cuda() if not v.is_cuda else v, i32(table), i32(seq), len(seq), Hkv, P,
                  *pools, *sc, prev_len=None if prev is None else i32(prev), status=status, **kw)
    torch.cuda.synchronize()
    out = []
    for i, new in enumerate((x, v)):
        ec, es = C8.append8(new.double().cpu().numpy(), prev, seq, table, codes[i], scales[i], fmt, P)
        assert np.array_equal(sc[i].cpu().numpy(), es.astype(np.float32))
        got = codes_of(pools[i])
        # NaN codes compare as NaN whatever their sign
        same = (got == ec) | (np.isnan(C8.decode(got, fmt)) & np.isnan(C8.decode(ec, fmt)))
        assert same.all()
        out.append((got, es))
    return out, int(status)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("B,Hkv,P,top", [(1, 1, 16, 1), (3, 2, 32, 100), (4, 8, 64, 300), (70, 1, 16, 40)])
def test_append8_prompt_then_decode_steps(fmt, B, Hkv, P, top):
    rng = np.random.default_rng(P + B)
    seq = rng.integers(0, top + 1, B)
    seq[0] = top
    steps = [seq]
    for d in (1, 1, 3, P):
        steps.append(steps[-1] + np.where(rng.random(B) < 0.8, d, 0))
    cap = -(-int(steps[-1].max()) // P) + 1
    table, n_slots = make_tables(rng, steps[-1], Hkv, P, cap)
    codes = [rng.integers(0, 120, (n_slots, P, D)).astype(np.uint8) for _ in range(2)]
    scales = [np.full(n_slots, 2.0 ** -3) for _ in range(2)]
    prev = None
    for i, s in enumerate(steps):
        n = int(s.sum() - (0 if prev is None else prev.sum()))
        x, v = (bf16_values(rng, (n, Hkv, D)) * 2.0 ** (2 * i - 3) for _ in range(2))  # each step larger: scales grow
        if n:
            out, status = run_append8(rng, x, v, prev, s, table, n_slots, codes, scales, fmt, P)
            assert status == 0
            codes, scales = [c for c, _ in out], [c for _, c in out]
            again, _ = run_append8(rng, x, v, prev, s, table, n_slots, codes, scales, fmt, P)  # changes nothing
            assert all(np.array_equal(a[0], c) for a, c in zip(again, codes))
        prev = s


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_append8_after_scales_that_are_no_powers_of_two(fmt):
    # another writer's scales: kept as they are while they cover, outgrown by a power of two otherwise;
    # the arithmetic is fp32: x * (1 / scale), and code * (old / new)
    rng = np.random.default_rng(8)
    prev, seq, P = [5, 20, 31], [9, 32, 64], 32
    table, n_slots = make_tables(rng, seq, 2, P, 2)
    codes = finite_codes(rng, (n_slots, P, D), fmt)
    # against new values of up to 15: 448 * 0.021 and 57344 * 0.00016 cover 9.4, so some scales grow and some stay
    old = ((rng.random(n_slots) * 0.02 + 1e-3) * (448.0 / C8.LARGEST[fmt])).astype(np.float32)
    n = sum(seq) - sum(prev)
    x = bf16_values(rng, (n, 2, D))
    x[:4] *= 2.0 ** -9
    pools, sc = [pool8(codes, fmt) for _ in range(2)], [dev(old) for _ in range(2)]
    bs.append_kv8(x.cuda(), x.cuda(), i32(table), i32(seq), 3, 2, P, *pools, *sc, prev_len=i32(prev))
    row, f32 = 0, np.float32
    exp, es = codes.copy(), old.copy()
    for b in range(3):
        for h in range(2):
            s, had = table[b, h, prev[b] // P], prev[b] % P
            hi = min(seq[b], (prev[b] // P + 1) * P) - prev[b]
            new = x[row:row + hi, h].float().numpy()
            need = f32(C8.block_scale(new.astype(np.float64), fmt))
            if need > old[s]:
                es[s] = need
                exp[s, :had] = C8.encode((C8.decode(codes[s, :had], fmt).astype(f32) * (old[s] / need)).astype(np.float64), fmt)
            exp[s, had:had + hi] = C8.encode((new * (f32(1) / es[s])).astype(np.float64), fmt)
        row += seq[b] - prev[b]
    first = [table[b, h, prev[b] // P] for b in range(3) for h in range(2)]
    assert (es[first] == old[first]).any() and (es[first] != old[first]).any()
    for p, s in zip(pools, sc):
        assert np.array_equal(codes_of(p)[first], exp[first]) and np.array_equal(s.cpu().numpy()[first], es[first])


def test_append8_odd_values_and_strides():
    rng = np.random.default_rng(5)
    seq, Hkv, P = [37, 16, 80], 2, 16
    table, n_slots = make_tables(rng, seq, Hkv, P, 6)
    wide = bf16_values(rng, (133, 3 * Hkv * D)).cuda()
    x, v = wide[:, Hkv * D:2 * Hkv * D].view(133, Hkv, D), wide[:, 2 * Hkv * D:].view(133, Hkv, D)
    x[3, 0, 5], x[4, 1, 6], x[40, 0, 0] = float("inf"), float("nan"), float("-inf")
    x[17:32, 1] = 0.0
    x[32:37, 0] = float("nan")
    v[:16, 0] = 2.0 ** -133  # bf16 subnormals: the smallest scale
    v[60] = 3.3e38
    for fmt in ("e4m3", "e5m2"):
        codes = [np.full((n_slots, P, D), 0x31, np.uint8) for _ in range(2)]
        out, status = run_append8(rng, x, v, None, seq, table, n_slots, codes, [np.ones(n_slots)] * 2, fmt, P)
        assert status == 0
        assert (out[0][0][table[0, 0, 2], 5:] == 0x31).all()  # rows past the sequence's end


def test_append8_bad_blocks_are_skipped_and_reported():
    rng = np.random.default_rng(6)
    seq, Hkv, P = [40, 70], 2, 32
    table, n_slots = make_tables(rng, seq, Hkv, P, 3)
    x, v = bf16_values(rng, (110, Hkv, D)), bf16_values(rng, (110, Hkv, D))
    codes = [np.full((n_slots, P, D), 0x31, np.uint8) for _ in range(2)]
    table[0, 1, 1], table[1, 0, 0] = -1, n_slots
    _, status = run_append8(rng, x, v, None, seq, table, n_slots, codes, [np.ones(n_slots)] * 2, "e4m3", P)
    assert status == 1
    # fewer rows than the lengths say: the blocks that need the missing rows are skipped
    pools = [pool8(c, "e4m3") for c in codes]
    sc = [torch.ones(n_slots, device="cuda") for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, n_slots = make_tables(rng, seq, Hkv, P, 3)
    bs.append_kv8(x[:100].cuda(), v[:100].cuda(), i32(table), i32(seq), 2, Hkv, P, *pools, *sc, status=st)
    assert int(st) == 1
    got = codes_of(pools[0])
    assert (got[table[1, :, 0]] != 0x31).any(axis=(1, 2)).all()  # block 0 takes token rows 40..71
    assert (got[table[1, :, 1:3]] == 0x31).all()                 # blocks 1 and 2 need rows up to 103 and 109
    st.zero_()
    bs.append_kv8(x.cuda(), v.cuda(), i32(table), i32([40, 999]), 2, Hkv, P, *pools, *sc, status=st)
    assert int(st) & 4


# ---------------------------------------------------------------------------
# build_digest8
# ---------------------------------------------------------------------------
def finite_codes(rng, shape, fmt):
    c = rng.integers(0, 256, shape).astype(np.uint8)
    c[~np.isfinite(C8.decode(c, fmt))] = 0x35
    return c


def check_digest(got, exp, kind, written, mag=None):
    if kind == "minmax":
        lo, hi = got[..., 0, :].astype(np.float64)[written], got[..., 1, :].astype(np.float64)[written]
        elo, ehi = exp[..., 0, :][written], exp[..., 1, :][written]
        assert (lo <= elo).all() and (hi >= ehi).all()
        step = 2.0 ** -7  # the next bf16 number is at most this far, relative (normal values)
        assert (elo - lo <= step * np.abs(elo)).all() and (hi - ehi <= step * np.abs(ehi)).all()
        b = torch.from_numpy
        for x, e in ((lo, elo), (hi, ehi)):  # exact wherever the value is a bf16 number
            f = b(e.astype(np.float32)).to(torch.bfloat16).double().numpy()
            assert (x == e)[f == e].all()
    else:
        assert (np.abs(got.astype(np.float64) - exp)[written] <= 10 * 2.0 ** -24 * mag[written]).all()
    assert (got[~written] == 4096.0).all()


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("kind,fmt,B,Hkv,P,top", [
    ("minmax", "e4m3", 1, 1, 16, 1), ("minmax", "e4m3", 3, 2, 32, 301), ("minmax", "e5m2", 2, 3, 64, 500),
    ("mean", "e4m3", 2, 2, 16, 77), ("mean", "e5m2", 3, 1, 32, 200), ("mean", "e4m3", 2, 2, 64, 333)])
def test_digest8(kind, fmt, B, Hkv, P, top, pow2):
    rng = np.random.default_rng(P)
    seq = rng.integers(1, top + 1, B)
    seq[0] = top
    cap = -(-top // P) + 2
    table, n_slots = make_tables(rng, seq, Hkv, P, cap)
    codes = finite_codes(rng, (n_slots, P, D), fmt)
    scales = (2.0 ** rng.integers(-9, 3, n_slots) if pow2 else rng.random(n_slots) + 1e-3).astype(np.float32)
    shape = (B, Hkv, cap, 2, D) if kind == "minmax" else (B, Hkv, cap, D)
    ddt = torch.bfloat16 if kind == "minmax" else torch.float32
    exp = C8.digest8(kind, codes, scales, table, seq, fmt, P, np.full(shape, 4096.0))
    mag = C8.digest8(kind, codes & 0x7F, scales, table, seq, fmt, P, np.full(shape, 4096.0))  # of the magnitudes
    written = np.broadcast_to((np.arange(cap) * P < seq[:, None])[:, None, :], (B, Hkv, cap))
    dg = torch.full(shape, 4096.0, dtype=ddt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (kind, pool8(codes, fmt), dev(scales), i32(table), i32(seq), B, Hkv, P)
    bs.build_digest8(*args, dg, status=status)
    check_digest(dg.float().cpu().numpy(), exp, kind, written, mag)
    assert int(status) == 0
    # by list: padding is skipped, the rest of the digest stays
    pick = [(u, j) for u in range(B * Hkv) for j in range(cap) if written.reshape(-1, cap)[u, j]][::2]
    lst = np.full((len(pick) + 3, 2), -1)
    lst[1:len(pick) + 1] = pick
    dg.fill_(4096.0)
    bs.build_digest8(*args, dg, block_list=i32(lst), status=status)
    sel = np.zeros((B * Hkv, cap), bool)
    sel[tuple(np.array(pick).T)] = True
    check_digest(dg.float().cpu().numpy(), exp, kind, sel.reshape(B, Hkv, cap), mag)
    assert int(status) == 0
    bs.build_digest8(*args, dg, block_list=i32([[B * Hkv, 0], [0, -1], [-1, 0], [0, cap]]), status=status)
    assert int(status) == 1


# ---------------------------------------------------------------------------
# sparse_attn8
# ---------------------------------------------------------------------------
class Attn:
    """One problem: host arrays and their device copies."""

    def __init__(self, seed, fmt="e4m3", B=2, Hkv=2, G=4, P=32, top=600, k=8, scales="mixed", lens=None, spare=2):
        rng = self.rng = np.random.default_rng(seed)
        self.fmt, self.B, self.Hkv, self.G, self.P, self.k = fmt, B, Hkv, G, P, k
        self.seq = np.array(lens if lens is not None else rng.integers(1, top + 1, B))
        self.cap = -(-int(self.seq.max()) // P) + 1
        self.table, self.n_slots = make_tables(rng, self.seq, Hkv, P, self.cap, spare)
        self.q = bf16_values(rng, (B, Hkv * G, D))
        std = {"e4m3": 40.0, "e5m2": 40.0}[fmt]
        self.kc, self.vc = (C8.encode(np.clip(rng.standard_normal((self.n_slots, P, D)) * std, -440, 440), fmt)
                            for _ in range(2))
        if scales == "mixed":
            self.ks, self.vs = ((rng.random(self.n_slots) + 0.2) / 30 for _ in range(2))
        elif scales == "wild":  # blocks whose values differ by many binades
            self.ks, self.vs = 2.0 ** rng.integers(-9, -3, self.n_slots), 2.0 ** rng.integers(-60, 60, self.n_slots)
        else:
            self.ks, self.vs = np.full(self.n_slots, 2.0 ** -5), np.full(self.n_slots, 2.0 ** -5)
        self.ks, self.vs = self.ks.astype(np.float32), self.vs.astype(np.float32)
        self.lists = -np.ones((B, Hkv, k), int)
        self.counts = np.zeros((B, Hkv), int)
        for b in range(B):
            valid = -(-int(self.seq[b]) // P)
            for h in range(Hkv):
                c = int(rng.integers(0, min(k, valid) + 1)) if (b + h) % 3 else min(k, valid)
                pick = np.sort(rng.permutation(valid)[:c])
                if c and (b + h) % 2 == 0:
                    pick[-1] = valid - 1  # the partly filled last block
                self.lists[b, h, :c], self.counts[b, h] = pick, c
        self.scale = float(np.float32(D ** -0.5))
        self.O_cpu = rng.standard_normal((B, Hkv * G, D)).astype(np.float32)
        self.lse_cpu = (rng.standard_normal((B, Hkv * G)) * 3).astype(np.float32)
        self.lse_cpu[:, ::2] = -np.inf

    def device(self):
        t = (self.q.cuda(), pool8(self.kc, self.fmt), pool8(self.vc, self.fmt), dev(self.ks), dev(self.vs),
             i32(self.table), i32(self.seq), i32(self.lists), i32(self.counts))
        return t + (self.B, self.Hkv * self.G, self.Hkv, self.P, self.k, self.scale)

    def workspace(self):
        return bs.sparse_attn8_workspace(self.B, self.Hkv * self.G, self.Hkv, self.P)

    def expect(self):
        return C8.attn8(self.q.double().numpy(), self.kc, self.vc, self.ks, self.vs, self.fmt, self.table, self.seq,
                        self.lists, self.counts, self.P, self.scale)

    def check(self, O_got, lse_got, merged=False):
        eO, el, mag, big, n = self.expect()
        es = (17 * 2.0 ** -23 + 2.0 ** -22) * big
        rel = 2 * es + 2.0 ** -20 + n * 2.0 ** -24
        lim, lim_l = rel[..., None] * mag, rel + 2.0 ** -22 * np.where(np.isfinite(el), np.abs(el), 0)
        O_got, lse_got = O_got.double().cpu().numpy(), lse_got.double().cpu().numpy()
        if merged:
            mO, ml = C8.merge(eO, el, self.O_cpu.astype(np.float64), self.lse_cpu.astype(np.float64))
            lim = lim + 2.0 ** -8 * np.abs(mO) + (2 * rel[..., None] + 2.0 ** -20) * (np.abs(eO) + np.abs(self.O_cpu))
            lim_l = lim_l + 2.0 ** -20 * (1 + np.where(np.isfinite(ml), np.abs(ml), 0))
            eO, el = mO, ml
        assert np.array_equal(np.isfinite(lse_got), np.isfinite(el))
        assert (lse_got[~np.isfinite(el)] == -np.inf).all() and (O_got[~np.isfinite(el)] == 0).all()
        f = np.isfinite(el)
        assert (np.abs(lse_got - np.where(f, el, 0))[f] <= lim_l[f]).all()
        bad = np.abs(O_got - eO) > lim
        assert not bad.any(), (np.abs(O_got - eO)[bad].max(), lim[bad].min())

    def run(self, **kw):
        t, ws = self.device(), self.workspace()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        O_, l = bs.sparse_attn8(*t, ws, status=st, **kw)
        self.check(O_, l)
        Om, lm = bs.sparse_attn8_merge(*t, ws, dev(self.O_cpu), dev(self.lse_cpu), status=st, **kw)
        self.check(Om, lm, merged=True)
        assert int(st) == 0
        assert int(ws[:131072].view(torch.int32).abs().sum()) == 0
        return O_, l


# few units, many units, a long one among many, the even split
SPLITS = [dict(B=3, Hkv=4, G=5, P=32, top=4000, k=100), dict(B=40, Hkv=8, G=5, P=32, top=2000, k=40),
          dict(B=40, Hkv=8, G=3, P=16, lens=[3000] + [90] * 39, k=180), dict(B=2, Hkv=4, G=4, P=64, top=30000, k=400)]


@pytest.mark.parametrize("G", range(1, 9))
def test_attn8_groups(G):
    Attn(G, G=G, fmt="e4m3" if G % 2 else "e5m2", P=(16, 32, 64)[G % 3]).run()


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("lens", [[1], [15], [16], [17, 1], [31, 33], [63, 64, 65], [2000, 3, 999]])
def test_attn8_lengths(P, fmt, lens):
    Attn(len(lens) * 7 + lens[0], fmt=fmt, B=len(lens), Hkv=1, P=P, lens=lens, k=130).run()


@pytest.mark.parametrize("scales", ["pow2", "wild"])
@pytest.mark.parametrize("max_ctas", [1, 3, 7, None])
def test_attn8_splits(scales, max_ctas):
    # one CTA has every unit, few cut them at odd places, many cut each into pieces
    Attn(11, B=3, Hkv=3, G=5, P=32, top=3000, k=70, scales=scales).run(max_ctas=max_ctas)


@pytest.mark.parametrize("B,Hkv,k,P", [(1, 1, 9, 32), (1, 3, 40, 16), (2, 5, 33, 32), (7, 4, 100, 16), (9, 8, 17, 64),
                                       (16, 8, 64, 32), (19, 8, 12, 64), (1, 2, 256, 32), (1, 2, 257, 32)])
@pytest.mark.parametrize("G", [1, 8])
def test_attn8_few_units_with_short_lists(B, Hkv, k, P, G):
    # units shared by several CTAs of a cluster: lists from empty to k, parts without a step
    a = Attn(B * 100 + k, B=B, Hkv=Hkv, G=G, P=P, top=k * P + 5, k=k, scales="wild" if G == 1 else "mixed")
    a.counts[0, 0] = 0
    a.run()
    a.run(max_ctas=2 * B * Hkv + 1)


def test_attn8_long_list_over_the_whole_grid():
    Attn(12, B=1, Hkv=2, G=8, P=16, lens=[20011], k=1300).run()


def test_attn8_more_units_than_ctas():
    Attn(13, B=64, Hkv=8, G=2, P=16, top=90, k=6).run()


def test_attn8_the_most_units():
    Attn(24, B=512, Hkv=8, G=1, P=16, top=40, k=3).run()


def test_attn8_a_long_list_among_many():
    # units enough for a cluster to take several, one of them longer than a cluster's share
    a = Attn(25, B=40, Hkv=8, G=5, P=32, lens=[6000] + [100] * 39, k=180)
    a.run()
    assert a.counts[0, 0] == 180 and a.counts[1:].max() <= 4


@pytest.mark.parametrize("split", range(4))
def test_attn8_is_the_same_every_time(split):
    a = Attn(14, **SPLITS[split])
    t, ws = a.device(), a.workspace()
    O0, l0 = bs.sparse_attn8(*t, ws)
    a.check(O0, l0)
    for _ in range(20):
        O1, l1 = bs.sparse_attn8(*t, ws)
        assert torch.equal(O0, O1) and torch.equal(l0, l1)


def test_attn8_one_workspace_for_calls_of_any_shape():
    probs = [Attn(26 + i, **c) for i, c in enumerate(SPLITS)]
    ws = probs[0].workspace()
    dv = [a.device() for a in probs]
    assert all(a.workspace().numel() == ws.numel() for a in probs)
    for i in (0, 3, 1, 2, 3, 0, 2, 1):
        probs[i].check(*bs.sparse_attn8(*dv[i], ws))


@pytest.mark.parametrize("split", range(4))
def test_attn8_early_start_and_capture_without_a_call_before(split):
    # as a programmatic dependent of the kernel before it, and captured: each kernel of the four splits
    a = Attn(30, **SPLITS[split])
    t, ws = a.device(), a.workspace()
    O_, l = torch.zeros((a.B, a.Hkv * a.G, D), device="cuda"), torch.zeros((a.B, a.Hkv * a.G), device="cuda")
    d, s = t[:9], torch.cuda.Stream()
    torch.cuda.synchronize()
    call = bs.Prepared("scout_sparse_attn8", 0, *[x.data_ptr() for x in d[:5]], a.n_slots, *[x.data_ptr() for x in d[5:]],
                       a.B, a.Hkv * a.G, a.Hkv, D, a.P, a.cap, a.k, a.scale, O_.data_ptr(), l.data_ptr(), ws.data_ptr(),
                       ws.numel(), None, bs._launch(None, pdl=True), s.cuda_stream)
    for _ in range(5):
        call()
    torch.cuda.synchronize()
    a.check(O_, l)
    O_.zero_(), l.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
        call()
    g.replay()
    torch.cuda.synchronize()
    a.check(O_, l)


def test_attn8_garbage_in_masked_places():
    # NaN codes past the sequence's end, in slots no list names and as scales of those
    a = Attn(15, B=2, Hkv=2, G=3, P=32, lens=[70, 33], k=4)
    for b in range(2):
        j, n = (int(a.seq[b]) - 1) // 32, (int(a.seq[b]) - 1) % 32 + 1
        for h in range(2):
            a.kc[a.table[b, h, j], n:] = 0x7F
            a.vc[a.table[b, h, j], n:] = 0xFF
    used = {int(a.table[b, h, j]) for b in range(2) for h in range(2) for j in a.lists[b, h, : a.counts[b, h]]}
    for s in set(range(a.n_slots)) - used:
        a.kc[s], a.vc[s], a.ks[s], a.vs[s] = 0x7F, 0x7F, np.nan, np.nan
    a.run()


def test_attn8_nan_in_a_live_place_is_seen():
    a = Attn(16, B=1, Hkv=2, G=2, P=32, lens=[128], k=4, scales="pow2")
    a.kc[a.table[0, 0, a.lists[0, 0, 0]], 3, 7] = 0x7F
    O_, l = bs.sparse_attn8(*a.device(), a.workspace())
    assert torch.isnan(l[0, :2]).all() and torch.isnan(O_[0, :2]).all()
    assert torch.isfinite(l[0, 2:]).all() and torch.isfinite(O_[0, 2:]).all()
    # and through the merge, beside an empty CPU partial too
    lc = dev(np.array([[-np.inf, 1.0, -np.inf, 1.0]], np.float32))
    O_, l = bs.sparse_attn8_merge(*a.device(), a.workspace(), torch.ones((1, 4, D), device="cuda"), lc)
    assert torch.isnan(l[0, :2]).all() and torch.isnan(O_[0, :2]).all()
    assert torch.isfinite(l[0, 2:]).all() and torch.isfinite(O_[0, 2:]).all()


@pytest.mark.parametrize("split", range(4))
def test_attn8_an_empty_cpu_partial_is_not_read(split):
    a = Attn(40, **SPLITS[split])
    a.counts[0, 0] = 0  # with and without blocks on the GPU
    oc = dev(np.where(np.isinf(a.lse_cpu)[..., None], np.nan, a.O_cpu).astype(np.float32))
    a.O_cpu[np.isinf(a.lse_cpu)] = 0
    a.check(*bs.sparse_attn8_merge(*a.device(), a.workspace(), oc, dev(a.lse_cpu)), merged=True)


def test_attn8_zero_and_tiny_values():
    a = Attn(17, B=2, Hkv=2, G=4, P=32, lens=[300, 200], k=10, scales="pow2")
    a.vs[a.table[0, 0, 0]] = 0.0
    a.ks[a.table[0, 0, 1]] = 0.0
    a.vs[a.table[1]] = np.float32(2.0 ** -126)   # a block of zeros as the writer leaves it
    a.q[1, 0] = 0.0
    a.q[1, 1] *= 2.0 ** -100
    a.q[0, 1] *= 2.0 ** 40
    a.ks[a.table[0]] *= np.float32(2.0 ** -40)
    a.run()


def test_attn8_all_probability_on_a_block_of_tiny_values():
    # one token takes the softmax, in a block whose values are 2^-70 of the others'
    a = Attn(18, B=1, Hkv=1, G=1, P=32, lens=[96], k=3, scales="pow2")
    a.lists[0, 0], a.counts[0, 0] = [0, 1, 2], 3
    s = a.table[0, 0, 1]
    a.vs[s] = np.float32(2.0 ** -75)
    a.q[0, 0] = torch.full((D,), 8.0, dtype=torch.bfloat16)
    a.kc[s, 5] = C8.encode(np.full(D, 440.0), "e4m3")
    O_, _ = a.run()
    v = C8.decode(a.vc[s, 5], "e4m3") * 2.0 ** -75
    assert np.allclose(O_[0, 0].double().cpu().numpy(), v, rtol=1e-5, atol=0)


@pytest.mark.parametrize("what", ["block", "negative", "slot", "past_end"])
def test_attn8_bad_entries_are_skipped_and_reported(what):
    a = Attn(19, B=2, Hkv=2, G=2, P=16, lens=[200, 100], k=9)
    if what == "block":
        a.lists[0, 0, 1] = a.cap
    elif what == "negative":
        a.lists[0, 0, 1] = -2
    elif what == "past_end":
        a.lists[0, 0, a.counts[0, 0] - 1] = a.cap - 1
    else:
        a.table[0, 0, a.lists[0, 0, 0]] = a.n_slots
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    O_, l = bs.sparse_attn8(*a.device(), a.workspace(), status=st)
    a.check(O_, l)
    assert int(st) == 1


def test_attn8_slots_beyond_32_bit_offsets():
    # a pool of more than 2^32 bytes: the used slots lie at its end
    a = Attn(20, B=1, Hkv=2, G=4, P=32, lens=[500], k=16, scales="pow2")
    n = (1 << 32) // (32 * D) + a.n_slots
    t = list(a.device())
    far = n - a.n_slots
    for i in (1, 2):
        big = torch.empty((n, 32, D), dtype=torch.uint8, device="cuda")
        big[far:] = t[i].view(torch.uint8)
        t[i] = big.view(DT[a.fmt])
    for i in (3, 4):
        s = torch.zeros(n, device="cuda")
        s[far:] = t[i]
        t[i] = s
    t[5] = i32(np.where(a.table >= 0, a.table + far, -1))
    a.check(*bs.sparse_attn8(*t, a.workspace()))
    dg = torch.zeros((1, 2, a.cap, 2, D), dtype=torch.bfloat16, device="cuda")
    bs.build_digest8("minmax", t[1], t[3], t[5], t[6], 1, 2, 32, dg)
    exp = C8.digest8("minmax", a.kc, a.ks, a.table, a.seq, a.fmt, 32, np.zeros((1, 2, a.cap, 2, D)))
    assert np.array_equal(dg.double().cpu().numpy(), exp)
    x = bf16_values(a.rng, (500, 2, D))
    bs.append_kv8(x.cuda(), x.cuda(), t[5], t[6], 1, 2, 32, t[1], t[2], t[3], t[4])
    ec, es = C8.append8(x.double().numpy(), None, a.seq, a.table, a.kc, a.ks, a.fmt, 32)
    assert np.array_equal(codes_of(t[1][far:]), ec) and np.array_equal(t[3][far:].cpu().numpy(), es)


def test_attn8_on_other_streams_and_in_graphs():
    probs = [Attn(21, B=2, Hkv=2, G=4, P=32, top=3000, k=60), Attn(22, B=3, Hkv=4, G=2, P=16, top=900, k=40, fmt="e5m2")]
    work = []
    for a in probs:
        t, ws, s = a.device(), a.workspace(), torch.cuda.Stream()
        O_ = torch.zeros((a.B, a.Hkv * a.G, D), device="cuda")
        l = torch.zeros((a.B, a.Hkv * a.G), device="cuda")
        torch.cuda.synchronize()
        bs.sparse_attn8(*t, ws, O=O_, lse=l, stream=s)
        torch.cuda.synchronize()
        a.check(O_, l)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bs.sparse_attn8(*t, ws, O=O_, lse=l)
        O_.zero_(), l.zero_()
        work.append((a, g, s, O_, l, t, ws))
    torch.cuda.synchronize()
    for _ in range(30):  # two graphs with a workspace each, replayed side by side
        for _, g, s, *_ in work:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, _, _, O_, l, *_ in work:
        a.check(O_, l)


@pytest.mark.parametrize("split", range(4))
def test_attn8_started_early_by_an_event(split):
    # the first call's partial is the second one's CPU partial, on another stream that waits for the event
    # the first call fires before it completes
    a, b = Attn(34, **SPLITS[split]), Attn(35, **SPLITS[split])
    ta, tb, wa, wb = a.device(), b.device(), a.workspace(), b.workspace()
    s1, s2, ev = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Event()
    Hq = a.Hkv * a.G
    O1, l1 = torch.empty((a.B, Hq, D), device="cuda"), torch.empty((a.B, Hq), device="cuda")
    O2 = torch.empty((a.B, Hq, D), dtype=torch.bfloat16, device="cuda")
    l2 = torch.empty((a.B, Hq), device="cuda")
    ev.record(s1)
    torch.cuda.synchronize()
    p = lambda t: [x.data_ptr() for x in t]  # noqa: E731
    one = bs.Prepared("scout_sparse_attn8", 0, *p(ta[:5]), a.n_slots, *p(ta[5:9]), a.B, Hq, a.Hkv, D, a.P, a.cap, a.k, a.scale,
                      *p((O1, l1, wa)), wa.numel(), None, bs._launch(None, early_event=ev), s1.cuda_stream)
    two = bs.Prepared("scout_sparse_attn8_merge", 0, *p(tb[:5]), b.n_slots, *p(tb[5:9]), b.B, Hq, b.Hkv, D, b.P, b.cap, b.k,
                      b.scale, *p((O1, l1, O2, l2, wb)), wb.numel(), None, None, s2.cuda_stream)
    for _ in range(3):
        O1.fill_(3.0), l1.fill_(3.0)
        torch.cuda.synchronize()
        one()
        s2.wait_event(ev)
        two()
        torch.cuda.synchronize()
        a.check(O1, l1)
        b.O_cpu, b.lse_cpu = O1.cpu().numpy(), l1.cpu().numpy()
        b.check(O2, l2, merged=True)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,P", [("e4m3", 32), ("e5m2", 16)])
def test_prompt_and_decode_steps_through_the_whole_path(fmt, P):
    """Lengths -> tables -> quantised write -> digests -> selection -> merged attention, for a
    prompt and then token by token, each stage checked against the oracle on the stage before."""
    rng = np.random.default_rng(P)
    B, Hkv, G, k = 3, 2, 4, 6
    Hq, U = Hkv * G, B * Hkv
    seq = np.array([300, 47, 5 * P])
    cap = -(-int(seq.max() + P + 2) // P)  # the steps below add P + 2 tokens at most
    words, n_slots = -(-cap // 32), U * cap
    free = i32(rng.permutation(n_slots))
    table = torch.empty((B, Hkv, cap), dtype=torch.int32, device="cuda")
    bits = torch.empty((B, Hkv, words), dtype=torch.int32, device="cuda")
    pools = [torch.zeros((n_slots, P, D), dtype=torch.uint8, device="cuda").view(DT[fmt]) for _ in range(2)]
    scales = [torch.zeros(n_slots, device="cuda") for _ in range(2)]
    dg = torch.zeros((B, Hkv, cap, 2, D), dtype=torch.bfloat16, device="cuda")
    ws_t, ws_a = bs.score_topk_workspace(B, Hkv, cap), bs.sparse_attn8_workspace(B, Hq, Hkv, P)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    counts = torch.zeros(3, dtype=torch.int32, device="cuda")
    plain = [torch.zeros((n_slots, P, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    prev, used = None, 0
    for step, grow in enumerate((None, [1, 1, 1], [1, 0, 1], [P, 3, 1])):
        now = seq if grow is None else prev + np.array(grow)
        n = int(now.sum() - (0 if prev is None else prev.sum()))
        K, V = bf16_values(rng, (n, Hkv, D)).cuda(), bf16_values(rng, (n, Hkv, D)).cuda()
        q = bf16_values(rng, (B, Hq, D)).cuda()
        lst = torch.empty((n * Hkv + U, 2), dtype=torch.int32, device="cuda")
        smap = torch.empty((n + 2, Hkv), dtype=torch.int64, device="cuda")
        pl = None if prev is None else i32(prev)
        bs.build_tables(i32(now), free[used:], n_slots, B, Hkv, P, table, bits, prev_len=pl, slot_map=smap,
                        block_list=lst, counts=counts, status=status)
        bs.append_kv(K, V, smap[:n], Hkv, P, *plain, status=status)
        bs.append_kv8(K, V, table, i32(now), B, Hkv, P, *pools, *scales, prev_len=pl, status=status)
        bs.build_digest8("minmax", pools[0], scales[0], table, i32(now), B, Hkv, P, dg, block_list=lst, status=status)
        scores = torch.empty((B, Hkv, cap), device="cuda")
        sel = bs.score_topk("minmax", q, dg, i32(now), bits, B, Hq, Hkv, P, cap, k, ws_t, scores=scores, status=status)
        O_cpu, lse_cpu = torch.zeros((B, Hq, D), device="cuda"), torch.full((B, Hq), -np.inf, device="cuda")
        Om, lm = bs.sparse_attn8_merge(q, *pools, *scales, table, i32(now), sel["res"], sel["res_count"], B, Hq, Hkv, P,
                                       k, D ** -0.5, ws_a, O_cpu, lse_cpu, status=status)
        assert int(status) == 0
        used += int(counts[2])
        tab = table.cpu().numpy()
        # every block is resident, so the attention's list is the whole selection
        assert torch.equal(sel["res_count"], sel["topk_count"])
        codes = [codes_of(p) for p in pools]
        sc = [s.cpu().numpy() for s in scales]
        exp = C8.digest8("minmax", codes[0], sc[0], tab, now, fmt, P, np.zeros((B, Hkv, cap, 2, D)))
        assert np.array_equal(dg.double().cpu().numpy(), exp)
        for b in range(B):
            for h in range(Hkv):
                m = -(-int(now[b]) // P)
                for i in range(2):  # what the codes stand for is near what was written (half a code step)
                    page = C8.decode(codes[i][tab[b, h, :m]], fmt) * sc[i][tab[b, h, :m]][:, None, None]
                    want = plain[i].double().cpu().numpy()[tab[b, h, :m]]
                    live = np.arange(m * P).reshape(m, P, 1) < now[b]
                    # half a step of the code, or of its smallest normal; twice that after a recoding
                    half = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}[fmt]
                    low = {"e4m3": 2.0 ** -6, "e5m2": 2.0 ** -14}[fmt] * sc[i][tab[b, h, :m]][:, None, None]
                    assert (np.abs(page - want) <= np.where(live, 2 * half * np.maximum(np.abs(want), low), np.inf)).all()
                s = scores[b, h, :m].double().cpu().numpy()
                kk = min(k, m)
                assert sel["topk"][b, h, :kk].tolist() == sorted(np.lexsort((np.arange(m), -s))[:kk].tolist())
        e = C8.attn8(q.double().cpu().numpy(), *codes, *sc, fmt, tab, now, sel["res"].cpu().numpy(),
                     sel["res_count"].cpu().numpy(), P, D ** -0.5)
        rel = 2 * (17 * 2.0 ** -23 + 2.0 ** -22) * e[3] + 2.0 ** -20 + e[4] * 2.0 ** -24
        lim = (rel[..., None] + 2.0 ** -8) * e[2]
        assert (np.abs(Om.double().cpu().numpy() - e[0]) <= lim).all()
        prev = now


def test_calls_refuse_tensors_elsewhere_and_of_other_sizes():
    a = Attn(23)
    t, ws = list(a.device()), a.workspace()
    for i, bad in ((0, t[0][:1]), (3, t[3][:-1]), (5, t[5].long()), (7, t[7].cpu()), (2, t[2][:-1])):
        with pytest.raises(bs.ScoutError):
            bs.sparse_attn8(*t[:i], bad, *t[i + 1:], ws)
    with pytest.raises(bs.ScoutError):
        bs.sparse_attn8(*t, ws[:100])
    with pytest.raises(bs.ScoutError):
        bs.build_digest8("minmax", t[1], t[3], t[5], t[6], a.B, a.Hkv, a.P, torch.zeros(4, device="cuda"))
    dg = torch.full((a.B, a.Hkv, a.cap, 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    bs.build_digest8("minmax", t[1], t[3], t[5], t[6], a.B, a.Hkv, a.P, dg, block_list=i32(np.zeros((0, 2))))
    assert (dg == 5.0).all()  # an empty list is no block, not every block


def test_outputs_of_the_binding():
    """Given outputs come back as the same objects, new ones belong to the call's stream and are freed with the
    last reference; a refused call keeps nothing."""
    a = Attn(24, B=2, Hkv=2, G=4, P=32, top=900, k=20)
    t, ws = a.device(), a.workspace()
    O_, l = torch.zeros((a.B, a.Hkv * a.G, D), device="cuda"), torch.zeros((a.B, a.Hkv * a.G), device="cuda")
    r = bs.sparse_attn8(*t, ws, O=O_, lse=l)
    assert r[0] is O_ and r[1] is l
    a.check(O_, l)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (s, None):
        with torch.cuda.stream(s):  # named, and current
            r = bs.sparse_attn8(*t, ws, stream=given)
        torch.cuda.synchronize()
        assert r[0].shape == O_.shape and r[0].dtype == torch.float32 and torch.equal(r[0], O_) and torch.equal(r[1], l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = bs.sparse_attn8(*t, ws)  # outputs from the graph's pool
    r[0].zero_(), r[1].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r[0], O_) and torch.equal(r[1], l)
    refs, held = [sys.getrefcount(x) for x in (*t[:9], ws, O_, l)], torch.cuda.memory_allocated()
    for _ in range(200):
        bs.sparse_attn8(*t, ws)
        bs.sparse_attn8(*t, ws, O=O_)
        with pytest.raises(bs.ScoutError):
            bs.sparse_attn8(*t, ws, O=O_[:1], lse=l)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held and refs == [sys.getrefcount(x) for x in (*t[:9], ws, O_, l)]


def test_calls_from_several_threads():
    """Each thread with its own problem, workspace and stream, all calling at once."""
    probs = [Attn(30 + i, B=1 + i, Hkv=2, G=4, P=32, top=900, k=20) for i in range(4)]
    out, failed = [None] * 4, []
    dev = [(a.device(), a.workspace(), torch.cuda.Stream()) for a in probs]
    torch.cuda.synchronize()

    def run(i):
        try:
            t, ws, s = dev[i]
            for _ in range(100):
                out[i] = bs.sparse_attn8(*t, ws, stream=s)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not failed
    for a, (O_, l) in zip(probs, out):
        a.check(O_, l)
