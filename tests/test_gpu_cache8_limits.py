"""The tables, cache writes and 8-bit cache at the ends of what they take: batches around a limit of the
launch, calls without rows, tables wider than 32-bit token numbers, values that are not finite, counts
outside their lists, failures of a wait and of an allocation, recalled blocks."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from oracle import cache8_oracle as C8
from _parity import ensure_built
from test_gpu_cache8 import D, DT, SPLITS, Attn, bf16_values, codes_of, dev, finite_codes, i32, make_tables, pool8

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# build_tables
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B", [2437, 2438, 2457, 2458])
def test_tables_of_batches_around_48_kb_of_shared_memory(B):
    # (5 B + 3) * 4 bytes and the kernel's own 384 pass 48 KB from 2,438 sequences on; in a process of its own,
    # as a call with a larger batch would raise the kernel's limit for those after it
    text = f"""
import torch, block_sparse_kv_pred_gb300 as bs
n = torch.arange({B}, dtype=torch.int32, device="cuda") % 3
t = torch.full(({B}, 1, 1), -7, dtype=torch.int32, device="cuda")
w, cu = torch.full_like(t, -7), torch.zeros({B} + 1, dtype=torch.int32, device="cuda")
bs.build_tables(n, None, {B}, {B}, 1, 16, t, w, cu_tokens=cu)
has = n > 0
assert torch.equal(t.flatten()[has].long(), torch.arange(int(has.sum()), device="cuda")) and bool((t.flatten()[~has] == -1).all())
assert torch.equal(w.flatten(), has.int()) and torch.equal(cu[1:].long(), n.long().cumsum(0)) and cu[0] == 0
"""
    r = subprocess.run([sys.executable, "-c", text], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("which", ["slot_map", "block_list"])
def test_tables_with_an_empty_map_or_list(which):
    # asked for, with no room: what does not fit is reported, as with too little room
    kw = {"slot_map": torch.empty((0, 2), dtype=torch.int64, device="cuda"),
          "block_list": torch.empty((0, 2), dtype=torch.int32, device="cuda")}
    for n, want in ((5, 4), (0, 0)):
        st, t = word(), torch.full((1, 2, 2), -7, dtype=torch.int32, device="cuda")
        bs.build_tables(i32([n]), None, 4, 1, 2, 16, t, torch.zeros((1, 2, 1), dtype=torch.int32, device="cuda"),
                        status=st, **{which: kw[which]})
        assert int(st) == want and t.flatten().tolist() == ([0, -1, 1, -1] if n else [-1] * 4)


def test_tables_of_a_pool_with_the_most_slots():
    # slots whose rows' numbers pass 32 bits
    n, slots = (1 << 31) - 1, [(1 << 31) - 2, 5, (1 << 26) + 3]
    m, st = torch.full((130, 1), -7, dtype=torch.int64, device="cuda"), word()
    t, w = torch.zeros((1, 1, 3), dtype=torch.int32, device="cuda"), torch.zeros((1, 1, 1), dtype=torch.int32, device="cuda")
    bs.build_tables(i32([130]), i32(slots), n, 1, 1, 64, t, w, slot_map=m, status=st)
    assert int(st) == 0 and t.flatten().tolist() == slots
    assert m.flatten().tolist() == [slots[i // 64] * 64 + i % 64 for i in range(130)]


# ---------------------------------------------------------------------------
# append_kv
# ---------------------------------------------------------------------------
def test_append_rows_and_pools_past_32_bit_offsets():
    # rows 2^25 elements apart, into the last slots of pools of more than 2^31 elements
    rng = np.random.default_rng(58)
    n, Hkv, P, ld = 70, 2, 32, 1 << 25
    n_slots = (1 << 31) // (P * D) + 10
    at = n_slots * P - 1 - rng.permutation(n * Hkv).reshape(n, Hkv)
    x = bf16_values(rng, (n, Hkv, D)).cuda()
    wide = torch.empty((n, ld), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + Hkv * D] = x.view(n, -1)
    far, st = wide[:, 8:8 + Hkv * D].view(n, Hkv, D), word()
    pools = [torch.empty((n_slots, P, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for p in pools:
        p[-8:] = 9.0
    bs.append_kv(far, x, dev(at), Hkv, P, *pools, status=st)
    want = torch.full((8 * P, D), 9.0, dtype=torch.bfloat16, device="cuda")
    want[dev(at - (n_slots - 8) * P).flatten()] = x.view(-1, D)
    assert int(st) == 0 and all(torch.equal(p[-8:].view(-1, D), want) for p in pools)
    del pools
    # and the quantising write from the same rows
    codes, table = np.zeros((6, P, D), np.uint8), np.arange(6).reshape(1, Hkv, 3)
    pools, sc = [pool8(codes, "e4m3") for _ in range(2)], [torch.zeros(6, device="cuda") for _ in range(2)]
    bs.append_kv8(far, x, i32(table), i32([n]), 1, Hkv, P, *pools, *sc, status=st)
    ec, es = C8.append8(x.double().cpu().numpy(), None, [n], table, codes, np.zeros(6), "e4m3", P)
    assert int(st) == 0 and all(np.array_equal(codes_of(p), ec) for p in pools)
    assert all(np.array_equal(s.cpu().numpy(), es.astype(np.float32)) for s in sc)


# ---------------------------------------------------------------------------
# append_kv8
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("prev,seq,want", [(None, [40, 0], 1), ([8, 3], [8, 3], 0), ([8, 3], [8, 4], 1), (None, [0, 97], 5),
                                           (None, [0, -1], 1), ([8, 4], [8, 3], 1), (None, [0, 0], 0)])
def test_append8_without_rows_reports_what_the_lengths_say(prev, seq, want):
    Hkv, P, n_slots = 2, 32, 20
    pools = [pool8(np.full((n_slots, P, D), 0x31, np.uint8), "e4m3") for _ in range(2)]
    sc = [torch.full((n_slots,), 0.5, device="cuda") for _ in range(2)]
    table, st = i32(np.arange(2 * Hkv * 3).reshape(2, Hkv, 3)), word()
    none = torch.empty((0, Hkv, D), dtype=torch.bfloat16, device="cuda")
    bs.append_kv8(none, none, table, i32(seq), 2, Hkv, P, *pools, *sc, prev_len=None if prev is None else i32(prev),
                  status=st)
    assert int(st) == want
    assert all((codes_of(p) == 0x31).all() for p in pools) and all(bool((s == 0.5).all()) for s in sc)


@pytest.mark.parametrize("n", [1, 70, 1000])
def test_append8_stops_where_the_rows_end(n):
    # lengths that say far more than there are rows: the blocks whose rows are all there, and no others
    rng = np.random.default_rng(n)
    B, Hkv, P, cap, n_slots = 30, 2, 16, 200, 30 * 2 * 200
    seq = rng.integers(20, 60, B)
    seq[20:] = cap * P
    table = rng.permutation(n_slots).reshape(B, Hkv, cap)
    x = bf16_values(rng, (n, Hkv, D))
    codes = np.full((n_slots, P, D), 0x31, np.uint8)
    pools, sc, st = [pool8(codes, "e4m3") for _ in range(2)], [torch.ones(n_slots, device="cuda") for _ in range(2)], word()
    bs.append_kv8(x.cuda(), x.cuda(), i32(table), i32(seq), B, Hkv, P, *pools, *sc, status=st)
    # the oracle with the lengths cut to whole blocks that lie within the rows
    cut, at = np.zeros(B, int), 0
    for b in range(B):
        left = n - at
        cut[b] = seq[b] if left >= seq[b] else max(left, 0) // P * P
        at += int(seq[b])
    have = x.double().numpy()[: int(cut.sum())]
    ec, es = C8.append8(have, None, cut, table, codes, np.ones(n_slots), "e4m3", P)
    assert int(st) == 1
    for p, s in zip(pools, sc):
        assert np.array_equal(codes_of(p), ec) and np.array_equal(s.cpu().numpy(), es)


def test_append8_of_the_largest_batch_with_padding_rows():
    rng = np.random.default_rng(2)
    B, P, cap = 4096, 16, 3
    prev = rng.integers(0, 30, B)
    seq = prev + rng.integers(0, 4, B)
    table, n_slots = make_tables(rng, seq, 1, P, cap)
    n = int((seq - prev).sum())
    x = bf16_values(rng, (n + 100, 1, D))
    x[n:] = float("nan")  # rows of a padded batch, past the last new token
    codes, scales = finite_codes(rng, (n_slots, P, D), "e5m2"), 2.0 ** rng.integers(-20, -10, n_slots)
    pools, sc, st = [pool8(codes, "e5m2") for _ in range(2)], [dev(scales.astype(np.float32)) for _ in range(2)], word()
    bs.append_kv8(x.cuda(), x.cuda(), i32(table), i32(seq), B, 1, P, *pools, *sc, prev_len=i32(prev), status=st)
    ec, es = C8.append8(x.double().numpy()[:n], prev, seq, table, codes, scales, "e5m2", P)
    assert int(st) == 0
    for p, s in zip(pools, sc):
        assert np.array_equal(codes_of(p), ec) and np.array_equal(s.cpu().numpy(), es.astype(np.float32))


# ---------------------------------------------------------------------------
# tables wider than 2^31 tokens
# ---------------------------------------------------------------------------
def far_block(P):
    """(columns, block): the block starts at token 2^31 + 2 P."""
    j = (1 << 31) // P + 2
    return j + 1, j


@pytest.mark.parametrize("P", [32, 64])
def test_attn8_blocks_past_32_bit_token_numbers_are_past_the_end(P):
    a = Attn(50, B=1, Hkv=1, G=4, P=P, lens=[P], k=2)
    a.lists[0, 0], a.counts[0, 0] = [0, -1], 1
    cap, j = far_block(P)
    t, st = list(a.device()), word()
    t[5] = torch.full((1, 1, cap), int(a.table[0, 0, 0]), dtype=torch.int32, device="cuda")  # every entry names a slot
    t[7], t[8] = i32([[[0, j]]]), i32([[2]])
    O_, l = bs.sparse_attn8(*t, a.workspace(), status=st)
    a.check(O_, l)
    assert int(st) == 1


@pytest.mark.parametrize("P", [32, 64])
def test_attention_blocks_past_32_bit_token_numbers_are_past_the_end(P):
    rng = np.random.default_rng(51)
    q, K, V = (bf16_values(rng, s, outliers=False) for s in ((1, 4, D), (1, P, D), (1, P, D)))
    cap, j = far_block(P)
    table = torch.zeros((1, 1, cap), dtype=torch.int32, device="cuda")  # every entry names the only slot
    ws, st = bs.sparse_attn_workspace(1, 4, 1, P), word()
    O_, l = bs.sparse_attn(q.cuda(), K.cuda(), V.cuda(), table, i32([P]), i32([[[0, j]]]), i32([[2]]), 1, 4, 1, P, 2,
                           D ** -0.5, ws, status=st)
    s = q[0].double() @ K[0].double().T * D ** -0.5  # the block taken twice would raise the lse by log 2
    assert int(st) == 1
    assert ((l[0].cpu().double() - torch.logsumexp(s, 1)).abs() <= 2e-3).all()
    assert ((O_[0].cpu().double() - torch.softmax(s, 1) @ V[0].double()).abs() <= 2e-3).all()


@pytest.mark.parametrize("kind", ["minmax", "mean"])
def test_digests_of_blocks_past_32_bit_token_numbers_stay(kind):
    P = 64
    cap, j = far_block(P)
    table = torch.zeros((1, 1, cap), dtype=torch.int32, device="cuda")
    K, seq, lst = torch.ones((1, P, D), dtype=torch.bfloat16, device="cuda"), i32([P]), i32([[0, j], [0, 0]])
    dg = (torch.empty((1, 1, cap, 2, D), dtype=torch.bfloat16, device="cuda") if kind == "minmax" else
          torch.empty((1, 1, cap, D), device="cuda"))
    for build in (lambda: bs.build_digest(kind, K, table, seq, 1, 1, P, dg, block_list=lst),
                  lambda: bs.build_digest8(kind, pool8(np.full((1, P, D), 0x38, np.uint8), "e4m3"), torch.ones(1, device="cuda"),
                                           table, seq, 1, 1, P, dg, block_list=lst)):
        dg[0, 0, j] = 5.0
        dg[0, 0, 0] = 5.0
        build()
        assert bool((dg[0, 0, j] == 5.0).all()) and bool((dg[0, 0, 0] == 1.0).all())


# ---------------------------------------------------------------------------
# values that are not finite, counts outside the lists
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("split", [0, 1])
def test_attn8_a_v_scale_that_is_not_finite_is_seen(bad, P, split):
    # it spoils the output of its unit's heads and nothing else, their lse included
    a = Attn(52, B=(2, 40)[split], Hkv=(2, 8)[split], G=3, P=P, lens=None if split == 0 else [200] * 40, top=600, k=12)
    eO, el = a.expect()[:2]
    assert a.counts[0, 0] > 0
    a.vs[a.table[0, 0, a.lists[0, 0, 0]]] = bad
    t, ws = a.device(), a.workspace()
    O_, l = bs.sparse_attn8(*t, ws)
    Om, lm = bs.sparse_attn8_merge(*t, ws, dev(np.zeros_like(a.O_cpu)), dev(np.full_like(a.lse_cpu, -np.inf)))
    for o, s in ((O_, l), (Om, lm)):
        assert not torch.isfinite(o[0, :3]).any()
        assert np.isfinite(s[0, :3].cpu().numpy()).all() and np.abs(s[0, :3].cpu().numpy() - el[0, :3]).max() < 1e-4
        rest = o.float().cpu().numpy().reshape(-1, D)[3:]
        assert np.isfinite(rest).all() and np.abs(rest - eO.reshape(-1, D)[3:]).max() < 0.1


@pytest.mark.parametrize("shape", [dict(SPLITS[0], lens=[4000, 100, 3500]), dict(SPLITS[1], lens=[2000] * 3 + [500] * 37),
                                   SPLITS[2], dict(SPLITS[3], lens=[30000, 500])])
def test_attn8_counts_outside_the_lists_are_cut_to_them(shape):
    a = Attn(53, **shape)
    full = a.counts == a.k
    assert full.any()
    a.counts[full] = a.k + 3
    a.counts.flat[np.flatnonzero(~full)[0]] = -1
    a.run()


@pytest.mark.parametrize("shape", [dict(B=2, Hkv=2, G=4, P=16, lens=[300, 40], k=9), dict(SPLITS[3], lens=[30000, 500])])
def test_attn8_a_block_listed_more_than_once_counts_each_time(shape):
    a = Attn(59, **shape)
    c = int(a.counts[0, 0])
    a.lists[0, 0, :c] = np.sort(a.rng.choice(a.lists[0, 0, : (c + 1) // 2], c))
    a.lists[1, 1, :2], a.counts[1, 1] = 0, 2
    a.run()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("shape", [dict(B=2, Hkv=2, G=3, P=16, lens=[300, 40], k=9), dict(SPLITS[1], lens=[300] * 40, k=8)])
def test_attn8_a_query_that_is_not_finite_spoils_its_head_alone(bad, shape):
    a = Attn(60, **shape)
    assert a.counts[0, 0] > 0
    a.q[0, 1, 5] = bad
    O_, l = bs.sparse_attn8(*a.device(), a.workspace())
    assert not torch.isfinite(O_[0, 1]).any() and not torch.isfinite(l[0, 1])
    a.q[0, 1] = 0  # the other heads, to the tolerance of any call
    zero = bs.sparse_attn8(*a.device(), a.workspace())
    O_[0, 1], l[0, 1] = zero[0][0, 1], zero[1][0, 1]
    a.check(O_, l)


@pytest.mark.parametrize("shape", [*SPLITS, dict(B=64, Hkv=8, G=2, P=16, top=90, k=6), dict(B=1, Hkv=1, G=8, P=32, top=900, k=20)])
def test_attn8_with_every_list_empty(shape):
    a = Attn(61, **shape)
    a.counts[:], a.lists[:] = 0, -1
    O_, l = a.run()
    assert not O_.any() and torch.isinf(l).all()


@pytest.mark.parametrize("B,Hkv,P", [(1, 2, 32), (5, 8, 16), (64, 8, 32), (7, 4, 64)])
def test_attn8_short_lists_in_long_buffers(B, Hkv, P):
    a = Attn(62, B=B, Hkv=Hkv, G=4, P=P, top=6 * P, k=3000)
    assert a.counts.max() <= 6
    a.run()


def nan_codes(fmt):
    v = C8.code_values(fmt)
    return np.flatnonzero(np.isnan(v))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("P,n", [(16, 16), (32, 32), (32, 7), (64, 50)])
def test_digest8_passes_over_nan_codes(fmt, P, n):
    rng = np.random.default_rng(P + n)
    codes = finite_codes(rng, (1, P, D), fmt)
    bad = nan_codes(fmt)
    for c in range(0, D, 3):  # in some rows
        rows = rng.permutation(n)[: rng.integers(1, n)]
        codes[0, rows, c] = rng.choice(bad, len(rows))
    none = [5, 64, 127]       # in every row of a channel
    codes[0, :, none] = rng.choice(bad, (3, P))
    inf = np.array([], int)
    if fmt == "e5m2":
        inf = np.array([1, 70])
        codes[0, 0, inf] = 0x7C, 0xFC
    scale = np.float32(2.0 ** -3)
    x = C8.decode(codes[0, :n], fmt) * float(scale)
    x[:, none] = 0.0  # (silences numpy; replaced below)
    lo, hi = np.nanmin(x, 0), np.nanmax(x, 0)
    lo[none], hi[none] = np.inf, -np.inf
    dg = torch.zeros((1, 1, 1, 2, D), dtype=torch.bfloat16, device="cuda")
    args = pool8(codes, fmt), torch.tensor([scale], device="cuda"), i32([[[0]]]), i32([n]), 1, 1, P
    bs.build_digest8("minmax", *args, dg)
    got = dg.double().cpu().numpy()[0, 0, 0]
    assert np.array_equal(got, [lo, hi])
    if fmt == "e5m2":
        assert hi[1] == np.inf and lo[70] == -np.inf
    mean = torch.zeros((1, 1, 1, D), device="cuda")
    bs.build_digest8("mean", *args, mean)
    want = C8.decode(codes[0, :n], fmt).sum(0)
    m = mean.cpu().numpy()[0, 0, 0]
    assert np.array_equal(np.isnan(m), np.isnan(want)) and (m[inf] == want[inf]).all()


# ---------------------------------------------------------------------------
# failures
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("merge", [False, True])
@pytest.mark.parametrize("split", range(4))
def test_attn8_an_expired_wait_is_reported_and_spoils_its_units_alone(split, merge):
    # every warp gives up at its second step: what it left out shows as NaN, what was done before is right, and the
    # next call on the same workspace is right
    a = Attn(56, **SPLITS[split])
    t, ws, st = a.device(), a.workspace(), word()
    Hq = a.Hkv * a.G
    cpu = (dev(a.O_cpu), dev(a.lse_cpu)) if merge else ()
    O_ = torch.zeros((a.B, Hq, D), dtype=torch.bfloat16 if merge else torch.float32, device="cuda")
    l = torch.zeros((a.B, Hq), device="cuda")

    def call(inject):
        p = [x.data_ptr() for x in t[:9]]
        bs.Prepared("scout_sparse_attn8_merge" if merge else "scout_sparse_attn8", 0, *p[:5], a.n_slots, *p[5:], a.B, Hq, a.Hkv,
                    D, a.P, a.cap, a.k, a.scale, *[x.data_ptr() for x in cpu], O_.data_ptr(), l.data_ptr(), ws.data_ptr(),
                    ws.numel(), st.data_ptr(), bs._launch(None, inject=inject), torch.cuda.current_stream().cuda_stream)()
        torch.cuda.synchronize()
        return O_.clone(), l.clone()

    good = call(bs.INJECT_NONE)
    a.check(*good, merged=merge)
    assert int(st) == 0
    bad = call(bs.INJECT_ABANDON)
    assert int(st) == 2 and not ws[:bs._native().attn8_zero_bytes].any()
    lost = torch.isnan(bad[1])
    assert lost.any() and torch.equal(torch.isnan(bad[0]), lost[..., None].expand(-1, -1, D))
    units = lost.view(-1, a.G)
    assert torch.equal(units.all(1), units.any(1))  # all heads of a unit alike
    assert not units[torch.from_numpy(a.counts.flatten() == 0)].any()
    assert torch.equal(bad[0][~lost], good[0][~lost]) and torch.equal(bad[1][~lost], good[1][~lost])
    again = call(bs.INJECT_NONE)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    with pytest.raises(bs.ScoutError, match="INVALID_ARG"):
        call(bs.INJECT_COPY_FAIL)


def test_outputs_that_do_not_fit_raise_torch_out_of_memory():
    # no memory is filled: the process's share is set below what it holds, so that the allocator refuses
    a = Attn(54, B=256, Hkv=8, G=2, P=16, lens=[20] * 256, k=2)
    t, ws = a.device(), a.workspace()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = []
    try:
        torch.cuda.set_per_process_memory_fraction(1e-6)
        with pytest.raises(torch.OutOfMemoryError):
            while True:  # ends when the cached blocks are used up: what is left is smaller than the 2 MB output
                held.append(torch.empty((1 << 20) + 1, dtype=torch.uint8, device="cuda"))
        with pytest.raises(torch.OutOfMemoryError):
            bs.sparse_attn8(*t, ws)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
        del held
    a.check(*bs.sparse_attn8(*t, ws))


# ---------------------------------------------------------------------------
# recalled blocks
# ---------------------------------------------------------------------------
def test_a_recalled_block_is_written_as_a_sequence_of_its_own():
    """Blocks whose host copy is bf16 come back through append_kv8, each as a fresh sequence of one KV head, and their
    digests are rebuilt: the codes need not be those that were evicted, as a block that was filled piece by piece may
    have been rounded twice."""
    rng = np.random.default_rng(55)
    Hkv, P, n_slots = 2, 16, 12
    seq, grown = [20], [32]  # block 1 filled in two parts, the second with larger values
    x = bf16_values(rng, (32, Hkv, D))
    x[20:] *= 64.0
    pools = [pool8(np.zeros((n_slots, P, D), np.uint8), "e4m3") for _ in range(2)]
    sc = [torch.zeros(n_slots, device="cuda") for _ in range(2)]
    table = i32([[[0, 1], [2, 3]]])
    bs.append_kv8(x[:20].cuda(), x[:20].cuda(), table, i32(seq), 1, Hkv, P, *pools, *sc)
    bs.append_kv8(x[20:].cuda(), x[20:].cuda(), table, i32(grown), 1, Hkv, P, *pools, *sc, prev_len=i32(seq))
    dg = torch.zeros((1, Hkv, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    bs.build_digest8("minmax", pools[0], sc[0], table, i32(grown), 1, Hkv, P, dg)
    # both heads' block 1 leave slots 1 and 3 and come back into slots 9 and 5
    rows = torch.cat([x[16:32, h] for h in range(Hkv)]).view(2 * P, 1, D).cuda()
    bs.append_kv8(rows, rows, i32([[[9]], [[5]]]), i32([P, P]), 2, 1, P, *pools, *sc)
    table[0, 0, 1], table[0, 1, 1] = 9, 5
    bs.build_digest8("minmax", pools[0], sc[0], table, i32(grown), 1, Hkv, P, dg, block_list=i32([[0, 1], [1, 1]]))
    got, scale = codes_of(pools[0]), sc[0].cpu().numpy()
    for h, (was, now) in enumerate(((1, 9), (3, 5))):
        new = x[16:32, h].double().numpy()
        s = C8.block_scale(new, "e4m3")
        assert scale[now] == s and np.array_equal(got[now], C8.encode(new / s, "e4m3")) and scale[was] == s
        v = C8.decode(got[now], "e4m3") * s
        lo, hi = dg[0, h, 1].double().cpu().numpy()
        assert np.array_equal(lo, v.min(0)) and np.array_equal(hi, v.max(0))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class State:
    """Pools, tables and buffers of a batch that decodes; step() is one token for the sequences that grow."""

    def __init__(self, B, Hkv, G, P, cap, k, rows):
        self.B, self.Hkv, self.G, self.P, self.cap, self.k = B, Hkv, G, P, cap, k
        n_slots = B * Hkv * cap
        z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.prev, self.seq, self.counts, self.status = z(B), z(B), z(3), z(1)
        self.table, self.bits, self.free = z(B, Hkv, cap), z(B, Hkv, -(-cap // 32)), z(n_slots)
        self.map, self.list = z(rows, Hkv, dtype=torch.int64), z(rows * Hkv, 2)
        self.pools = [z(n_slots, P, D, dtype=torch.uint8).view(DT["e4m3"]) for _ in range(2)]
        self.plain = [z(n_slots, P, D, dtype=torch.bfloat16) for _ in range(2)]
        self.scales = [z(n_slots, dtype=torch.float32) for _ in range(2)]
        self.digest, self.K, self.V = (z(*s, dtype=torch.bfloat16) for s in ((B, Hkv, cap, 2, D), (rows, Hkv, D), (rows, Hkv, D)))
        self.q, self.O = z(B, Hkv * G, D, dtype=torch.bfloat16), z(B, Hkv * G, D, dtype=torch.bfloat16)
        self.lse, self.O_cpu = z(B, Hkv * G, dtype=torch.float32), z(B, Hkv * G, D, dtype=torch.float32)
        self.lse_cpu = torch.full_like(self.lse, -np.inf)
        self.sel = {n: z(B, Hkv, k) for n in ("topk", "res", "cpu", "delta")}
        self.sel.update({n + "_count": z(B, Hkv) for n in tuple(self.sel)})
        self.ws_t, self.ws_a = bs.score_topk_workspace(B, Hkv, cap), bs.sparse_attn8_workspace(B, Hkv * G, Hkv, P)

    def step(self, n, fresh=False):
        B, Hkv, P, st, p = self.B, self.Hkv, self.P, self.status, None if fresh else self.prev
        bs.build_tables(self.seq, self.free, self.free.numel(), B, Hkv, P, self.table, self.bits, prev_len=p, slot_map=self.map,
                        block_list=self.list, counts=self.counts, status=st)
        bs.append_kv(self.K[:n], self.V[:n], self.map[:n], Hkv, P, *self.plain, status=st)
        bs.append_kv8(self.K[:n], self.V[:n], self.table, self.seq, B, Hkv, P, *self.pools, *self.scales, prev_len=p, status=st)
        bs.build_digest8("minmax", self.pools[0], self.scales[0], self.table, self.seq, B, Hkv, P, self.digest,
                         block_list=self.list, status=st)
        bs.score_topk("minmax", self.q, self.digest, self.seq, self.bits, B, Hkv * self.G, Hkv, P, self.cap, self.k, self.ws_t,
                      out=self.sel, status=st)
        bs.sparse_attn8_merge(self.q, *self.pools, *self.scales, self.table, self.seq, self.sel["res"], self.sel["res_count"], B,
                              Hkv * self.G, Hkv, P, self.k, D ** -0.5, self.ws_a, self.O_cpu, self.lse_cpu, self.O, self.lse, st)
        self.prev.copy_(self.seq)


def test_decode_steps_captured_once_and_replayed():
    """A graph of a padded decode step (a row for every sequence, whether it grows or not), replayed as the lengths move
    on, against calls with the rows there are: tables, pools, scales, digests and outputs alike."""
    rng = np.random.default_rng(57)
    B, Hkv, G, P, cap, k = 5, 2, 4, 16, 12, 5
    seq = np.array([100, 15, 31, 1, 64])
    a, b = (State(B, Hkv, G, P, cap, k, int(seq.sum())) for _ in range(2))
    g = torch.cuda.CUDAGraph()
    free = rng.permutation(a.free.numel())
    for i in range(24):
        grow = seq if i == 0 else rng.integers(0, 2, B)
        n = int(grow.sum())
        x = [bf16_values(rng, s) for s in ((n, Hkv, D), (n, Hkv, D), (B, Hkv * G, D))]
        for s in (a, b):
            s.K[:n], s.V[:n], s.q[:] = (y.cuda() for y in x)
            s.K[n:], s.V[n:] = float("nan"), float("nan")
            s.seq += i32(grow)
            s.free[: len(free)] = i32(free)
        torch.cuda.synchronize()
        if i == 1:
            with torch.cuda.graph(g):
                a.step(B)
        g.replay() if i else a.step(n, fresh=True)
        b.step(n, fresh=i == 0)
        torch.cuda.synchronize()
        assert int(a.status) == 0 and int(b.status) == 0
        for x, y in ((getattr(a, m), getattr(b, m)) for m in ("prev", "table", "bits", "counts", "digest", "O", "lse")):
            assert torch.equal(x, y)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.pools + a.plain + a.scales, b.pools + b.plain + b.scales))
        assert torch.isfinite(a.O).all() and torch.isfinite(a.lse).all()
        free = free[int(a.counts[2]):]
