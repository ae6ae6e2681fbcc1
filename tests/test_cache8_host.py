"""Host side of the block tables, cache writes and 8-bit cache: refusals before any launch, and the
oracle of the codes (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from oracle import cache8_oracle as C8
from _parity import ensure_built

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    ensure_built()
    return bs.lib()


def call(fn, args, **change):
    names = list(args)
    v = dict(args, **{k: x for k, x in change.items()})
    assert set(v) == set(names)
    return fn(*[v[n] for n in names])


TABLES = dict(prev=None, seq=F, free=F, n_free=10, n_slots=10, B=2, Hkv=2, P=32, cap=8, table=F, bits=F, cu=F, map=F,
              max_tokens=64, list=F, max_list=8, counts=F, status=None, stream=None)
APPEND = dict(K=F, ld_k=256, V=F, ld_v=256, map=F, n=4, Hkv=2, D=128, P=32, Kp=F, Vp=F, n_slots=10, status=None,
              stream=None)
APPEND8 = dict(fmt=0, K=F, ld_k=256, V=F, ld_v=256, n=4, prev=None, seq=F, table=F, B=2, Hkv=2, D=128, P=32, cap=8, Kp=F,
               Vp=F, Ks=F, Vs=F, n_slots=10, status=None, stream=None)
DIGEST8 = dict(kind=0, fmt=0, Kp=F, Ks=F, n_slots=10, table=F, seq=F, B=2, Hkv=2, D=128, P=32, cap=8, list=None, n_list=0,
               digest=F, status=None, stream=None)
ATTN = dict(fmt=0, q=F, Kp=F, Vp=F, Ks=F, Vs=F, n_slots=10, table=F, seq=F, list=F, count=F, B=2, Hq=8, Hkv=2, D=128,
            P=32, cap=8, k=4, scale=0.1, O=F, lse=F, ws=F, wsb=1 << 30, status=None, launch=None, stream=None)
MERGE = dict(fmt=0, q=F, Kp=F, Vp=F, Ks=F, Vs=F, n_slots=10, table=F, seq=F, list=F, count=F, B=2, Hq=8, Hkv=2, D=128,
             P=32, cap=8, k=4, scale=0.1, Oc=F, lc=F, O=F, lse=F, ws=F, wsb=1 << 30, status=None, launch=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(seq=None), INVALID), (dict(table=None), INVALID), (dict(bits=None), INVALID), (dict(B=0), INVALID),
    (dict(Hkv=-1), INVALID), (dict(cap=0), INVALID), (dict(n_slots=0), INVALID), (dict(n_free=-1), INVALID),
    (dict(max_tokens=-1), INVALID), (dict(max_list=-1), INVALID), (dict(P=48), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(cap=8193), UNSUPPORTED), (dict(n_slots=1 << 31), UNSUPPORTED),
    (dict(B=4096, cap=8192, P=64), UNSUPPORTED), (dict(B=4096, cap=8192, Hkv=64, P=16), UNSUPPORTED),
    (dict(list=ctypes.c_void_p(4100)), UNSUPPORTED), (dict(map=ctypes.c_void_p(4100)), UNSUPPORTED)])
def test_build_tables_refusals(L, change, rc):
    assert call(L.scout_build_tables, TABLES, **change) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(map=None), INVALID), (dict(Kp=None), INVALID),
    (dict(Vp=None), INVALID), (dict(n=-1), INVALID), (dict(Hkv=0), INVALID), (dict(n_slots=0), INVALID),
    (dict(ld_k=255), INVALID), (dict(ld_v=248), INVALID), (dict(ld_k=260), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(P=8), UNSUPPORTED), (dict(K=ctypes.c_void_p(4104)), UNSUPPORTED), (dict(Vp=ODD), UNSUPPORTED),
    (dict(map=ctypes.c_void_p(4100)), UNSUPPORTED), (dict(n_slots=1 << 31), UNSUPPORTED), (dict(n=0), OK)])
def test_append_refusals(L, change, rc):
    assert call(L.scout_append_kv, APPEND, **change) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID),
    (dict(seq=None), INVALID), (dict(table=None), INVALID), (dict(Kp=None), INVALID), (dict(Vp=None), INVALID),
    (dict(Ks=None), INVALID), (dict(Vs=None), INVALID), (dict(n=-1), INVALID), (dict(B=0), INVALID),
    (dict(ld_k=128), INVALID), (dict(ld_v=257), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(P=0), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(cap=8193), UNSUPPORTED), (dict(B=4096, cap=8192, P=64), UNSUPPORTED),
    (dict(Kp=ODD), UNSUPPORTED), (dict(V=ctypes.c_void_p(4104)), UNSUPPORTED), (dict(n_slots=1 << 31), UNSUPPORTED),
    (dict(B=4096, cap=8192, P=16, Hkv=64, ld_k=8192, ld_v=8192), UNSUPPORTED), (dict(n=0), OK)])
def test_append8_refusals(L, change, rc):
    assert call(L.scout_append_kv8, APPEND8, **change) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(kind=2), INVALID), (dict(fmt=3), INVALID), (dict(Kp=None), INVALID), (dict(Ks=None), INVALID),
    (dict(table=None), INVALID), (dict(seq=None), INVALID), (dict(digest=None), INVALID), (dict(B=0), INVALID),
    (dict(n_list=-1, list=F), INVALID), (dict(D=64), UNSUPPORTED), (dict(P=128), UNSUPPORTED),
    (dict(Kp=ODD), UNSUPPORTED), (dict(digest=ctypes.c_void_p(4104)), UNSUPPORTED), (dict(list=F, n_list=0), OK),
    (dict(B=1 << 20, cap=1 << 12), UNSUPPORTED), (dict(n_slots=1 << 31), UNSUPPORTED)])
def test_digest8_refusals(L, change, rc):
    assert call(L.scout_build_digest8, DIGEST8, **change) == rc


COMMON = [
    (dict(fmt=2), INVALID), (dict(q=None), INVALID), (dict(Kp=None), INVALID), (dict(Vp=None), INVALID),
    (dict(Ks=None), INVALID), (dict(Vs=None), INVALID), (dict(table=None), INVALID), (dict(seq=None), INVALID),
    (dict(list=None), INVALID), (dict(count=None), INVALID), (dict(O=None), INVALID), (dict(B=0), INVALID),
    (dict(Hq=7), INVALID), (dict(k=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(Hq=18), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(P=24), UNSUPPORTED), (dict(B=2049), UNSUPPORTED),
    (dict(k=(1 << 26) + 1), UNSUPPORTED), (dict(n_slots=1 << 27), UNSUPPORTED), (dict(Kp=ODD), UNSUPPORTED),
    (dict(q=ctypes.c_void_p(4100)), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(wsb=1024), WORKSPACE),
    (dict(ws=ctypes.c_void_p(4104)), UNSUPPORTED), (dict(launch=ctypes.pointer(bs.Launch(-1))), INVALID)]


@pytest.mark.parametrize("change,rc", COMMON + [(dict(lse=None), INVALID), (dict(O=ctypes.c_void_p(4100)), UNSUPPORTED)])
def test_attn8_refusals(L, change, rc):
    assert call(L.scout_sparse_attn8, ATTN, **change) == rc


@pytest.mark.parametrize("change,rc", COMMON + [
    (dict(Oc=None), INVALID), (dict(lc=None), INVALID), (dict(O=ctypes.c_void_p(4098)), UNSUPPORTED),
    (dict(Oc=ctypes.c_void_p(4100)), UNSUPPORTED)])
def test_attn8_merge_refusals(L, change, rc):
    assert call(L.scout_sparse_attn8_merge, MERGE, **change) == rc


def test_workspace_bytes(L):
    assert L.scout_sparse_attn8_workspace_bytes(40, 40, 8, 128, 32) >= 4 * 320
    assert L.scout_sparse_attn8_workspace_bytes(0, 40, 8, 128, 32) == 0


def test_binding_refuses_host_and_mismatched_tensors(L):
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(bs.ScoutError, match="CUDA tensor"):
        bs.build_tables(t, None, 4, 4, 1, 32, t, t)
    with pytest.raises(bs.ScoutError, match="CUDA tensor"):
        bs.append_kv(t, t, t, 1, 32, t, t)
    x = torch.zeros((2, 32, 128), dtype=torch.float8_e4m3fn)
    with pytest.raises(bs.ScoutError, match="CUDA tensor"):
        bs.build_digest8("minmax", x, t, t, t, 1, 1, 32, t)
    f = torch.zeros(2)  # scales
    n = torch.ones(1, dtype=torch.int32)

    def write(rows=torch.zeros((1, 2, 128), dtype=torch.bfloat16), K=x, V=x, table=torch.zeros((1, 2, 1), dtype=torch.int32),
              scale=f, **kw):
        bs.append_kv8(rows, rows, table, n, 1, 2, 32, K, V, scale, scale, **kw)

    with pytest.raises(bs.ScoutError, match="float8"):
        write(K=x.view(torch.uint8))
    with pytest.raises(bs.ScoutError, match="alike"):
        write(V=x[:1])
    with pytest.raises(bs.ScoutError, match="alike"):
        write(V=x.view(torch.float8_e5m2))
    with pytest.raises(bs.ScoutError, match="elements"):
        write(scale=f[:1])
    with pytest.raises(bs.ScoutError, match="elements, got 2 Double"):
        write(scale=f.double())
    with pytest.raises(bs.ScoutError, match="strided"):
        write(scale=torch.zeros(4)[::2])
    with pytest.raises(bs.ScoutError, match="CUDA tensor, got list"):
        write(scale=[1.0, 1.0])
    with pytest.raises(bs.ScoutError, match="heads of a token"):
        write(torch.zeros((3, 128, 2), dtype=torch.bfloat16).transpose(1, 2))
    with pytest.raises(bs.ScoutError, match=r"\[n_tokens\]\[2\]\[128\]"):
        write(torch.zeros((3, 3, 128), dtype=torch.bfloat16))
    with pytest.raises(bs.ScoutError, match="K_pool must be a CUDA tensor on"):  # everything else fits
        write()
    rows = torch.zeros((5, 3 * 128), dtype=torch.bfloat16)[:, 128:].view(5, 2, 128)  # heads contiguous, tokens strided
    with pytest.raises(bs.ScoutError, match="K_pool must be a CUDA tensor on"):
        write(rows)


def test_binding_refuses_sizes_that_wrap(L):
    """Products of sizes that pass 64 bits, and sizes that pass a C int, fit no tensor."""
    t = torch.zeros(0, dtype=torch.int32)
    with pytest.raises(bs.ScoutError, match="elements"):
        bs.build_tables(t, None, 4, 1 << 30, 1 << 30, 32, t.view(0, 16), t)  # 2^64 elements, not 0
    with pytest.raises(bs.ScoutError, match="32-bit"):
        bs.build_tables(t, None, 4, 1 << 32, 1, 32, t, t)
    wide = torch.zeros((0, 32, (1 << 32) + 128), dtype=torch.uint8)  # 128 in 32 bits
    with pytest.raises(bs.ScoutError, match="32-bit"):
        bs.build_digest8("mean", wide.view(torch.float8_e5m2), t, t, t, 0, 1, 32, t)
    with pytest.raises(bs.ScoutError, match=r"\[n_slots\]"):
        bs.append_kv(t, t, t, 1, 32, wide, wide)
    with pytest.raises(TypeError):
        bs.build_tables(t, None, 4, 1.5, 1, 32, t, t)


def test_binding_attention_arguments(L):
    """Host tensors that fit in everything but their place: each argument's own refusal comes first."""
    B, Hq, Hkv, P, k, D, slots, cap = 2, 4, 2, 32, 3, 128, 5, 4
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros((slots, P, D), dtype=torch.float8_e5m2)
    good = [torch.zeros((B, Hq, D), dtype=torch.bfloat16), pool, pool.clone(), torch.zeros(slots), torch.zeros(slots),
            i(B, Hkv, cap), i(B), i(B, Hkv, k), i(B, Hkv)]
    names = ["q", "", "", "K_scale", "V_scale", "page_table", "seq_len", "res_list", "res_count"]
    ws = torch.zeros(1 << 18, dtype=torch.uint8)
    part = torch.zeros((B, Hq, D)), torch.zeros((B, Hq))

    def run(t=good, ws=ws, part=None, **kw):
        a = (*t, B, Hq, Hkv, P, k, D ** -0.5, ws)
        return bs.sparse_attn8(*a, **kw) if part is None else bs.sparse_attn8_merge(*a, *part, **kw)

    for p in (None, part):
        with pytest.raises(bs.ScoutError, match="q must be a CUDA tensor on"):
            run(part=p)
        for at, name in enumerate(names):
            with pytest.raises(bs.ScoutError, match=f"^{name}.*(elements|alike)"):
                run([*good[:at], good[at][:1], *good[at + 1:]], part=p)
        with pytest.raises(bs.ScoutError, match="workspace"):
            run(ws=ws.int(), part=p)
        with pytest.raises(bs.ScoutError, match="^O must be"):
            run(part=p, **{"O" if p is None else "O_out": part[0][:1]})
        with pytest.raises(bs.ScoutError, match="^lse must be"):
            run(part=p, **{"lse" if p is None else "lse_out": part[1][:1]})
        with pytest.raises(bs.ScoutError, match="status must be"):
            run(part=p, status=i(2))
    for at, name in enumerate(("O_cpu", "lse_cpu")):
        with pytest.raises(bs.ScoutError, match=name):
            run(part=[part[j][:1] if j == at else part[j] for j in (0, 1)])
        with pytest.raises(bs.ScoutError, match=name):
            run(part=[None if j == at else part[j] for j in (0, 1)])


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_oracle_codes_match_the_formats(fmt, dtype):
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(dtype).to(torch.float64).numpy()
    assert np.array_equal(C8.decode(codes.numpy(), fmt), ref, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * np.exp2(rng.integers(-20, 9, 4000)), ref[np.isfinite(ref)]])
    x = np.clip(x, -C8.LARGEST[fmt], C8.LARGEST[fmt]).astype(np.float32)
    want = torch.from_numpy(x).to(dtype).view(torch.uint8).numpy()
    assert np.array_equal(C8.encode(x, fmt), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_oracle_scale_covers_the_block(fmt):
    top = C8.LARGEST[fmt]
    for x in (top, np.nextafter(top, 1e9), 3.0, 2.0 ** -140, 0.0, 3.3e38):
        s = C8.block_scale(np.array([x, -x / 3, np.inf, np.nan]), fmt)
        assert np.log2(s) == round(np.log2(s)) and x <= top * s
        assert s == 2.0 ** -126 or x > top * s / 2
