"""fp64 oracle of the block tables, the cache writes and the 8-bit paged cache (numpy, no torch, no
code shared with the library).  Bytes are carried as uint8, bf16 as its values in fp64."""
from __future__ import annotations

import math

import numpy as np

FIELDS = {"e4m3": (4, 3, 7), "e5m2": (5, 2, 15)}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def code_values(fmt: str) -> np.ndarray:
    """The value of each of the 256 codes."""
    e, m, bias = FIELDS[fmt]
    c = np.arange(256)
    ex, fr = (c >> m) & ((1 << e) - 1), (c & ((1 << m) - 1)) / float(1 << m)
    v = np.where(ex > 0, (1 + fr) * 2.0 ** (ex - bias), fr * 2.0 ** (1 - bias))
    if fmt == "e4m3":
        v[(c & 0x7F) == 0x7F] = np.nan
    else:
        top = ex == (1 << e) - 1
        v = np.where(top, np.where(fr == 0, np.inf, np.nan), v)
    return np.where(c >= 128, -v, v)


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    return code_values(fmt)[codes]


def encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest code, ties to the even one; infinities and larger values saturate, NaN is 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    v = code_values(fmt)[:128]
    v = v[np.isfinite(v)]  # ascending, code i has value v[i]
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=LARGEST[fmt], neginf=-LARGEST[fmt])), LARGEST[fmt])
    hi = np.clip(np.searchsorted(v, a), 1, len(v) - 1)
    lo = hi - 1
    dl, dh = a - v[lo], v[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = c | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, c).astype(np.uint8)


def block_scale(x: np.ndarray, fmt: str) -> float:
    """Smallest power of two >= 2^-126 whose multiple of the format's largest value covers x."""
    big = np.abs(x[np.isfinite(x)])
    big = float(big.max()) if big.size else 0.0
    e = -126
    while LARGEST[fmt] * 2.0 ** e < big:
        e += 1
    return 2.0 ** e


def spans(prev, seq, cap):
    seq = [min(max(int(n), 0), cap) for n in seq]
    prev = [0] * len(seq) if prev is None else [min(max(int(p), 0), n) for p, n in zip(prev, seq)]
    return prev, seq


def build_tables(prev, seq, free, n_slots, Hkv, P, cap, table=None, bits=None, max_tokens=None, max_list=None):
    """-> dict of table [B][Hkv][cap], bits (bool [B][Hkv][cap]), cu, slot_map, block_list, counts, status.
    table / bits: the state before (required with prev)."""
    B = len(seq)
    status = 0
    for b in range(B):
        n, p = int(seq[b]), 0 if prev is None else int(prev[b])
        status |= (4 if n > cap * P else 0) | (1 if n < 0 or p < 0 or p > max(n, 0) else 0)
    fresh = prev is None
    prev, seq = spans(prev, seq, cap * P)
    table = np.full((B, Hkv, cap), -1, np.int64) if fresh else np.array(table, np.int64)
    bits = np.zeros((B, Hkv, cap), bool) if fresh else np.array(bits, bool)
    taken = 0
    touched = []
    for b in range(B):
        for h in range(Hkv):
            for j in range(-(-prev[b] // P), -(-seq[b] // P)):
                s = -1
                if taken >= len(free):
                    status |= 4
                elif 0 <= free[taken] < n_slots:
                    s = int(free[taken])
                else:
                    status |= 1
                taken += 1
                table[b, h, j] = s
                bits[b, h, j] = s >= 0
            if seq[b] > prev[b]:
                touched += [(b * Hkv + h, j) for j in range(prev[b] // P, -(-seq[b] // P))]
    cu = np.concatenate([[0], np.cumsum([n - p for n, p in zip(seq, prev)])])
    rows = []
    for b in range(B):
        for t in range(prev[b], seq[b]):
            s = table[b, :, t // P]
            ok = (s >= 0) & (s < n_slots)
            if t // P < -(-prev[b] // P) and not ok.all():
                status |= 1
            rows.append(np.where(ok, s * P + t % P, -1))
    n = len(rows)
    max_tokens = n if max_tokens is None else max_tokens
    max_list = len(touched) if max_list is None else max_list
    slot_map = np.full((max_tokens, Hkv), -1, np.int64)
    lst = np.full((max_list, 2), -1, np.int64)
    m = min(n, max_tokens)
    if m:
        slot_map[:m] = np.array(rows)[:m]
    m = min(len(touched), max_list)
    if m:
        lst[:m] = np.array(touched)[:m]
    if n > max_tokens or len(touched) > max_list:
        status |= 4
    return {"table": table, "bits": bits, "cu": cu, "slot_map": slot_map, "block_list": lst,
            "counts": np.array([n, len(touched), taken]), "status": status}


def append8(x, prev, seq, table, codes, scales, fmt, P):
    """One of K and V: x fp64 [n_tokens][Hkv][D]; codes uint8 [n_slots][P][D], scales [n_slots]
    (fp64 of fp32 values) are updated in copies -> (codes, scales).  Scales must be powers of two."""
    codes, scales = codes.copy(), scales.copy()
    cap = table.shape[-1]
    prev, seq = spans(prev, seq, cap * P)
    row = 0
    for b, (p, n) in enumerate(zip(prev, seq)):
        for j in range(p // P, -(-n // P) if n > p else p // P):
            lo, hi = max(p, j * P), min(n, (j + 1) * P)
            for h in range(x.shape[1]):
                s = int(table[b, h, j])
                if s < 0 or s >= codes.shape[0]:
                    continue
                new = x[row + lo - p: row + hi - p, h]
                scale = block_scale(new, fmt)
                had = lo - j * P
                if had > 0:
                    scale = max(scale, float(scales[s]))
                    if scale > scales[s]:
                        codes[s, :had] = encode(decode(codes[s, :had], fmt) * (float(scales[s]) / scale), fmt)
                codes[s, had:hi - j * P] = encode(new / scale, fmt)
                scales[s] = scale
        row += n - p
    return codes, scales


def digest8(kind, codes, scales, table, seq, fmt, P, digest, units=None):
    """digest fp64 [B][Hkv][cap][2][D] or [..][D], updated in a copy: exact minima and maxima, or means."""
    out = np.array(digest, np.float64)
    B, Hkv, cap = table.shape
    for b in range(B):
        for h in range(Hkv):
            for j in range(cap):
                if units is not None and (b * Hkv + h, j) not in units:
                    continue
                n = min(P, int(seq[b]) - j * P)
                s = int(table[b, h, j])
                if n <= 0 or s < 0 or s >= codes.shape[0]:
                    continue
                x = decode(codes[s, :n], fmt) * float(scales[s])
                if kind == "minmax":
                    out[b, h, j, 0], out[b, h, j, 1] = np.nanmin(x, 0), np.nanmax(x, 0)
                else:
                    out[b, h, j] = x.mean(0)
    return out


def attn8(q, k_codes, v_codes, ks, vs, fmt, table, seq, lists, counts, P, scale):
    """q fp64 [B][Hq][D] -> O, lse, and the bounds' ingredients: sum p|v| [B][Hq][D], largest
    scale * sum |q k| and tokens of each head."""
    B, Hq, D = q.shape
    Hkv, cap = table.shape[1:]
    G = Hq // Hkv
    O, mag = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, big, cnt = np.full((B, Hq), -np.inf), np.zeros((B, Hq)), np.zeros((B, Hq), int)
    for b in range(B):
        for h in range(Hkv):
            K, V = [], []
            for j in lists[b, h, : max(0, min(int(counts[b, h]), lists.shape[-1]))]:
                n = min(P, int(seq[b]) - int(j) * P) if 0 <= j < cap else 0
                s = int(table[b, h, j]) if n > 0 else -1
                if s < 0 or s >= k_codes.shape[0]:
                    continue
                K.append(decode(k_codes[s, :n], fmt) * float(ks[s]))
                V.append(decode(v_codes[s, :n], fmt) * float(vs[s]))
            if not K:
                continue
            K, V = np.concatenate(K), np.concatenate(V)
            for hq in range(h * G, (h + 1) * G):
                s = K @ q[b, hq] * scale
                m = s.max()
                p = np.exp(s - m)
                lse[b, hq] = m + math.log(p.sum())
                p /= p.sum()
                O[b, hq], mag[b, hq] = p @ V, p @ np.abs(V)
                big[b, hq] = (np.abs(K) @ np.abs(q[b, hq])).max() * scale
                cnt[b, hq] = len(K)
    return O, lse, mag, big, cnt


def merge(O, lse, O_cpu, lse_cpu):
    m = np.maximum(lse, lse_cpu)
    safe = np.where(np.isfinite(m), m, 0.0)
    a, c = np.exp(lse - safe), np.exp(lse_cpu - safe)
    t = a + c
    w = np.where(t > 0, t, 1.0)
    with np.errstate(divide="ignore"):
        return (a[..., None] * O + c[..., None] * O_cpu) / w[..., None], np.where(t > 0, safe + np.log(t), -np.inf)
