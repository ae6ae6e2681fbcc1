"""fp64 oracle of a layer's row operators: rotary positions, residual stream and norms, the cache read
back (numpy, no torch, no code shared with the library).  bf16 is carried as its values in fp64."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def frequencies(base, rot, scaling=None):
    """([rot / 2] angles a position step, amplitude), a pair at a time."""
    s = scaling or {}
    kind, k = s.get("kind"), s.get("factor")
    if kind == "ntk":
        base = base * k ** (rot / (rot - 2.0))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if kind == "linear":
            f = f / k
        elif kind == "rotations":
            lo, hi = s.get("low", 1.0), s.get("high", 4.0)
            made = s["original"] * f / (2 * math.pi)
            keep = min(max((made - lo) / (hi - lo), 0.0), 1.0)
            f = f * keep + (1 - keep) * f / k
        elif kind == "index":
            pair = lambda n: rot * math.log(s["original"] / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
            a = max(math.floor(pair(s.get("high", 32.0))), 0)
            b = min(math.ceil(pair(s.get("low", 1.0))), rot - 1)
            slow = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f * (1 - slow) + slow * f / k
        elif kind == "divisors":
            f = f / s["divisors"][i]
        out.append(f)
    amp = s.get("amplitude") or (0.1 * math.log(k) + 1.0 if kind == "index" and k > 1 else 1.0)
    return np.array(out), amp


def angles(pos, turns):
    """[n][pairs] angles in [-pi, pi) of integer positions, from turns as integers of 2^-64 (exact products)."""
    out = np.empty((len(pos), len(turns)))
    for i, p in enumerate(pos):
        for j, t in enumerate(turns):
            x = (int(p) * int(t)) % (1 << 64)
            out[i, j] = 2 * math.pi * float(Fraction(x - (1 << 64) if x >= 1 << 63 else x, 1 << 64))
    return out


def rms(x, w, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def pairs(x, rot, layout):
    """(first, second) of each pair of the last axis."""
    return (x[..., : rot // 2], x[..., rot // 2: rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])


def rotate(x, angle, rot, layout, amp, norm=None, eps=0.0):
    """x [n][heads][D], angle [n][rot / 2] -> (turned heads, the length of each channel's pair: what errors scale with)."""
    if norm is not None:
        x = rms(x, norm, eps)
    y, size = x.copy(), np.abs(x)
    a, b = pairs(x, rot, layout)
    c, s = np.cos(angle)[:, None] * amp, np.sin(angle)[:, None] * amp
    for view, value in zip(pairs(y, rot, layout), (a * c - b * s, a * s + b * c)):
        view[...] = value
    for view in pairs(size, rot, layout):
        view[...] = amp * np.hypot(a, b)
    return y, size


def norm(x, kind, w, b, eps):
    mean = x.mean(-1, keepdims=True) if kind == "layer" else 0.0
    z = (x - mean) / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    return z * w + (0.0 if b is None else b), z


def read(pool, table, seq, P, out, blocks=None):
    """pool [n_slots][P][D] values into a copy of out [B][Hkv][T][D]; blocks: (unit, block) pairs, None: all that have a slot."""
    out = out.copy()
    B, Hkv, cap = table.shape
    blocks = [(u, j) for u in range(B * Hkv) for j in range(cap)] if blocks is None else blocks
    for u, j in blocks:
        b, h = divmod(u, Hkv)
        for r in range(P):
            t = j * P + r
            if t < min(seq[b], out.shape[2]) and 0 <= table[b, h, j] < len(pool):
                out[b, h, t] = pool[table[b, h, j], r]
    return out
