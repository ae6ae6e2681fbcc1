"""A layer's row operators around the paged cache: what is measured, and their plain forms.

Six kinds of cases, each reached through ``block_sparse_kv_pred_gb300``:

* ``addnorm``  add_norm: a block's output, optionally normalised, gated and scaled, added to the residual
               stream, and the stream normalised for this layer and for the next layer's query prediction.
* ``rotate``   rotate: heads normalised and turned by their tokens' positions (rotary positions).
* ``append``   append_rotated_kv: the same for a step's keys and queries, the keys and values on their way
               into a bf16 paged cache.
* ``append8``  append_rotated_kv8: the same into an 8-bit paged cache, quantised as it is written.
* ``predict``  predict_q_rotated: the predicted query's projection with its heads normalised and turned.
* ``read``     read_kv / read_kv8: blocks of a paged cache back as bf16 rows in the order of their tokens.

``run`` computes them with elementary torch operations, or with the library where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

D = 128
EPS = 1e-6
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
#: pool entries that no operator may touch hold this byte (a finite code in both formats)
FILL = 0x31


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the Qwen3-14B-shaped batch: the stream normalised for this layer and for the prediction
        {"name": "addnorm_decode_b40", "op": "addnorm", "M": 40, "N": 5120, "kind": "rms", "post": False, "gate": "none",
         "alpha": 1.0, "h": "bf16", "ahead": True, "pad": 0},
        # prompts of the Qwen3-8B-shaped batch, a stream in fp32, norms before and after the block, a gate for each channel
        {"name": "addnorm_prompt_b8_16k", "op": "addnorm", "M": 131072, "N": 4096, "kind": "rms", "post": True,
         "gate": "vector", "alpha": 0.5, "h": "fp32", "ahead": False, "pad": 0},
        # the queries of one decode step of the Qwen3-8B-shaped batch: latency
        {"name": "rotate_decode_b8", "op": "rotate", "n": 8, "heads": 32, "norm": True, "layout": "half", "rot": 128,
         "base": 1e6, "scaling": "none", "top": 16384, "pad": 0},
        # a chunk of a long prompt, half of each head turned, in neighbouring pairs, positions scaled for a long context
        {"name": "rotate_chunk_9k_part", "op": "rotate", "n": 9001, "heads": 12, "norm": False, "layout": "interleaved",
         "rot": 64, "base": 1e4, "scaling": "index", "top": 131072, "pad": 256},
        # one decode step: each sequence's query, and its key and value into the cache
        {"name": "append_decode_b40", "op": "append", "B": 40, "Hq": 40, "Hkv": 8, "T": 32768, "P": 32, "new": 1,
         "ragged": True, "norm": True, "layout": "half", "rot": 128, "base": 1e6, "scaling": "none"},
        # prompts, queries, keys and values inside a fused projection's output
        {"name": "append_prompt_b8_16k", "op": "append", "B": 8, "Hq": 32, "Hkv": 8, "T": 16384, "P": 32, "new": 0,
         "ragged": True, "norm": True, "layout": "half", "rot": 128, "base": 1e6, "scaling": "none"},
        # the same two into an 8-bit cache
        {"name": "append8_decode_b40", "op": "append8", "fmt": "e4m3", "B": 40, "Hq": 40, "Hkv": 8, "T": 2048, "P": 32,
         "new": 1, "ragged": True, "norm": True, "layout": "half", "rot": 128, "base": 1e6, "scaling": "none"},
        {"name": "append8_prompt_b8_16k", "op": "append8", "fmt": "e4m3", "B": 8, "Hq": 32, "Hkv": 8, "T": 16384, "P": 32,
         "new": 0, "ragged": True, "norm": True, "layout": "half", "rot": 128, "base": 1e6, "scaling": "none"},
        # the predicted queries of the two batches
        {"name": "predict_b8_4096", "op": "predict", "M": 8, "Hq": 32, "K": 4096, "norm": True, "layout": "half",
         "rot": 128, "base": 1e6, "scaling": "none", "top": 16384},
        {"name": "predict_b40_5120", "op": "predict", "M": 40, "Hq": 40, "K": 5120, "norm": True, "layout": "half",
         "rot": 128, "base": 1e6, "scaling": "none", "top": 32768},
        # a decode step's touched blocks, for the copy of the cache that the CPU side reads
        {"name": "read_touched_b40", "op": "read", "fmt": "bf16", "B": 40, "Hkv": 8, "T": 2048, "P": 32, "ragged": True,
         "list": 320, "order": "blocks"},
        # whole prompts out of an 8-bit cache
        {"name": "read8_prompt_b8_16k", "op": "read", "fmt": "e4m3", "B": 8, "Hkv": 8, "T": 16384, "P": 32, "ragged": True,
         "list": 0, "order": "blocks"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rope(rng, c):
    c["layout"] = rng.choice(["half", "interleaved"])
    c["rot"] = rng.choice([128, 128, 16 * rng.randint(1, 8)])
    c["base"] = rng.choice([1e4, 5e5, 1e6])
    c["scaling"] = rng.choice(["none", "none", "linear", "ntk", "rotations", "index"])
    c["norm"] = rng.random() < 0.5


def draw(rng):
    op = rng.choice(["addnorm", "rotate", "append", "append8", "predict", "read"])
    c = {"op": op}
    if op == "addnorm":
        c["N"] = 8 * _log(rng, 16, 1024)
        c["M"] = _log(rng, 1, min(131072, 131072 * 4096 // (2 * c["N"])))
        c["kind"] = rng.choice(["rms", "rms", "layer"])
        c["post"], c["ahead"] = rng.random() < 0.4, rng.random() < 0.4
        c["gate"] = rng.choice(["none", "none", "vector", "rows"])
        c["alpha"], c["h"] = rng.choice([1.0, 0.5, round(rng.uniform(0.1, 2.0), 3)]), rng.choice(["bf16", "fp32"])
        c["pad"] = rng.choice([0, 0, 8 * rng.randint(1, 40)])
    elif op == "rotate":
        _draw_rope(rng, c)
        c["n"], c["heads"] = _log(rng, 1, 32768), rng.randint(1, 64)
        c["top"], c["pad"] = _log(rng, 64, 1 << 20), rng.choice([0, 8 * rng.randint(1, 40)])
    elif op in ("append", "append8"):
        _draw_rope(rng, c)
        if op == "append8":
            c["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        c["P"], c["B"], c["Hkv"] = rng.choice([16, 32, 64]), _log(rng, 1, 40), rng.choice([1, 2, 4, 5, 8])
        c["Hq"] = c["Hkv"] * rng.randint(0, 4)
        c["ragged"] = rng.random() < 0.7
        c["T"] = _log(rng, 1, min(32768, 8 * 8 * 16384 // (2 * c["B"] * c["Hkv"])))
        # 0: whole prompts; otherwise at most so many new tokens for each sequence (a decode step, a chunk)
        c["new"] = rng.choice([0, 1, 1, _log(rng, 1, c["T"])])
    elif op == "predict":
        _draw_rope(rng, c)
        c["M"], c["Hq"], c["K"] = _log(rng, 1, 256), rng.randint(1, 40), 64 * _log(rng, 1, 80)
        c["top"] = _log(rng, 64, 1 << 20)
    else:
        c["fmt"] = rng.choice(["bf16", "e4m3", "e4m3", "e5m2"])
        c["P"], c["B"], c["Hkv"] = rng.choice([16, 32, 64]), _log(rng, 1, 40), rng.choice([1, 2, 4, 8])
        c["ragged"], c["order"] = rng.random() < 0.7, rng.choice(["blocks", "tokens"])
        c["T"] = _log(rng, 1, min(32768, 8 * 8 * 16384 // (2 * c["B"] * c["Hkv"])))
        c["list"] = rng.choice([0, _log(rng, 1, 2000)])
    return c


def _lens(case):
    """Sequence lengths: all T, or spread over 1..T."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, int(T * (((b + 1) * 0.6180339887498949) % 1.0))) for b in range(B)]


def _prev(case):
    """Lengths before the new tokens: 0 (whole prompts), or up to `new` tokens fewer."""
    lens, new = _lens(case), case["new"]
    if new == 0:
        return [0] * len(lens)
    return [max(0, n - (new if b % 3 != 2 or new == 1 else 1 + new // 2)) for b, n in enumerate(lens)]


#: the original length and the factor of the cases whose positions are scaled
ORIGINAL, FACTOR = 32768, 4.0


def _frequencies(case):
    """(angle of a position step of each pair in fp64, amplitude) of the case's rotary positions."""
    rot, base, scaling = case["rot"], case["base"], case["scaling"]
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":  # a longer base: the slowest pair's step falls by the factor
        base = base * FACTOR ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / FACTOR
    elif scaling == "rotations":  # slowed by the turns that a pair makes over the original length: 1 or fewer, 4 or more
        keep = np.clip((ORIGINAL * f / (2 * np.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = keep * f + (1 - keep) * f / FACTOR
    elif scaling == "index":  # the same by the index of the pair, from that with 32 turns to that with one
        at = lambda turns: rot * np.log(ORIGINAL / (2 * np.pi * turns)) / (2 * np.log(base))  # noqa: E731
        lo, hi = max(np.floor(at(32.0)), 0.0), min(np.ceil(at(1.0)), rot - 1.0)
        slow = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        f = (1 - slow) * f + slow * f / FACTOR
        return f, 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _library_rope(case):
    import block_sparse_kv_pred_gb300 as bs

    s = case["scaling"]
    scaling = {"none": None, "linear": {"kind": "linear", "factor": FACTOR}, "ntk": {"kind": "ntk", "factor": FACTOR},
               "rotations": {"kind": "rotations", "factor": FACTOR, "original": ORIGINAL, "low": 1.0, "high": 4.0},
               "index": {"kind": "index", "factor": FACTOR, "original": ORIGINAL, "low": 1.0, "high": 32.0}}[s]
    return bs.rope(case["base"], case["rot"], layout=case["layout"], scaling=scaling)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _weight(g, n):
    """A norm's learned weight: near one."""
    return (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)


def _rows(g, n, width, pad, gain=False):
    """bf16 rows whose stride is `pad` elements more than their width; `gain`: a few channels of each head larger."""
    x = _bf16(g, n, width + pad)[:, :width]
    if gain:
        x.view(n, width // D, D)[..., torch.randperm(D, generator=g, device="cuda")[:4]] *= 6.0
    return x


def _positions(g, n, top):
    """Positions of n tokens of a batch: neighbours of a chunk, or sequences of any length; the last of them padding."""
    if n > 256:
        p = torch.arange(n, device="cuda") + max(0, top - n)
    else:
        p = torch.randint(0, top, (n,), generator=g, device="cuda")
    if n > 2:
        p[n - max(1, n // 100):] = -1
    return p.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op != "addnorm" and op != "read":
        f, st["amp"] = _frequencies(case)
        st["freq"] = torch.tensor(f, device="cuda")
        st["qw"] = _weight(g, D) if case["norm"] else None
        st["kw"] = _weight(g, D) if case["norm"] else None
    if op == "addnorm":
        M, N = case["M"], case["N"]
        st["Y"] = _rows(g, M, N, case["pad"])
        wide = torch.bfloat16 if case["h"] == "bf16" else torch.float32
        st["H"] = torch.randn((M, N + case["pad"]), generator=g, device="cuda", dtype=wide)[:, :N]
        st["H"] *= 3.0
        st["H_out"] = torch.empty((M, N + case["pad"]), device="cuda", dtype=wide)[:, :N]
        bias = (lambda: _bf16(g, N)) if case["kind"] == "layer" else (lambda: None)
        st["w"], st["b"], st["X"] = _weight(g, N), bias(), torch.empty((M, N), device="cuda", dtype=torch.bfloat16)
        st["w_post"], st["b_post"] = (_weight(g, N), bias()) if case["post"] else (None, None)
        st["gate"] = None if case["gate"] == "none" else _bf16(g, N) if case["gate"] == "vector" else _bf16(g, M, N)
        if case["ahead"]:
            st["w_ahead"], st["b_ahead"], st["X_ahead"] = _weight(g, N), bias(), torch.empty_like(st["X"])
        return st
    if op == "rotate":
        n, heads = case["n"], case["heads"]
        st["x"] = _rows(g, n, heads * D, case["pad"], gain=True).unflatten(1, (heads, D))
        st["pos"] = _positions(g, n, case["top"])
        st["out"] = torch.full((n, heads, D), 0.5, dtype=torch.bfloat16, device="cuda")
        return st
    if op == "predict":
        M, N, K = case["M"], case["Hq"] * D, case["K"]
        st["X"] = _bf16(g, M, K)
        st["W"] = _bf16(g, N, K)
        st["W"] *= 0.02
        st["pos"] = torch.randint(0, case["top"], (M,), generator=g, device="cuda").to(torch.int32)
        return st

    B, Hkv, P = case["B"], case["Hkv"], case["P"]
    lens = _lens(case)
    nblk = [-(-n // P) for n in lens]
    cap = max(nblk) + (1 if case["ragged"] else 0)
    n_slots = sum(nblk) * Hkv + 5
    st |= {"B": B, "Hkv": Hkv, "P": P, "cap": cap, "seq_len": _i32(lens), "n_slots": n_slots}
    table = torch.full((B, Hkv, cap), -1, dtype=torch.int32, device="cuda")
    valid = (torch.arange(cap, device="cuda") < _i32(nblk)[:, None])[:, None, :].expand(B, Hkv, cap)
    table[valid] = torch.randperm(n_slots, generator=g, device="cuda").to(torch.int32)[: sum(nblk) * Hkv]
    st["table"] = table
    fp8 = case.get("fmt", "bf16") != "bf16"
    if op == "read":
        for x in "KV":
            if fp8:
                st[x + "_pool"] = (_bf16(g, n_slots, P, D) * 60.0).float().clamp_(-FMAX[case["fmt"]], FMAX[case["fmt"]]).to(FP8[case["fmt"]])
                st[x + "_scale"] = torch.exp2(torch.randint(-8, -4, (n_slots,), generator=g, device="cuda").float())
            else:
                st[x + "_pool"] = _bf16(g, n_slots, P, D)
        shape = (B, Hkv, cap * P, D) if case["order"] == "blocks" else (B, cap * P, Hkv, D)
        for x in "KV":
            out = torch.full(shape, 0.5, dtype=torch.bfloat16, device="cuda")
            st[x + "_out"] = out if case["order"] == "blocks" else out.transpose(1, 2)
        st["list"] = None
        if case["list"]:  # a choice of the valid blocks, each once
            u, j = valid.reshape(B * Hkv, cap).nonzero(as_tuple=True)
            pick = torch.randperm(u.numel(), generator=g, device="cuda")[: case["list"]]
            st["list"] = torch.stack([u[pick], j[pick]], 1).to(torch.int32)
        return st
    prev, Hq = _prev(case), case["Hq"]
    n_tok = sum(lens) - sum(prev)
    st |= {"prev_len": _i32(prev) if case["new"] else None, "n_tok": n_tok, "Hq": Hq}
    b, t = _tokens(st, n_tok)
    st["pos"] = t.to(torch.int32)
    if case["ragged"]:  # slices of one fused projection's output
        qkv = _rows(g, n_tok, (Hq + 2 * Hkv) * D, 0, gain=True)
        parts = [qkv[:, : Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]]
    else:
        parts = [_rows(g, n_tok, h * D, 0, gain=True) for h in (Hq, Hkv, Hkv)]
    st["q"], st["K_new"], st["V_new"] = [x.unflatten(1, (h, D)) if h else None for x, h in zip(parts, (Hq, Hkv, Hkv))]
    st["q_out"] = torch.empty((n_tok, Hq, D), dtype=torch.bfloat16, device="cuda") if Hq else None
    if op == "append":
        slot = table.permute(0, 2, 1)[b, t // P].long()
        st["slot_map"] = (slot * P + (t % P)[:, None]).contiguous()
        for x in "KV":
            st[x + "_pool"] = torch.full((n_slots, P, D), 0.5, dtype=torch.bfloat16, device="cuda")
        return st
    for x in "KV":
        if case["new"]:  # blocks that hold tokens already; tails of the new ones may be larger than they are
            codes = (_bf16(g, n_slots, P, D) * 20.0).float().clamp_(-FMAX[case["fmt"]], FMAX[case["fmt"]])
            st[x + "_pool"] = codes.to(FP8[case["fmt"]])
            st[x + "_scale"] = torch.exp2(torch.randint(-8, -4, (n_slots,), generator=g, device="cuda").float())
        else:
            st[x + "_pool"] = torch.full((n_slots, P, D), FILL, dtype=torch.uint8, device="cuda").view(FP8[case["fmt"]])
            st[x + "_scale"] = torch.full((n_slots,), 0.5, device="cuda")
    return st


def _tokens(st, n):
    """(sequence, position) of n new tokens, packed by sequence."""
    seq = st["seq_len"].long()
    prev = torch.zeros_like(seq) if st["prev_len"] is None else st["prev_len"].long()
    cu = torch.cumsum(seq - prev, 0)
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, i, right=True)
    return b, i - (cu - seq + prev)[b] + prev[b]


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_norm(x, kind, w, b):
    """fp32 rows normalised: by their root mean square, or to mean 0 and variance 1."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return x if b is None else x + b.float()


def _plain_rotate(st, x, pos, w):
    """fp32 heads [n][heads][D], normalised (w) and turned by pos [n]; the angles in 64 bits."""
    case, rot = st["case"], st["case"]["rot"]
    if w is not None:
        x = _plain_norm(x, "rms", w, None)
    angle = pos.double()[:, None] * st["freq"]
    cos, sin = (angle.cos() * st["amp"]).float()[:, None], (angle.sin() * st["amp"]).float()[:, None]
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = [a * cos - b * sin, b * cos + a * sin]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = [torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)]
    return torch.cat(turned + [x[..., rot:]], -1)


def _plain_addnorm(st):
    case = st["case"]
    y = st["Y"].float()
    if case["post"]:
        y = _plain_norm(y, case["kind"], st["w_post"], st["b_post"])
    if st["gate"] is not None:
        y = y * st["gate"].float()
    h = st["H"].float() + case["alpha"] * y
    del y
    out = {"H": h.to(st["H"].dtype), "X": _plain_norm(h, case["kind"], st["w"], st["b"]).to(torch.bfloat16)}
    if case["ahead"]:
        out["X_ahead"] = _plain_norm(h, case["kind"], st["w_ahead"], st["b_ahead"]).to(torch.bfloat16)
    return out


def _plain_rotate_case(st):
    y = _plain_rotate(st, st["x"].float(), st["pos"], st["qw"]).to(torch.bfloat16)
    st["out"].copy_(torch.where((st["pos"] >= 0)[:, None, None], y, st["out"]))  # padding rows stay
    return {"out": st["out"]}


def _plain_append(st):
    out = {}
    if st["q"] is not None:
        out["q"] = _plain_rotate(st, st["q"].float(), st["pos"], st["qw"]).to(torch.bfloat16)
    k = _plain_rotate(st, st["K_new"].float(), st["pos"], st["kw"]).to(torch.bfloat16)
    if st["case"]["op"] == "append":
        rows = st["slot_map"].reshape(-1)
        st["K_pool"].view(-1, D)[rows] = k.reshape(-1, D)
        st["V_pool"].view(-1, D)[rows] = st["V_new"].reshape(-1, D)
        return out | {"K_pool": st["K_pool"], "V_pool": st["V_pool"]}
    B, Hkv, P, cap = st["B"], st["Hkv"], st["P"], st["cap"]
    fmt = st["case"]["fmt"]
    seq = st["seq_len"].long()
    prev = torch.zeros_like(seq) if st["prev_len"] is None else st["prev_len"].long()
    cu = torch.cumsum(seq - prev, 0) - (seq - prev)
    col = torch.arange(cap, device="cuda")
    touched = (col >= (prev // P)[:, None]) & (col < ((seq + P - 1) // P)[:, None]) & (seq > prev)[:, None]
    b, j = touched.nonzero(as_tuple=True)  # touched blocks [m] of each KV head
    t = j[:, None] * P + torch.arange(P, device="cuda")[None, :]  # [m, P]
    fresh = ((t >= prev[b][:, None]) & (t < seq[b][:, None]))[:, None, :, None]
    kept = (t < prev[b][:, None])[:, None, :, None]
    row = (cu[b][:, None] + t - prev[b][:, None]).clamp(0, st["n_tok"] - 1)
    slot = st["table"].permute(0, 2, 1)[b, j].long()  # [m, Hkv]

    def one(new, pool, scale):
        x = new[row].permute(0, 2, 1, 3).float()  # [m, Hkv, P, D]
        mag = torch.where(fresh, x.abs(), 0.0).amax(dim=(2, 3))
        frac, exp = torch.frexp(mag)  # mag = frac 2^exp, frac in [0.5, 1); FMAX = 0.875 2^top
        top = 9 if fmt == "e4m3" else 16
        e = torch.where(mag > 0, (exp - top + (frac > 0.875).to(exp.dtype)).clamp(-126, 127), -126)
        need = ((e + 127) << 23).to(torch.int32).view(torch.float32)
        old = scale[slot]
        s = torch.where((prev[b] > j * P)[:, None], torch.maximum(need, old), need)
        codes = (x / s[:, :, None, None]).clamp(-FMAX[fmt], FMAX[fmt])
        before = pool.view(torch.uint8)[slot]
        again = before.view(FP8[fmt]).float() * (old / s)[:, :, None, None]
        new_codes = torch.where(kept, again, codes).to(FP8[fmt]).view(torch.uint8)
        pool.view(torch.uint8)[slot] = torch.where(fresh | kept, new_codes, before)
        scale[slot] = s

    one(k, st["K_pool"], st["K_scale"])
    one(st["V_new"], st["V_pool"], st["V_scale"])
    return out | {n: st[n] for n in ("K_pool", "V_pool", "K_scale", "V_scale")}


def _plain_predict(st):
    q = (st["X"].float() @ st["W"].float().T).view(st["case"]["M"], -1, D)
    return {"Q": _plain_rotate(st, q, st["pos"], st["qw"]).to(torch.bfloat16)}


def _plain_read(st):
    B, Hkv, P, cap = st["B"], st["Hkv"], st["P"], st["cap"]
    want = torch.zeros((B * Hkv, cap), dtype=torch.bool, device="cuda")
    if st["list"] is None:
        want[:] = True
    else:
        want[st["list"][:, 0].long(), st["list"][:, 1].long()] = True
    t = torch.arange(cap * P, device="cuda")
    live = want.view(B, Hkv, cap).repeat_interleave(P, 2) & (t < st["seq_len"][:, None])[:, None, :]
    slot = st["table"].long().clamp_min(0)
    for x in "KV":
        v = st[x + "_pool"]
        if v.dtype == torch.bfloat16:
            v = v[slot]
        else:
            v = v.view(torch.uint8)[slot].view(v.dtype).float() * st[x + "_scale"][slot][..., None, None]
        v = v.to(torch.bfloat16).view(B, Hkv, cap * P, D)
        st[x + "_out"].copy_(torch.where(live[..., None], v, st[x + "_out"]))
    return {"K": st["K_out"], "V": st["V_out"]}


def _own(st):
    """The same through the library, as a user's program calls it; the rotary positions' table is kept with the state."""
    import block_sparse_kv_pred_gb300 as bs

    case, op = st["case"], st["case"]["op"]
    if op == "addnorm":
        more = {"w_ahead": st["w_ahead"], "b_ahead": st["b_ahead"], "X_ahead": st["X_ahead"]} if case["ahead"] else {}
        bs.add_norm(case["kind"], st["Y"], st["H"], st["w"], EPS, b=st["b"], w_post=st["w_post"], b_post=st["b_post"],
                    gate=st["gate"], alpha=case["alpha"], H_out=st["H_out"], X=st["X"], **more)
        out = {"H": st["H_out"], "X": st["X"]}
        return out | {"X_ahead": st["X_ahead"]} if case["ahead"] else out
    if op == "read":
        if case["fmt"] == "bf16":
            bs.read_kv(st["K_pool"], st["V_pool"], st["table"], st["seq_len"], st["B"], st["Hkv"], st["P"], st["K_out"],
                       st["V_out"], block_list=st["list"])
        else:
            bs.read_kv8(st["K_pool"], st["V_pool"], st["K_scale"], st["V_scale"], st["table"], st["seq_len"], st["B"],
                        st["Hkv"], st["P"], st["K_out"], st["V_out"], block_list=st["list"])
        return {"K": st["K_out"], "V": st["V_out"]}
    if "rope" not in st:
        st["rope"] = _library_rope(case)
    if op == "rotate":
        bs.rotate(st["x"], st["pos"], st["rope"], norm=st["qw"], eps=EPS, out=st["out"])
        return {"out": st["out"]}
    if op == "predict":
        Q = bs.predict_q_rotated(st["X"], st["W"], st["pos"], st["rope"], norm=st["qw"], eps=EPS)
        return {"Q": Q.view(case["M"], case["Hq"], D)}
    more = {"q": st["q"], "q_out": st["q_out"], "q_norm": st["qw"]} if st["q"] is not None else {}
    if op == "append":
        bs.append_rotated_kv(st["K_new"], st["V_new"], st["pos"], st["rope"], st["slot_map"], st["Hkv"], st["P"],
                             st["K_pool"], st["V_pool"], k_norm=st["kw"], eps=EPS, **more)
        out = {n: st[n] for n in ("K_pool", "V_pool")}
    else:
        bs.append_rotated_kv8(st["K_new"], st["V_new"], st["rope"], st["table"], st["seq_len"], st["B"], st["Hkv"],
                              st["P"], st["K_pool"], st["V_pool"], st["K_scale"], st["V_scale"], prev_len=st["prev_len"],
                              k_norm=st["kw"], eps=EPS, **more)
        out = {n: st[n] for n in ("K_pool", "V_pool", "K_scale", "V_scale")}
    return {"q": st["q_out"]} | out if st["q"] is not None else out


def run(state):
    if own:
        return _own(state)
    plain = {"addnorm": _plain_addnorm, "rotate": _plain_rotate_case, "append": _plain_append, "append8": _plain_append,
             "predict": _plain_predict, "read": _plain_read}
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "addnorm":
        M, N, wide = case["M"], case["N"], 2 if case["h"] == "bf16" else 4
        rows = 2 + 2 * wide + 2 * (1 + case["ahead"]) + (2 if case["gate"] == "rows" else 0)
        vectors = (1 + case["ahead"] + case["post"]) * (2 if case["kind"] == "layer" else 1) + (case["gate"] == "vector")
        return {"bytes": M * N * rows + 2 * N * vectors, "flops": M * N * (8 + 4 * case["post"])}
    if op == "rotate":
        live = case["n"] - (max(1, case["n"] // 100) if case["n"] > 2 else 0)
        return {"bytes": live * case["heads"] * 4 * D + 4 * case["n"] + 4 * case["rot"],
                "flops": live * case["heads"] * (3 * case["rot"] + 4 * D * case["norm"])}
    if op == "predict":
        M, N, K = case["M"], case["Hq"] * D, case["K"]
        return {"bytes": 2 * (N * K + M * K + M * N) + 4 * M + 4 * case["rot"], "flops": 2 * M * N * K}
    B, Hkv, P, lens = case["B"], case["Hkv"], case["P"], _lens(case)
    nblk = [-(-n // P) for n in lens]
    if op == "read":
        wide, scale = (2, 0) if case["fmt"] == "bf16" else (1, 4)
        blocks, tokens = sum(nblk) * Hkv, sum(lens) * Hkv
        if case["list"]:  # about as many tokens a block as the batch has
            tokens = tokens * min(case["list"], blocks) // blocks
            blocks = min(case["list"], blocks)
        return {"bytes": tokens * 2 * D * (wide + 2) + blocks * (4 + 2 * scale + (8 if case["list"] else 0)) + 4 * B,
                "flops": 0 if wide == 2 else 2 * tokens * D}
    prev = _prev(case)
    tokens = sum(lens) - sum(prev)
    touched = sum(-(-n // P) - p // P for n, p in zip(lens, prev) if n > p) * Hkv
    rows = tokens * case["Hq"] * 4 * D + 4 * case["rot"]
    flops = tokens * (case["Hq"] + Hkv) * (3 * case["rot"] + 4 * D * case["norm"])
    if op == "append":
        return {"bytes": rows + tokens * (Hkv * (2 * 2 * 2 * D + 8) + 4), "flops": flops}
    return {"bytes": rows + tokens * Hkv * 2 * 3 * D + touched * (4 + 2 * 4) + 8 * B, "flops": flops + 4 * tokens * Hkv * D}


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definitions, a part of the rows at a time
# ---------------------------------------------------------------------------
def _decode(codes, fmt):
    """Bytes -> the values they stand for, from the formats' bit fields."""
    c = codes.view(torch.uint8).long()
    ebits, mbits, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    sign = torch.where(c >= 128, -1.0, 1.0).double()
    e = (c >> mbits) & ((1 << ebits) - 1)
    frac = (c & ((1 << mbits) - 1)).double() / (1 << mbits)
    return sign * torch.where(e > 0, (1 + frac) * torch.exp2((e - bias).double()), frac * 2.0 ** (1 - bias))


def _exact_steps(case):
    """The pairs' angles a position step, one pair at a time, and the amplitude."""
    rot, out = case["rot"], []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(case["base"]))
        if case["scaling"] == "linear":
            f /= FACTOR
        elif case["scaling"] == "ntk":
            f *= math.exp(-2.0 * i / (rot - 2) * math.log(FACTOR))
        elif case["scaling"] == "rotations":
            turns = ORIGINAL * f / (2 * math.pi)
            keep = 0.0 if turns <= 1 else 1.0 if turns >= 4 else (turns - 1) / 3
            f *= keep + (1 - keep) / FACTOR
        elif case["scaling"] == "index":
            pair = [rot / 2 * math.log(ORIGINAL / (2 * math.pi * turns), case["base"]) for turns in (32, 1)]
            lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
            slow = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f *= 1 - slow + slow / FACTOR
        out.append(f)
    return (torch.tensor(out, dtype=torch.float64, device="cuda"),
            1.0 + 0.1 * math.log(FACTOR) if case["scaling"] == "index" else 1.0)


def _exact_heads(case, x, pos, w):
    """fp64 heads [n][heads][D]: each pair a complex number, multiplied by the amplitude and exp(i angle)."""
    if w is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * w.double()
    step, amp = _exact_steps(case)
    turn = torch.polar(torch.full_like(step, amp).expand(len(pos), -1), pos.double()[:, None] * step)[:, None]
    rot, half = case["rot"], case["rot"] // 2
    pair = [slice(0, half), slice(half, rot)] if case["layout"] == "half" else [slice(0, rot, 2), slice(1, rot, 2)]
    z = torch.complex(x[..., pair[0]].contiguous(), x[..., pair[1]].contiguous()) * turn
    y = x.clone()
    y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
    return y


def _exact_rows(x, kind, w, b):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS) * w.double()
    return y if b is None else y + b.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "addnorm":
        M, N = case["M"], case["N"]
        names = ["H", "X"] + (["X_ahead"] if case["ahead"] else [])
        out = {n: torch.empty((M, N), dtype=torch.float64, device="cuda") for n in names}
        for r in range(0, M, 8192):
            s = slice(r, min(M, r + 8192))
            y = st["Y"][s].double()
            if case["post"]:
                y = _exact_rows(y, case["kind"], st["w_post"], st["b_post"])
            if case["gate"] != "none":
                y = y * (st["gate"] if case["gate"] == "vector" else st["gate"][s]).double()
            out["H"][s] = st["H"][s].double() + np.float32(case["alpha"]).item() * y
            out["X"][s] = _exact_rows(out["H"][s], case["kind"], st["w"], st["b"])
            if case["ahead"]:
                out["X_ahead"][s] = _exact_rows(out["H"][s], case["kind"], st["w_ahead"], st["b_ahead"])
        return out
    if op == "rotate":
        out = st["out"].double()
        live = int((st["pos"] >= 0).sum())  # padding is at the end
        for r in range(0, live, 4096):
            s = slice(r, min(live, r + 4096))
            out[s] = _exact_heads(case, st["x"][s].double(), st["pos"][s], st["qw"])
        return {"out": out}
    if op == "predict":
        q = torch.stack([(st["W"].double() * x.double()).sum(1) for x in st["X"]]).view(case["M"], -1, D)
        return {"Q": _exact_heads(case, q, st["pos"], st["qw"])}
    B, Hkv, P, lens = case["B"], case["Hkv"], case["P"], _lens(case)
    if op == "read":
        out = {x: st[x + "_out"].double() for x in "KV"}
        blocks = None if st["list"] is None else {tuple(e) for e in st["list"].tolist()}
        for u in range(B * Hkv):
            b, h = divmod(u, Hkv)
            js = [j for j in range(-(-lens[b] // P)) if blocks is None or (u, j) in blocks]
            if not js:
                continue
            slot = st["table"][b, h, js].long()
            at = (torch.tensor(js, device="cuda")[:, None] * P + torch.arange(P, device="cuda")).view(-1)
            ok = at < lens[b]
            for x in "KV":
                pool = st[x + "_pool"]
                v = pool[slot].double() if case["fmt"] == "bf16" else (
                    _decode(pool.view(torch.uint8)[slot], case["fmt"]) * st[x + "_scale"][slot].double()[:, None, None])
                out[x][b, h, at[ok]] = v.reshape(-1, D)[ok]
        return out
    prev, row0, out = _prev(case), 0, {}
    if st["q"] is not None:
        out["q"] = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for x in "KV":
        if op == "append":
            out[x + "_pool"] = st[x + "_pool"].double()
        else:
            out[x + "_pool"] = _decode(st[x + "_pool"], case["fmt"])
            out[x + "_scale"] = st[x + "_scale"].double()
    for b in range(B):
        n_new = lens[b] - prev[b]
        if n_new == 0:
            continue
        s = slice(row0, row0 + n_new)
        pos = torch.arange(prev[b], lens[b], device="cuda")
        if st["q"] is not None:
            out["q"][s] = _exact_heads(case, st["q"][s].double(), pos, st["qw"])
        rows = {"K": _exact_heads(case, st["K_new"][s].double(), pos, st["kw"]), "V": st["V_new"][s].double()}
        row0 += n_new
        if op == "append":
            slot = st["table"][b].long()[:, pos // P]  # [Hkv, n_new]
            for x in "KV":
                out[x + "_pool"][slot, pos % P] = rows[x].permute(1, 0, 2)
            continue
        j0, j1 = prev[b] // P, -(-lens[b] // P)
        slots = st["table"][b, :, j0:j1].long()  # [Hkv, blocks]
        head = prev[b] - j0 * P  # tokens of the first block that are cached already
        for x in "KV":
            new = rows[x].to(torch.bfloat16).double().permute(1, 0, 2)  # a cached key is one of bf16, as in a bf16 cache
            new = torch.nn.functional.pad(new, (0, 0, head, (j1 - j0) * P - head - n_new)).view(Hkv, j1 - j0, P, D)
            big = new.abs().amax((2, 3)) / FMAX[case["fmt"]]
            half, power = torch.frexp(big.clamp_min(2.0 ** -126))  # a power of two itself has half = 0.5
            scale = torch.ldexp(torch.ones_like(half), power - (half == 0.5).to(power.dtype))
            codes, was = out[x + "_pool"], out[x + "_scale"]
            if head:
                scale[:, 0] = torch.maximum(scale[:, 0], was[slots[:, 0]])
            page = codes[slots]
            at = torch.arange((j1 - j0) * P, device="cuda").view(1, -1, P, 1)
            page = torch.where((at >= head) & (at < head + n_new), new / scale[:, :, None, None], page)
            if head:
                grown = page[:, 0] * (was[slots[:, 0]] / scale[:, 0])[:, None, None]
                page[:, 0] = torch.where(at[:, 0] < head, grown, page[:, 0])
            codes[slots], was[slots] = page, scale
    return out
