"""The 8-bit paged cache, from request lengths to attention: what is measured, and its plain form.

Five operators, each reached through ``block_sparse_kv_pred_gb300``:

* ``tables``   build_tables: page table, residency bits, slot map and list of touched blocks from
               the lengths of a batch before and after its new tokens.
* ``append``   append_kv: new bf16 K/V rows into a bf16 pool, by slot map.
* ``append8``  append_kv8: new bf16 K/V rows into an 8-bit pool with one scale per slot (a block of
               one KV head).
* ``digest8``  build_digest8: block digests (min/max or mean) of an 8-bit pool.
* ``attn8``    sparse_attn8 / sparse_attn8_merge: attention over the listed blocks of an 8-bit pool.

``run`` computes them with elementary torch operations, or with the library where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

D = 128
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
#: pool entries that no operator may touch hold this byte (a finite code in both formats)
FILL = 0x31


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the Qwen3-14B-shaped batch: 40 sequences grow by one token
        {"name": "tables_decode_b40", "op": "tables", "B": 40, "Hkv": 8, "T": 32768, "P": 32, "new": 1, "ragged": True},
        # a fresh batch: every table row, and the slot of every (token, KV head)
        {"name": "tables_prompt_b40_32k", "op": "tables", "B": 40, "Hkv": 8, "T": 32768, "P": 32, "new": 0,
         "ragged": True},
        # one decode step of the Qwen3-8B-shaped batch: latency
        {"name": "append_decode_b8", "op": "append", "B": 8, "Hkv": 8, "T": 16384, "P": 32, "new": 1, "ragged": False},
        # prompts of the same batch, K and V rows inside a fused projection's output
        {"name": "append_prompt_b8_16k", "op": "append", "B": 8, "Hkv": 8, "T": 16384, "P": 32, "new": 0,
         "ragged": True},
        # one decode step: a token into each sequence's tail block
        {"name": "append8_decode_b40", "op": "append8", "fmt": "e4m3", "B": 40, "Hkv": 8, "T": 2048, "P": 32, "new": 1,
         "ragged": True},
        # prompts, quantised as they are written
        {"name": "append8_prompt_b8_16k", "op": "append8", "fmt": "e4m3", "B": 8, "Hkv": 8, "T": 16384, "P": 32,
         "new": 0, "ragged": True},
        # all digests of a batch after its prompts
        {"name": "digest8_minmax_b8_16k", "op": "digest8", "fmt": "e4m3", "kind": "minmax", "B": 8, "Hkv": 8,
         "T": 16384, "P": 32, "ragged": False},
        # mean digests, large blocks, ragged lengths
        {"name": "digest8_mean_b5_p64", "op": "digest8", "fmt": "e5m2", "kind": "mean", "B": 5, "Hkv": 4, "T": 9001,
         "P": 64, "ragged": True},
        # a single short sequence: latency
        {"name": "attn8_b1_4k", "op": "attn8", "fmt": "e4m3", "B": 1, "Hq": 8, "Hkv": 2, "T": 4096, "P": 32, "k": 16,
         "fill": 0.75, "merge": True, "ragged": False},
        # small pages, odd lengths, a partial result in fp32
        {"name": "attn8_b7_p16_partial", "op": "attn8", "fmt": "e5m2", "B": 7, "Hq": 12, "Hkv": 4, "T": 5001, "P": 16,
         "k": 100, "fill": 0.6, "merge": False, "ragged": True},
        # the Qwen3-14B-shaped decode step: budget of 2,048 tokens, most of it resident
        {"name": "attn8_b40_32k", "op": "attn8", "fmt": "e4m3", "B": 40, "Hq": 40, "Hkv": 8, "T": 32768, "P": 32,
         "k": 64, "fill": 0.9, "merge": True, "ragged": False},
        # dense attention over long contexts: every block listed
        {"name": "attn8_dense_b4_128k", "op": "attn8", "fmt": "e4m3", "B": 4, "Hq": 32, "Hkv": 8, "T": 131072, "P": 32,
         "k": 4096, "fill": 1.0, "merge": False, "ragged": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "append8", "digest8", "attn8", "attn8"])
    P = rng.choice([16, 32, 64])
    c = {"op": op, "P": P, "B": _log(rng, 1, 40), "Hkv": rng.choice([1, 2, 4, 8]), "ragged": rng.random() < 0.7}
    if op != "tables" and op != "append":
        c["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op == "attn8":
        c["Hq"] = c["Hkv"] * rng.randint(1, 8)
        c["merge"] = rng.random() < 0.5
        c["fill"] = round(rng.uniform(0.3, 1.0), 2)
        c["T"] = _log(rng, 1, 131072)
        most = 4 * 8 * 131072 // (c["B"] * c["Hkv"] * P)  # blocks a unit, to stay below the largest listed case
        blocks = -(-c["T"] // P)
        c["k"] = _log(rng, 1, max(1, min(blocks, most)))
        c["T"] = min(c["T"], 6 * c["k"] * P)
    else:
        c["T"] = _log(rng, 1, min(32768, 8 * 8 * 16384 // (c["B"] * c["Hkv"])))
    if op == "digest8":
        c["kind"] = rng.choice(["minmax", "mean"])
    if op in ("tables", "append", "append8"):
        # 0: whole prompts; otherwise at most so many new tokens for each sequence (a decode step, a chunk)
        c["new"] = rng.choice([0, 1, 1, _log(rng, 1, c["T"])])
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


def _counts(case):
    """Listed blocks of each unit: about `fill` of min(k, valid blocks); with `ragged` one unit in 13 has none."""
    lens, Hkv = _lens(case), case["Hkv"]

    def of_unit(u):
        m = min(case["k"], -(-lens[u // Hkv] // case["P"]))
        f = min(1.0, case["fill"] * (0.8 + 0.4 * ((u * 0.7548776662) % 1.0))) if case["fill"] < 1.0 else 1.0
        return 0 if case["ragged"] and u % 13 == 12 else max(1, int(round(m * f)))

    return [of_unit(u) for u in range(len(lens) * Hkv)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _keys(g, *shape):
    """Keys as models make them: near-normal, with a few channels several times larger."""
    gain = torch.ones(D, device="cuda")
    gain[torch.randperm(D, generator=g, device="cuda")[:4]] = 6.0
    return _randn(g, *shape) * gain


def _quantised(x, fmt):
    """(codes, scales) of blocks [n, P, D], by a plain max-scaling that is none of the operators'."""
    s = (x.abs().amax(dim=(1, 2)) / FMAX[fmt]).clamp_min(1e-20)
    return (x / s[:, None, None]).clamp(-FMAX[fmt], FMAX[fmt]).to(FP8[fmt]), s


def prepare(case, seed):
    g = _gen(seed)
    op, B, Hkv, P = case["op"], case["B"], case["Hkv"], case["P"]
    U = B * Hkv
    lens = _lens(case)
    nblk = [-(-n // P) for n in lens]
    cap = max(nblk) + (1 if case["ragged"] else 0)
    st = {"case": case, "B": B, "Hkv": Hkv, "P": P, "cap": cap, "seq_len": _i32(lens)}
    if op in ("tables", "append", "append8"):
        prev = _prev(case)
        n_tok = sum(lens) - sum(prev)
        had = [-(-p // P) for p in prev]
        st["prev_len"] = _i32(prev) if case["new"] else None
        st["n_tok"] = n_tok
        n_slots = sum(nblk) * Hkv + 5
        slots = torch.randperm(n_slots, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, Hkv, cap), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(cap, device="cuda")
        in_table = (col < _i32(had)[:, None])[:, None, :].expand(B, Hkv, cap)
        n_had = sum(had) * Hkv
        table[in_table] = slots[:n_had]
        free = slots[n_had:].contiguous()
    if op == "tables":
        words = -(-cap // 32)
        bits = torch.zeros((B, Hkv, words * 32), dtype=torch.int64, device="cuda")
        bits[..., :cap] = in_table.long()
        bits = (bits.view(B, Hkv, words, 32) << torch.arange(32, device="cuda")).sum(-1)
        st |= {"n_slots": n_slots, "free": free, "table": table, "words": words,
               "bits": (bits - ((bits >> 31) << 32)).to(torch.int32), "max_tokens": n_tok + 3,
               "max_list": sum(-(-n // P) - p // P for n, p in zip(lens, prev) if n > p) * Hkv + 2,
               "cu_tokens": torch.empty(B + 1, dtype=torch.int32, device="cuda"),
               "counts": torch.empty(3, dtype=torch.int32, device="cuda"),
               "slot_map": torch.empty((n_tok + 3, Hkv), dtype=torch.int64, device="cuda")}
        st["block_list"] = torch.empty((st["max_list"], 2), dtype=torch.int32, device="cuda")
    elif op in ("append", "append8"):
        # K and V rows are slices of a fused projection's output where the lengths are ragged
        pad = 2 * Hkv * D if case["ragged"] else 0
        st["K_new"] = torch.empty((n_tok, Hkv * D + pad), dtype=torch.bfloat16, device="cuda")
        st["K_new"][:, :Hkv * D] = _keys(g, n_tok, Hkv, D).view(n_tok, Hkv * D)
        st["K_new"] = st["K_new"][:, :Hkv * D].view(n_tok, Hkv, D)
        st["V_new"] = torch.empty((n_tok, Hkv * D + pad), dtype=torch.bfloat16, device="cuda")
        st["V_new"][:, :Hkv * D] = _randn(g, n_tok, Hkv * D)
        st["V_new"] = st["V_new"][:, :Hkv * D].view(n_tok, Hkv, D)
        new_in = (col < _i32(nblk)[:, None])[:, None, :].expand(B, Hkv, cap) & ~in_table
        table[new_in] = free[: (sum(nblk) - sum(had)) * Hkv]
        st["table"], st["n_slots"] = table, n_slots
        if op == "append":
            st["slot_map"] = _slots_of(st)
            st["K_pool"] = torch.full((n_slots, P, D), 0.5, dtype=torch.bfloat16, device="cuda")
            st["V_pool"] = torch.full((n_slots, P, D), 0.5, dtype=torch.bfloat16, device="cuda")
        else:
            for x, make in (("K", _keys), ("V", _randn)):
                if case["new"]:  # blocks that hold tokens already; tails of the new one may be larger than they are
                    codes = make(g, n_slots, P, D).mul_(20.0).clamp_(-FMAX[case["fmt"]], FMAX[case["fmt"]])
                    st[x + "_pool"] = codes.to(FP8[case["fmt"]])
                    st[x + "_scale"] = torch.exp2(torch.randint(-8, -4, (n_slots,), generator=g, device="cuda").float())
                else:
                    st[x + "_pool"] = torch.full((n_slots, P, D), FILL, dtype=torch.uint8, device="cuda").view(FP8[case["fmt"]])
                    st[x + "_scale"] = torch.full((n_slots,), 0.5, device="cuda")
    elif op == "digest8":
        n_slots = sum(nblk) * Hkv + 3
        st["n_slots"] = n_slots
        st["K_pool"], st["K_scale"] = _quantised(_keys(g, n_slots, P, D), case["fmt"])
        table = torch.full((B, Hkv, cap), -1, dtype=torch.int32, device="cuda")
        valid = (torch.arange(cap, device="cuda") < _i32(nblk)[:, None])[:, None, :].expand(B, Hkv, cap)
        table[valid] = torch.randperm(n_slots, generator=g, device="cuda").to(torch.int32)[: sum(nblk) * Hkv]
        st["table"] = table
        if case["kind"] == "minmax":
            st["digest"] = torch.zeros((B, Hkv, cap, 2, D), dtype=torch.bfloat16, device="cuda")
        else:
            st["digest"] = torch.zeros((B, Hkv, cap, D), dtype=torch.float32, device="cuda")
    else:
        Hq, k, G = case["Hq"], case["k"], case["Hq"] // Hkv
        counts = _counts(case)
        n_slots = sum(counts) + 3
        st |= {"Hq": Hq, "k": k, "scale": D ** -0.5, "n_slots": n_slots}
        st["K_pool"], st["K_scale"] = _quantised(_keys(g, n_slots, P, D), case["fmt"])
        st["V_pool"], st["V_scale"] = _quantised(_randn(g, n_slots, P, D), case["fmt"])
        # the listed blocks of a unit: a random ascending choice among its valid ones, all resident
        blocks = torch.tensor(nblk, device="cuda").repeat_interleave(Hkv)[:, None]
        pri = torch.rand((U, cap), generator=g, device="cuda")
        pri[torch.arange(cap, device="cuda")[None, :] >= blocks] = 2.0
        cnt = torch.tensor(counts, device="cuda")
        m = min(k, cap)
        pick = pri.argsort(dim=1)[:, :m]
        col = torch.arange(m, device="cuda")[None, :]
        pick = torch.where(col < cnt[:, None], pick, cap).sort(dim=1).values
        lst = torch.full((U, k), -1, dtype=torch.int32, device="cuda")
        lst[:, :m] = torch.where(pick < cap, pick, -1).to(torch.int32)
        table = torch.full((U, cap + 1), -1, dtype=torch.int32, device="cuda")
        slots = torch.full((U, m), -1, dtype=torch.int32, device="cuda")
        slots[col < cnt[:, None]] = torch.randperm(n_slots, generator=g, device="cuda").to(torch.int32)[: sum(counts)]
        table.scatter_(1, pick, slots)
        st["table"] = table[:, :cap].contiguous().view(B, Hkv, cap)
        st["res_list"], st["res_count"] = lst.view(B, Hkv, k), cnt.to(torch.int32).view(B, Hkv)
        # queries that look at some keys in particular: the softmax has peaks
        first = table[:, :cap].max(dim=1).values.clamp_min(0).long()
        near = st["K_pool"].view(torch.uint8)[first, 0].view(FP8[case["fmt"]]).float() * st["K_scale"][first][:, None]
        st["q"] = (_randn(g, U, G, D) + 0.3 * near[:, None]).view(B, Hq, D).to(torch.bfloat16)
        if case["merge"]:
            st["O_cpu"], st["lse_cpu"] = _randn(g, B, Hq, D) * 0.1, _randn(g, B, Hq) + 4.0
            if case["ragged"]:
                st["lse_cpu"][:, ::3] = -math.inf  # heads whose blocks are all on the GPU
                st["O_cpu"][:, ::3] = 0.0
    return st


def _slots_of(st):
    """Slot map of a state whose page table holds every block."""
    B, Hkv, P, n_tok = st["B"], st["Hkv"], st["P"], st["n_tok"]
    b, t = _tokens(st, n_tok)
    slot = st["table"].permute(0, 2, 1)[b, t // P].long()
    return (slot * P + (t % P)[:, None]).contiguous()


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
def _plain_tables(st):
    B, Hkv, P, cap = st["B"], st["Hkv"], st["P"], st["cap"]
    seq = st["seq_len"].long()
    prev = torch.zeros_like(seq) if st["prev_len"] is None else st["prev_len"].long()
    col = torch.arange(cap, device="cuda")
    new = ((col >= ((prev + P - 1) // P)[:, None]) & (col < ((seq + P - 1) // P)[:, None]))
    new = new[:, None, :].expand(B, Hkv, cap)
    order = torch.cumsum(new.reshape(-1).long(), 0) - 1
    slot = st["free"].long()[order.clamp(0, st["free"].numel() - 1)].view(B, Hkv, cap)
    had = -1 if st["prev_len"] is None else st["table"].long()
    table = torch.where(new, slot, had)
    st["table"].copy_(table)
    # residency words
    bit = torch.zeros((B, Hkv, st["words"] * 32), dtype=torch.int64, device="cuda")
    bit[..., :cap] = new.long()
    word = (bit.view(B, Hkv, st["words"], 32) << torch.arange(32, device="cuda")).sum(-1)
    if st["prev_len"] is not None:
        word = word | (st["bits"].long() & 0xFFFFFFFF)
    st["bits"].copy_((word - ((word >> 31) << 32)).to(torch.int32))
    # tokens
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(seq - prev, 0)])
    st["cu_tokens"].copy_(cu)
    i = torch.arange(st["max_tokens"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp_max(B - 1)
    t = i - cu[b] + prev[b]
    live = i < cu[B]
    rows = table.permute(0, 2, 1)[b, (t // P).clamp(0, cap - 1)] * P + (t % P)[:, None]
    st["slot_map"].copy_(torch.where(live[:, None], rows, -1))
    # touched blocks, in (sequence, head, block) order
    lo, hi = prev // P, (seq + P - 1) // P
    touched = (col >= lo[:, None]) & (col < hi[:, None]) & (seq > prev)[:, None]
    touched = touched[:, None, :].expand(B, Hkv, cap).reshape(-1)
    at = torch.cumsum(touched.long(), 0)
    n_list = at[-1]
    where = torch.where(touched, at - 1, st["max_list"])
    lst = torch.full((st["max_list"] + 1, 2), -1, dtype=torch.int32, device="cuda")
    flat = torch.arange(B * Hkv * cap, device="cuda")
    lst[where] = torch.stack([flat // cap, flat % cap], 1).to(torch.int32)
    st["block_list"].copy_(lst[: st["max_list"]])
    st["counts"].copy_(torch.stack([cu[B], n_list, new.sum()]))
    return {n: st[n] for n in ("table", "bits", "cu_tokens", "slot_map", "block_list", "counts")}


def _plain_append(st):
    rows = st["slot_map"].reshape(-1)
    st["K_pool"].view(-1, D)[rows] = st["K_new"].reshape(-1, D)
    st["V_pool"].view(-1, D)[rows] = st["V_new"].reshape(-1, D)
    return {"K": st["K_pool"], "V": st["V_pool"]}


def _plain_append8(st):
    B, Hkv, P, cap = st["B"], st["Hkv"], st["P"], st["cap"]
    fmt = st["case"]["fmt"]
    seq = st["seq_len"].long()
    prev = torch.zeros_like(seq) if st["prev_len"] is None else st["prev_len"].long()
    cu = torch.cumsum(seq - prev, 0) - (seq - prev)
    col = torch.arange(cap, device="cuda")
    touched = (col >= (prev // P)[:, None]) & (col < ((seq + P - 1) // P)[:, None]) & (seq > prev)[:, None]
    b, j = touched.nonzero(as_tuple=True)  # touched blocks [m] of each KV head
    t = j[:, None] * P + torch.arange(P, device="cuda")[None, :]  # [m, P]
    fresh = (t >= prev[b][:, None]) & (t < seq[b][:, None])
    kept = t < prev[b][:, None]
    row = (cu[b][:, None] + t - prev[b][:, None]).clamp(0, st["n_tok"] - 1)
    slot = st["table"].permute(0, 2, 1)[b, j].long()  # [m, Hkv]
    fresh, kept = fresh[:, None, :, None], kept[:, None, :, None]

    def one(new, pool, scale):
        x = new[row].permute(0, 2, 1, 3).float()  # [m, Hkv, P, D]
        mag = torch.where(fresh & torch.isfinite(x), x.abs(), 0.0).amax(dim=(2, 3))
        frac, exp = torch.frexp(mag)  # mag = frac 2^exp, frac in [0.5, 1); FMAX = 0.875 2^top
        top = 9 if fmt == "e4m3" else 16
        e = (exp - top + (frac > 0.875).to(exp.dtype)).clamp(-126, 127)
        e = torch.where(mag > 0, e, -126)
        need = ((e + 127) << 23).to(torch.int32).view(torch.float32)
        old = scale[slot]
        s = torch.where((prev[b] > j * P)[:, None], torch.maximum(need, old), need)
        codes = (x / s[:, :, None, None]).clamp(-FMAX[fmt], FMAX[fmt])
        before = pool.view(torch.uint8)[slot]
        again = before.view(FP8[fmt]).float() * (old / s)[:, :, None, None]
        out = torch.where(kept, again, codes).to(FP8[fmt]).view(torch.uint8)
        pool.view(torch.uint8)[slot] = torch.where(fresh | kept, out, before)
        scale[slot] = s

    one(st["K_new"], st["K_pool"], st["K_scale"])
    one(st["V_new"], st["V_pool"], st["V_scale"])
    return {n: st[n] for n in ("K_pool", "V_pool", "K_scale", "V_scale")}


def _towards(x, up):
    """fp64 -> bf16, rounded up or down (finite values)."""
    y = x.to(torch.float32).to(torch.bfloat16)
    off = (y.double() < x) if up else (y.double() > x)
    bits = y.view(torch.int16).int()
    away = (y > 0) == up  # away from zero: the next larger magnitude
    bits = torch.where(off, torch.where(y == 0, 1 if up else -0x7FFF, bits + torch.where(away, 1, -1)), bits)
    return bits.to(torch.int16).view(torch.bfloat16)


def _plain_digest8(st):
    B, Hkv, P, cap = st["B"], st["Hkv"], st["P"], st["cap"]
    fmt = st["case"]["fmt"]
    slot = st["table"].long().clamp_min(0).view(-1)
    n = (st["seq_len"].long()[:, None] - torch.arange(cap, device="cuda") * P).clamp(0, P)  # valid tokens
    n = n[:, None, :].expand(B, Hkv, cap).reshape(-1)
    live = (torch.arange(P, device="cuda") < n[:, None])[:, :, None]
    x = st["K_pool"].view(torch.uint8)[slot].view(FP8[fmt]).float()
    if st["case"]["kind"] == "minmax":
        s = st["K_scale"][slot].double()[:, None]
        lo = _towards(torch.where(live, x, math.inf).amin(1).clamp_max(FMAX[fmt]).double() * s, False)
        hi = _towards(torch.where(live, x, -math.inf).amax(1).clamp_min(-FMAX[fmt]).double() * s, True)
        d = torch.stack([lo, hi], 1)
    else:  # codes span many binades: the sum in 64 bits
        s = torch.where(live, x, 0.0).double().sum(1) * st["K_scale"][slot].double()[:, None]
        d = (s / n.clamp_min(1)[:, None]).float()
    keep = (n > 0).view(B, Hkv, cap, *([1] * (d.dim() - 1)))
    st["digest"].copy_(torch.where(keep, d.view(st["digest"].shape), st["digest"]))
    return {"digest": st["digest"]}


def _plain_attn8(st):
    B, Hkv, P, cap, Hq, k = st["B"], st["Hkv"], st["P"], st["cap"], st["Hq"], st["k"]
    U, G, fmt = B * Hkv, Hq // Hkv, st["case"]["fmt"]
    k = min(k, cap)
    lst = st["res_list"].view(U, -1)[:, :k].long()
    listed_ = torch.arange(k, device="cuda")[None, :] < st["res_count"].view(U, 1)
    slot = st["table"].view(U, cap).gather(1, lst.clamp_min(0)).long().clamp_min(0)
    t = lst[:, :, None] * P + torch.arange(P, device="cuda")
    live = (listed_[:, :, None] & (t < st["seq_len"].long().repeat_interleave(Hkv)[:, None, None])).view(U, 1, k * P)
    K = (st["K_pool"].view(torch.uint8)[slot].view(FP8[fmt]).float() * st["K_scale"][slot][:, :, None, None])
    s = torch.bmm(st["q"].view(U, G, D).float() * st["scale"], K.view(U, k * P, D).transpose(1, 2))
    del K
    s = torch.where(live, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    V = (st["V_pool"].view(torch.uint8)[slot].view(FP8[fmt]).float() * st["V_scale"][slot][:, :, None, None])
    O = torch.bmm(p, torch.where(live.view(U, k * P, 1), V.view(U, k * P, D), 0.0))
    O = torch.where(l > 0, O / l, 0.0).view(B, Hq, D)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf).view(B, Hq)
    if not st["case"]["merge"]:
        return {"O": O, "lse": lse}
    top = torch.maximum(lse, st["lse_cpu"])
    base = torch.where(top == -math.inf, 0.0, top)
    a, c = torch.exp(lse - base), torch.exp(st["lse_cpu"] - base)
    both = a + c
    O = (a[..., None] * O + c[..., None] * st["O_cpu"]) / torch.where(both > 0, both, 1.0)[..., None]
    return {"O": O.to(torch.bfloat16), "lse": torch.where(both > 0, base + torch.log(both), -math.inf)}


def _own(st):
    """The same through the library, as a user's program calls it; workspaces are kept with the state."""
    import block_sparse_kv_pred_gb300 as bs

    case, B, Hkv, P = st["case"], st["B"], st["Hkv"], st["P"]
    op = case["op"]
    if op == "tables":
        bs.build_tables(st["seq_len"], st["free"], st["n_slots"], B, Hkv, P, st["table"], st["bits"],
                        prev_len=st["prev_len"], cu_tokens=st["cu_tokens"], slot_map=st["slot_map"],
                        block_list=st["block_list"], counts=st["counts"])
        return {n: st[n] for n in ("table", "bits", "cu_tokens", "slot_map", "block_list", "counts")}
    if op == "append":
        bs.append_kv(st["K_new"], st["V_new"], st["slot_map"], Hkv, P, st["K_pool"], st["V_pool"])
        return {"K": st["K_pool"], "V": st["V_pool"]}
    if op == "append8":
        bs.append_kv8(st["K_new"], st["V_new"], st["table"], st["seq_len"], B, Hkv, P, st["K_pool"], st["V_pool"],
                      st["K_scale"], st["V_scale"], prev_len=st["prev_len"])
        return {n: st[n] for n in ("K_pool", "V_pool", "K_scale", "V_scale")}
    if op == "digest8":
        bs.build_digest8(case["kind"], st["K_pool"], st["K_scale"], st["table"], st["seq_len"], B, Hkv, P, st["digest"])
        return {"digest": st["digest"]}
    if "ws" not in st:
        st["ws"] = bs.sparse_attn8_workspace(B, st["Hq"], Hkv, P)
    cache = (st["q"], st["K_pool"], st["V_pool"], st["K_scale"], st["V_scale"], st["table"], st["seq_len"],
             st["res_list"], st["res_count"], B, st["Hq"], Hkv, P, st["k"], st["scale"], st["ws"])
    if case["merge"]:
        O, lse = bs.sparse_attn8_merge(*cache, st["O_cpu"], st["lse_cpu"])
    else:
        O, lse = bs.sparse_attn8(*cache)
    return {"O": O, "lse": lse}


def run(state):
    if own:
        return _own(state)
    plain = {"tables": _plain_tables, "append": _plain_append, "append8": _plain_append8, "digest8": _plain_digest8,
             "attn8": _plain_attn8}
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, B, Hkv, P = case["op"], case["B"], case["Hkv"], case["P"]
    U, lens = B * Hkv, _lens(case)
    nblk = [-(-n // P) for n in lens]
    cap = max(nblk) + (1 if case["ragged"] else 0)
    if op in ("tables", "append", "append8"):
        prev = _prev(case)
        tokens = sum(lens) - sum(prev)
        new = sum(-(-n // P) - -(-p // P) for n, p in zip(lens, prev)) * Hkv
        touched = sum(-(-n // P) - p // P for n, p in zip(lens, prev) if n > p) * Hkv
    if op == "tables":
        whole = 4 * U * cap + 4 * U * -(-cap // 32) if case["new"] == 0 else 8 * new
        return {"bytes": 8 * B + 4 * new + whole + 8 * (tokens + 3) * Hkv + 8 * (touched + 2) + 4 * (B + 4),
                "flops": 0}
    if op == "append":
        return {"bytes": tokens * Hkv * (2 * 2 * 2 * D + 8), "flops": 0}
    if op == "append8":
        return {"bytes": tokens * Hkv * 2 * 3 * D + touched * (4 + 2 * 4) + 8 * B, "flops": 4 * tokens * Hkv * D}
    if op == "digest8":
        return {"bytes": sum(lens) * Hkv * D + sum(nblk) * Hkv * (8 + 4 * D) + 4 * B, "flops": 2 * sum(lens) * Hkv * D}
    counts = _counts(case)
    G = case["Hq"] // Hkv
    tokens = 0
    for u, c in enumerate(counts):  # a list may hold the sequence's partial last block
        tokens += min(c * P, lens[u // Hkv])
    out = (2 + 4) * D + 8 if case["merge"] else 4 * D + 4
    return {"bytes": tokens * 2 * D + sum(counts) * 16 + 4 * U + B * case["Hq"] * (2 * D + out),
            "flops": 4 * tokens * G * D}


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definitions, one sequence or unit at a time
# ---------------------------------------------------------------------------
def _decode(codes, fmt):
    """Bytes -> the values they stand for, from the formats' bit fields."""
    c = codes.view(torch.uint8).long()
    ebits, mbits, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    sign = torch.where(c >= 128, -1.0, 1.0).double()
    e = (c >> mbits) & ((1 << ebits) - 1)
    frac = (c & ((1 << mbits) - 1)).double() / (1 << mbits)
    return sign * torch.where(e > 0, (1 + frac) * torch.exp2((e - bias).double()), frac * 2.0 ** (1 - bias))


def exact(case, seed):
    st = prepare(case, seed)
    op, B, Hkv, P = case["op"], case["B"], case["Hkv"], case["P"]
    if op in ("tables", "append"):
        return None  # whole numbers and copies: nothing is rounded
    lens = _lens(case)
    if op == "append8":
        prev, row0, out = _prev(case), 0, {}
        for x in "KV":
            out[x + "_pool"] = _decode(st[x + "_pool"], case["fmt"])
            out[x + "_scale"] = st[x + "_scale"].double()
        for b in range(B):
            n_new = lens[b] - prev[b]
            if n_new == 0:
                continue
            j0, j1 = prev[b] // P, -(-lens[b] // P)
            slots = st["table"][b, :, j0:j1].long()  # [Hkv, blocks]
            head = prev[b] - j0 * P  # tokens of the first block that are cached already
            for x in "KV":
                new = st[x + "_new"][row0:row0 + n_new].double().permute(1, 0, 2)
                new = torch.nn.functional.pad(new, (0, 0, head, (j1 - j0) * P - head - n_new)).view(Hkv, j1 - j0, P, D)
                big = new.abs().amax((2, 3)) / FMAX[case["fmt"]]
                half, power = torch.frexp(big.clamp_min(2.0 ** -126))  # a power of two itself has half = 0.5
                s = torch.ldexp(torch.ones_like(half), power - (half == 0.5).to(power.dtype))
                codes, was = out[x + "_pool"], out[x + "_scale"]
                if head:
                    s[:, 0] = torch.maximum(s[:, 0], was[slots[:, 0]])
                page = codes[slots]
                pos = torch.arange((j1 - j0) * P, device="cuda").view(1, -1, P, 1)
                page = torch.where((pos >= head) & (pos < head + n_new), new / s[:, :, None, None], page)
                if head:
                    grown = page[:, 0] * (was[slots[:, 0]] / s[:, 0])[:, None, None]
                    page[:, 0] = torch.where(pos[:, 0] < head, grown, page[:, 0])
                codes[slots], was[slots] = page, s
            row0 += n_new
        return {n: out[n] for n in ("K_pool", "V_pool", "K_scale", "V_scale")}
    if op == "digest8":
        out = torch.zeros(st["digest"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            m = -(-lens[b] // P)
            slot = st["table"][b, :, :m].long()
            x = _decode(st["K_pool"].view(torch.uint8)[slot], case["fmt"]) * st["K_scale"][slot].double()[:, :, None, None]
            rest = lens[b] - (m - 1) * P
            if case["kind"] == "minmax":
                out[b, :, :m, 0], out[b, :, :m, 1] = x.amin(2), x.amax(2)
                out[b, :, m - 1, 0], out[b, :, m - 1, 1] = x[:, -1, :rest].amin(1), x[:, -1, :rest].amax(1)
            else:
                out[b, :, :m] = x.mean(2)
                out[b, :, m - 1] = x[:, -1, :rest].mean(1)
        return {"digest": out}
    Hq, G = case["Hq"], case["Hq"] // Hkv
    O = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for u, c in enumerate(_counts(case)):
        b, h = divmod(u, Hkv)
        if c == 0:
            continue
        j = st["res_list"][b, h, :c].long()
        slot = st["table"][b, h, j].long()
        live = (j[:, None] * P + torch.arange(P, device="cuda") < lens[b]).view(-1)
        K = (_decode(st["K_pool"].view(torch.uint8)[slot], case["fmt"]) * st["K_scale"][slot].double()[:, None, None]).view(-1, D)[live]
        V = (_decode(st["V_pool"].view(torch.uint8)[slot], case["fmt"]) * st["V_scale"][slot].double()[:, None, None]).view(-1, D)[live]
        s = st["q"][b, h * G:(h + 1) * G].double() @ K.T * st["scale"]
        lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, 1)
        O[b, h * G:(h + 1) * G] = torch.softmax(s, 1) @ V
    if not case["merge"]:
        return {"O": O, "lse": lse}
    both = torch.logaddexp(lse, st["lse_cpu"].double())
    part = lambda l: torch.where(l > -math.inf, torch.exp(l - torch.where(both > -math.inf, both, 0.0)), 0.0)[..., None]  # noqa: E731
    return {"O": part(lse) * O + part(st["lse_cpu"].double()) * st["O_cpu"].double(), "lse": both}
