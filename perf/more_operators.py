"""The 8-bit KV cache and eviction by accumulated attention weight, as cases to be timed.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as the
library's calls:

  store8   lat_kv_append_q8 + lat_kv_expand_q8: new K/V rows into the 8-bit cache, and rows of
           it read back as K/V
  attend8  lat_attn_decode_q8: one query token per sequence over the 8-bit cache
  weigh    lat_attn_key_weights: what each cached key was given by the last n_q query rows of
           its sequence, summed over rows and the KV head's query heads, onto a running sum
  evict    lat_kv_evict_choose + lat_kv_evict_rows: the n_keep keys of each KV head that stay
           (the first, the last and the heaviest others), and K/V rows moved up in place

The 8-bit cache.  block_size tokens of one KV head are one record: their rows (one after
another, 2 D bytes each: D codes of K, D of V, in the channels' order), then a 32-bit float
scale for K and one for V, padded to 128 bytes in all.  A code is an e4m3 number and stands for
code * scale, scale = 2^e with the least e in -100 .. 119 for which the block's largest
magnitude is at most 448 * 2^e.  Rows are cut into parts of 16 bytes; part p of row j lies at
place p ^ f(j % 8), f(r) = r ^ (4 * (r % 2)), but at head_dim 80 at place p.  Rows appended to a
block that was begun earlier raise its scale where they must: the codes before them are then
rounded to the new one.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HEAD_DIMS = (64, 80, 128, 256, 512)


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # the next chunk of eight prompts enters the cache, all rows read back for its prefill
        {"name": "store8_chunk", "op": "store8", "dt": "bf16", "B": 8, "Hkv": 8, "D": 128, "block": 64,
         "pos": 1536, "n_new": 512, "back": 0, "cap": 4096, "head_major": False},
        # one new token for each of 32 requests, inside a block; the block read back
        {"name": "store8_step", "op": "store8", "dt": "bf16", "B": 32, "Hkv": 8, "D": 128, "block": 64,
         "pos": 2027, "n_new": 1, "back": 1984, "cap": 4096, "head_major": False},
        # a chat turn of one user on a small model: latency is all there is
        {"name": "attend8_one_short", "op": "attend8", "dt": "bf16", "B": 1, "Hq": 16, "Hkv": 8, "D": 64, "block": 64,
         "cap": 512, "ragged": False, "head_major": False, "window": 0, "softcap": 0.0},
        # continuous batching: 32 requests of every age over 4096-slot caches
        {"name": "attend8_batch", "op": "attend8", "dt": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "D": 128, "block": 64,
         "cap": 4096, "ragged": True, "head_major": False, "window": 0, "softcap": 0.0},
        # whole-repository contexts, eight at once
        {"name": "attend8_128k", "op": "attend8", "dt": "bf16", "B": 8, "Hq": 32, "Hkv": 8, "D": 128, "block": 64,
         "cap": 131072, "ragged": False, "head_major": True, "window": 0, "softcap": 0.0},
        # a 32-bit evaluation run: odd lengths, head_dim 80, small blocks, a window and a score cap
        {"name": "attend8_f32_capped", "op": "attend8", "dt": "f32", "B": 9, "Hq": 10, "Hkv": 2, "D": 80, "block": 16,
         "cap": 5003, "ragged": True, "head_major": False, "window": 2500, "softcap": 30.0},
        # after a decode step of continuous batching: its weights onto the running sums
        {"name": "weigh_step", "op": "weigh", "dt": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "D": 128, "n_q": 1,
         "cap": 4096, "ragged": True, "head_major": False, "window": 0, "softcap": 0.0},
        # the end of four long prompts: what their last 64 tokens looked at
        {"name": "weigh_window", "op": "weigh", "dt": "bf16", "B": 4, "Hq": 32, "Hkv": 8, "D": 128, "n_q": 64,
         "cap": 32768, "ragged": True, "head_major": False, "window": 0, "softcap": 0.0},
        # a whole prompt with capped scores
        {"name": "weigh_prompt", "op": "weigh", "dt": "bf16", "B": 1, "Hq": 16, "Hkv": 8, "D": 256, "n_q": 8192,
         "cap": 8192, "ragged": False, "head_major": False, "window": 0, "softcap": 50.0},
        # a 32-bit evaluation run over a handful of new tokens, with a window
        {"name": "weigh_f32", "op": "weigh", "dt": "f32", "B": 5, "Hq": 12, "Hkv": 4, "D": 64, "n_q": 7,
         "cap": 3001, "ragged": True, "head_major": True, "window": 1000, "softcap": 0.0},
        # long prompts cut down to a quarter before they are decoded from
        {"name": "evict_prompt", "op": "evict", "dt": "bf16", "B": 4, "Hkv": 8, "D": 128, "cap": 65536,
         "n_keep": 16384, "n_first": 4, "n_last": 64, "ragged": False, "head_major": False},
        # a few short 32-bit sequences that ran over their budget
        {"name": "evict_f32", "op": "evict", "dt": "f32", "B": 3, "Hkv": 2, "D": 64, "cap": 701,
         "n_keep": 515, "n_first": 2, "n_last": 33, "ragged": True, "head_major": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store8", "attend8", "attend8", "weigh", "weigh", "evict"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    while True:
        D = rng.choice(HEAD_DIMS)
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 12])
        B = _log(rng, 1, 48)
        cap = _log(rng, 64, 131072)
        block = rng.choice([16, 32, 64, 128])
        if B * cap * Hkv * D > (1 << 28):  # a quarter of the largest case's channels
            continue
        c = {"op": op, "dt": dt, "B": B, "Hkv": Hkv, "D": D, "cap": cap, "head_major": rng.random() < 0.5}
        if op == "store8":
            n_new = _log(rng, 1, min(cap, 8192))
            pos = rng.randint(0, cap - n_new)
            return {**c, "block": block, "n_new": n_new, "pos": pos, "back": rng.choice([0, pos // block * block])}
        c["ragged"] = rng.random() < 0.6
        if op == "evict":
            n_keep = _log(rng, max(1, cap // 16), cap)
            n_last = rng.randint(0, min(64, n_keep))
            return {**c, "n_keep": n_keep, "n_first": rng.randint(0, min(4, n_keep - n_last)), "n_last": n_last}
        window = rng.choice([0, 0, _log(rng, 1, 2 * cap)])
        c = {**c, "Hq": Hq, "window": window, "softcap": rng.choice([0.0, 0.0, 30.0])}
        if op == "attend8":
            return {**c, "block": block}
        n_q = rng.choice([1, 1, _log(rng, 1, min(cap, 4096))])
        # the plain form holds all scores; 32-bit products cost what they cost
        if B * Hq * n_q * cap > (1 << 29) or (dt == "f32" and B * Hq * n_q * cap * D > (1 << 35)):
            continue
        return {**c, "n_q": n_q}


# --------------------------------------------------------------------------------- inputs
def _record_bytes(D, block):
    return -(-(block * 2 * D + 8) // 128) * 128


def _lens(c, g):
    """Cached lengths: every one of them `cap`, or spread over 1 .. cap with one at cap."""
    if not c["ragged"]:
        return torch.full((c["B"],), c["cap"], dtype=torch.int32, device="cuda")
    n = torch.randint(1, c["cap"] + 1, (c["B"],), generator=g, device="cuda").int()
    n[c["B"] // 2] = c["cap"]
    return n


def _keys_like(rows, Hkv, D, g):
    """Keys as projections give them: channels of unequal size, some with a standing offset."""
    h = torch.randn(2, Hkv, D, generator=g, device="cuda")
    x = torch.randn(rows, Hkv, D, generator=g, device="cuda")
    return x.mul_(torch.exp(0.4 * h[0])).add_(0.5 * h[1])


def _strided(x, head_major):
    """[B, n, H, W] as a cache holds it: token-major as it is, or one run of tokens per head."""
    return x.transpose(1, 2).contiguous().transpose(1, 2) if head_major else x.contiguous()


def _two_to(e):
    return ((e + 127) << 23).int().view(torch.float32)


def _exponent(amax):
    """The least e in -100 .. 119 with amax <= 448 * 2^e = 0.875 * 2^(e + 9)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(-100, 119).int()


def _swapped(rows, D):
    """rows [..., block, 2 D] of bytes with their 16-byte parts at the other places."""
    if D == 80:
        return rows
    j = torch.arange(rows.shape[-2], device=rows.device) % 8
    part = torch.arange(D // 8, device=rows.device) ^ (j ^ (j % 2 * 4))[:, None]
    x = rows.unflatten(-1, (D // 8, 16))
    return x.gather(-2, part[..., None].expand(x.shape)).flatten(-2)


def _pack(k, v, block):
    """K and V rows [blocks, block, Hkv, D] in 32 bits as records [blocks, Hkv, bytes]."""
    D = k.shape[-1]
    x = torch.stack([k, v]).transpose(2, 3)  # 2, blocks, Hkv, block, D
    e = _exponent(x.abs().amax((-1, -2)))
    codes = (x * _two_to(-e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.zeros(*x.shape[1:3], _record_bytes(D, block), dtype=torch.uint8, device=k.device)
    out[..., :block * 2 * D] = _swapped(torch.cat([codes[0], codes[1]], -1), D).flatten(-2)
    out[..., block * 2 * D:block * 2 * D + 8] = _two_to(e).movedim(0, -1).contiguous().view(torch.uint8)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    dt = DTYPES[c["dt"]]
    B, Hkv, D, cap = c["B"], c["Hkv"], c["D"], c["cap"]
    s = {"case": c}
    if "ragged" in c:
        s["lens"] = _lens(c, g)
    if "Hq" in c:  # the queries sit in the rows of a fused projection
        qkv = torch.randn(B * c.get("n_q", 1), (c["Hq"] + 2 * Hkv) * D, generator=g, device="cuda").to(dt)
        s["q"] = qkv[:, :c["Hq"] * D]
    if c["op"] == "store8":
        n = B * c["n_new"]
        new = torch.empty(n, 2 * Hkv * D, device="cuda", dtype=dt)
        new[:, :Hkv * D] = _keys_like(n, Hkv, D, g).flatten(1)
        new[:, Hkv * D:] = torch.randn(n, Hkv * D, generator=g, device="cuda")
        s["k_new"], s["v_new"] = new[:, :Hkv * D], new[:, Hkv * D:]
        s["pos"] = torch.full((B,), c["pos"], dtype=torch.int32, device="cuda")
    if c["op"] in ("store8", "attend8"):  # the cache's records, filled a sequence at a time
        bs, nb, rb = c["block"], -(-cap // c["block"]), _record_bytes(D, c["block"])
        shape = (B, Hkv, nb, rb) if c["head_major"] else (B, nb, Hkv, rb)
        cache = torch.empty(shape, dtype=torch.uint8, device="cuda")
        cache = cache.transpose(1, 2) if c["head_major"] else cache
        step = max(1, 32768 // bs)
        for b in range(B):
            for lo in range(0, nb, step):
                m = min(step, nb - lo)
                k = _keys_like(m * bs, Hkv, D, g).to(dt).float()
                v = torch.randn(m * bs, Hkv, D, generator=g, device="cuda").to(dt).float()
                cache[b, lo:lo + m] = _pack(k.unflatten(0, (m, bs)), v.unflatten(0, (m, bs)), bs)
        s["cache"] = cache
    if c["op"] in ("weigh", "evict"):
        k = torch.empty(B, cap, Hkv, D, dtype=dt, device="cuda")
        for b in range(B):
            k[b] = _keys_like(cap, Hkv, D, g)
        s["k"] = _strided(k, c["head_major"])
        # what the keys were given by a few rows before: some have nearly all of it, some nothing
        w = torch.exp(2 * torch.randn(B, Hkv, cap, generator=g, device="cuda"))
        s["w"] = w * (torch.rand(B, Hkv, cap, generator=g, device="cuda") > 0.05) / cap
    if c["op"] == "weigh":  # the log-sum-exps that the rows' attention left
        s["lse"] = torch.cat([_lse(s, c, b) for b in range(B)])
    if c["op"] == "evict":
        v = torch.empty(B, cap, Hkv, D, dtype=dt, device="cuda")
        for b in range(B):
            v[b] = torch.randn(cap, Hkv, D, generator=g, device="cuda")
        s["v"] = _strided(v, c["head_major"])
    return s


def _lse(s, c, b):
    n = c["n_q"]
    x = _weigh_scores(s["q"][b * n:(b + 1) * n], s["k"][b:b + 1], s["lens"][b:b + 1], c)
    return torch.logsumexp(x, -1)[0].permute(2, 0, 1).flatten(1).contiguous()  # n_q, Hq


# ------------------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return {"store8": _own_store, "attend8": _own_attend, "weigh": _own_weigh, "evict": _own_evict}[c["op"]](state, c)
    return {"store8": _store, "attend8": _attend, "weigh": _weigh, "evict": _evict}[c["op"]](state, c)


# the plain forms ------------------------------------------------------------------------
def _unpack(rec, D, block):
    """Records [..., bytes] -> codes [..., block, 2, D] in 32 bits and scales [..., 2]."""
    n = block * 2 * D
    rows = _swapped(rec[..., :n].unflatten(-1, (block, 2 * D)), D)
    scale = rec[..., n:n + 8].contiguous().view(torch.float32)
    return rows.unflatten(-1, (2, D)).contiguous().view(torch.float8_e4m3fn).float(), scale


def _rows_of(rec, D, block):
    """Records [B, blocks, Hkv, bytes] -> K and V [B, Hkv, blocks * block, D] in 32 bits."""
    codes, scale = _unpack(rec, D, block)
    x = (codes * scale[..., None, :, None]).transpose(1, 2).flatten(2, 3)
    return x[..., 0, :], x[..., 1, :]


def _scores(q, k, D, cap):
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    return cap * torch.tanh(s / cap) if cap > 0 else s


def _attend(s, c):
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    k, v = _rows_of(s["cache"], D, c["block"])
    q = s["q"].float().view(B, Hkv, -1, D)
    at = torch.arange(k.shape[2], device="cuda")
    lens = s["lens"][:, None]
    seen = (at < lens) & (at >= (lens - c["window"] if c["window"] > 0 else 0 * lens))
    x = _scores(q, k, D, c["softcap"]).masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-3e38))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l.clamp(min=1e-30)
    return o.flatten(1).to(DTYPES[c["dt"]]), (m + torch.log(l)).flatten(1)


def _store(s, c):
    B, Hkv, D, p, n, bs = c["B"], c["Hkv"], c["D"], c["pos"], c["n_new"], c["block"]
    b0, b1, r0 = p // bs, -(-(p + n) // bs), c["back"] // bs
    new = torch.stack([s[x].float().reshape(B, n, Hkv, D) for x in ("k_new", "v_new")], 3)  # B, n, Hkv, 2, D
    new = torch.nn.functional.pad(new, (0, 0, 0, 0, 0, 0, p - b0 * bs, b1 * bs - p - n)).unflatten(1, (b1 - b0, bs))
    e = _exponent(new.abs().amax((2, 5)))  # B, blocks, Hkv, 2
    codes, scale = _unpack(s["cache"][:, b0:b1], D, bs)
    if p > b0 * bs:  # the first block was begun earlier
        e[:, 0] = torch.maximum(e[:, 0], torch.frexp(scale[:, 0])[1] - 1)
    now = _two_to(e)
    by = torch.where(torch.arange(b1 - b0, device="cuda")[:, None, None] == 0, scale / now, torch.ones_like(now))
    row = torch.arange(b0 * bs, b1 * bs, device="cuda").view(b1 - b0, 1, bs, 1, 1)
    old = codes * by[..., None, :, None]
    fresh = new.transpose(2, 3) * _two_to(-e)[..., None, :, None]
    took = torch.where((row >= p) & (row < p + n), fresh, torch.where(row < p, old, codes)).to(torch.float8_e4m3fn)
    rec = s["cache"][:, b0:b1].clone()
    rec[..., :2 * D * bs] = _swapped(took.view(torch.uint8).flatten(-2), D).flatten(-2)
    rec[..., 2 * D * bs:2 * D * bs + 8] = now.view(torch.uint8)
    s["cache"][:, b0:b1] = rec
    back = _rows_of(s["cache"][:, r0:b1], D, bs)
    lo, hi = c["back"] - r0 * bs, p + n - r0 * bs
    return [x[:, :, lo:hi].transpose(1, 2).reshape(-1, Hkv * D).to(DTYPES[c["dt"]]) for x in back]


def _weigh_scores(q, k, lens, c):
    """q [B n_q, Hq D], k [B, cap, Hkv, D] -> scores [B, Hkv, G, n_q, cap], -inf where unseen."""
    n, Hkv, D = c["n_q"], c["Hkv"], c["D"]
    B = k.shape[0]
    q = q.float().reshape(B, n, Hkv, -1, D).permute(0, 2, 3, 1, 4)
    x = _scores(q, k.float().transpose(1, 2)[:, :, None], D, c["softcap"])
    at = torch.arange(k.shape[1], device="cuda")
    pos = lens[:, None, None] - n + torch.arange(n, device="cuda")[:, None]
    unseen = (at > pos) | (pos - at >= c["window"]) if c["window"] > 0 else at > pos
    return x.masked_fill_(unseen[:, None, None], -math.inf)


def _weigh(s, c):
    B, n = c["B"], c["n_q"]
    lse = s["lse"].view(B, n, c["Hkv"], -1).permute(0, 2, 3, 1)[..., None]
    lse = lse.masked_fill(lse == -math.inf, math.inf)  # rows that see nothing
    x = _weigh_scores(s["q"], s["k"], s["lens"], c)
    s["w"] += x.sub_(lse).exp_().sum((2, 3))
    return s["w"]


def _picked(x, kept):
    rows = x.transpose(1, 2)
    return rows.gather(2, kept[..., None].expand(-1, -1, -1, x.shape[-1])).transpose(1, 2)


def _evict(s, c):
    Hkv, cap, n = c["Hkv"], c["cap"], c["n_keep"]
    lens = s["lens"][:, None, None]
    at = torch.arange(cap, device="cuda")
    rank = s["w"].masked_fill((at < c["n_first"]) | (at >= lens - c["n_last"]), math.inf)
    rank = rank.masked_fill(at >= lens, -math.inf)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :n].sort(-1).values
    new_lens = s["lens"].clamp(max=n)
    # sequences within the budget stay as they are
    kept = torch.where((lens <= n) | (at[:n] >= new_lens[:, None, None]), at[:n].expand(kept.shape), kept)
    live = at < new_lens[:, None, None]
    w = s["w"].gather(2, torch.nn.functional.pad(kept, (0, cap - n)))
    s["k"][:, :n], s["v"][:, :n] = (_picked(s[x], kept) for x in ("k", "v"))
    return {"kept": kept.masked_fill(~live[..., :n], -1).int(), "lens": new_lens,
            "weights": torch.where(live, w, torch.zeros_like(w)).masked_fill(at >= lens, 0), "k": s["k"], "v": s["v"]}


# the library's calls -------------------------------------------------------------------
def _lib():
    from gqa_attention_lat_gb300 import binding
    return binding


def _dt(L, c):
    return L.LAT_BF16 if c["dt"] == "bf16" else L.LAT_F32


def _status(s):
    if "status" not in s:
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s["status"]


def _strides(x):
    return x.stride(1), x.stride(2), x.stride(0)


def _own_attend(s, c):
    L = _lib()
    B, Hq, Hkv, D, cap, dt = c["B"], c["Hq"], c["Hkv"], c["D"], c["cap"], _dt(L, c)
    if "scratch" not in s:  # what a serving loop holds from step to step
        s["n_bytes"] = L.lat_attn_decode_q8_workspace_size(dt, B, Hq, Hkv, D, cap)
        s["scratch"] = torch.zeros(max(s["n_bytes"], 256), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, Hq * D, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(B, Hq, dtype=torch.float32, device="cuda")
    L.lat_attn_decode_q8(dt, s["q"], s["q"].stride(0), s["cache"], *_strides(s["cache"]), c["block"], s["lens"], cap,
                         out, out.stride(0), lse, B, Hq, Hkv, D, c["window"], 1.0 / math.sqrt(D), c["softcap"],
                         s["scratch"], s["n_bytes"], _status(s))
    return out, lse


def _own_store(s, c):
    L = _lib()
    B, Hkv, D, n, m, dt = c["B"], c["Hkv"], c["D"], c["n_new"], c["pos"] + c["n_new"] - c["back"], _dt(L, c)
    if "start" not in s:
        s["start"] = torch.full((B,), c["back"], dtype=torch.int32, device="cuda")
    L.lat_kv_append_q8(dt, s["cache"], *_strides(s["cache"]), c["block"], c["cap"], s["k_new"], s["v_new"],
                       s["k_new"].stride(0), s["pos"], n, B, Hkv, D, _status(s))
    k, v = (torch.empty(B * m, Hkv * D, dtype=s["k_new"].dtype, device="cuda") for _ in range(2))
    L.lat_kv_expand_q8(dt, s["cache"], *_strides(s["cache"]), c["block"], c["cap"], k, v, Hkv * D, s["start"], m, B,
                       Hkv, D, _status(s))
    return [k, v]


def _own_weigh(s, c):
    L = _lib()
    L.lat_attn_key_weights(_dt(L, c), s["q"], s["q"].stride(0), c["n_q"], s["k"], *_strides(s["k"]), s["lens"], c["cap"],
                           s["lse"], s["w"], s["w"].stride(1), s["w"].stride(0), c["B"], c["Hq"], c["Hkv"], c["D"], 1,
                           c["window"], 1.0 / math.sqrt(c["D"]), c["softcap"], _status(s))
    return s["w"]


def _own_evict(s, c):
    L = _lib()
    B, Hkv, D, cap, n = c["B"], c["Hkv"], c["D"], c["cap"], c["n_keep"]
    kept = torch.empty(B, Hkv, n, dtype=torch.int32, device="cuda")
    lens, w = torch.empty_like(s["lens"]), torch.zeros_like(s["w"])
    L.lat_kv_evict_choose(s["w"], s["w"].stride(1), s["w"].stride(0), s["lens"], cap, kept, n, c["n_first"], c["n_last"],
                          w, w.stride(1), w.stride(0), lens, B, Hkv, _status(s))
    L.lat_kv_evict_rows(_dt(L, c), s["k"], s["v"], *_strides(s["k"]), cap, kept, n, B, Hkv, D, _status(s))
    return {"kept": kept, "lens": lens, "weights": w, "k": s["k"], "v": s["v"]}


# --------------------------------------------------------------------- floors of one pass
def _mean_len(c):
    return (c["cap"] + 1) / 2 if c["ragged"] else c["cap"]


def work(case):
    c = case
    es = 2 if c["dt"] == "bf16" else 4
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    if c["op"] == "store8":
        n, bs = c["n_new"], c["block"]
        old, m = c["pos"] - c["back"], c["pos"] + n - c["back"]
        scales = 8 * (-(-(c["pos"] + n) // bs) - c["back"] // bs)
        return {"bytes": B * Hkv * (n * 2 * D * (es + 1) + m * 2 * D * es + old * 2 * D + 2 * scales),
                "flops": B * Hkv * D * (8 * n + 4 * m)}
    if c["op"] == "evict":
        # lists and weights, and the rows that move, of sequences that are over the budget
        n, cap = c["n_keep"], c["cap"]
        over = (cap - n) / cap if c["ragged"] else 1.0 if cap > n else 0.0
        return {"bytes": B * Hkv * (8 * _mean_len(c) + 4 * n + over * max(0, n - c["n_first"]) * 4 * D * es),
                "flops": B * Hkv * 4 * _mean_len(c)}
    io = B * c["Hq"] * (2 * D * es + 4)
    if c["op"] == "attend8":
        n = _mean_len(c)
        n = min(n, c["window"]) if c["window"] > 0 else n
        return {"bytes": B * Hkv * n * (2 * D + 8 / c["block"]) + io, "flops": 4 * B * c["Hq"] * D * n}
    n, q = _mean_len(c), c["n_q"]
    seen, rows = n, min(q, n)  # keys that some row sees, rows that there are
    pairs = rows * (n - (rows - 1) / 2)
    if c["window"] > 0:
        seen, pairs = min(n, c["window"] + rows - 1), min(pairs, rows * c["window"])
    return {"bytes": B * (Hkv * seen * (D * es + 8) + rows * c["Hq"] * (D * es + 4)), "flops": 2 * B * c["Hq"] * D * pairs}


# ------------------------------------------------------------ the definitions, in 64 bits
def _power(e):
    """2^e for whole e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(code):
    """The value of a byte: sign, 4 bits of exponent, 3 of mantissa."""
    e, m = (code.int() >> 3) & 15, (code.int() & 7).double()
    x = torch.where(e == 0, m / 512, (1 + m / 8) * _power(e - 7))
    x = torch.where((code & 127) == 127, torch.full_like(x, math.nan), x)
    return torch.where(code >= 128, -x, x)


def _to_e4m3(x):
    """The e4m3 number nearest to x (|x| <= 448), ties to even."""
    step = _power(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _cached(rec, j, D, block, which):
    """Row by row: K or V of cache rows j of one sequence's head, rec [blocks, bytes]."""
    n, r = j // block, j % block
    p = torch.arange(D, device=rec.device) + (D if which == "v" else 0)
    part, inner = p // 16, p % 16
    if D != 80:
        part = part[None, :] ^ (r % 8 ^ r % 2 * 4)[:, None]
    code = rec[n[:, None], r[:, None] * 2 * D + part * 16 + inner]
    raw = rec[n[:, None], torch.arange(4, device=rec.device) + 2 * D * block + (4 if which == "v" else 0)].int()
    scale = (raw[:, 0] | raw[:, 1] << 8 | raw[:, 2] << 16 | raw[:, 3] << 24).view(torch.float32).double()
    return code, scale


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    dev = "cuda"
    if c["op"] == "store8":
        p, n, bs = c["pos"], c["n_new"], c["block"]
        first, m = c["back"], c["pos"] + c["n_new"] - c["back"]
        edges = sorted({p, p + n} | {x * bs for x in range(p // bs + 1, (p + n - 1) // bs + 1)})
        got = []
        for which in ("k", "v"):
            x = s[which + "_new"].double().reshape(B, n, Hkv, D)
            y = torch.empty(B, m, Hkv, D, dtype=torch.float64, device=dev)
            for b in range(B if p > first else 0):
                for h in range(Hkv):
                    code, scale = _cached(s["cache"][b, :, h], torch.arange(first, p, device=dev), D, bs, which)
                    y[b, :p - first, h] = _e4m3(code) * scale[:, None]
            for lo, hi in zip(edges, edges[1:]):  # what the new rows add to each block
                part = x[:, lo - p:hi - p]
                top = part.abs().amax((1, 3)).clamp(min=1e-45)  # B, Hkv
                e = torch.ceil(torch.log2(top / 448))
                e = torch.where(448 * _power(e) < top, e + 1, torch.where(448 * _power(e - 1) >= top, e - 1, e))
                e = e.clamp(-100, 119)
                for b in range(B if lo % bs else 0):  # earlier rows of this block, under the scale that serves all
                    for h in range(Hkv):
                        at = torch.arange(lo // bs * bs, lo, device=dev)
                        code, scale = _cached(s["cache"][b, :, h], at, D, bs, which)
                        was = torch.round(torch.log2(scale[0]))
                        e[b, h] = torch.maximum(e[b, h], was)
                        old = _to_e4m3(_e4m3(code) * _power(was - e[b, h])) * _power(e[b, h])
                        keep = old[max(0, first - lo // bs * bs):]
                        y[b, lo - first - len(keep):lo - first, h] = keep
                by = _power(e)[:, None, :, None]
                y[:, lo - first:hi - first] = _to_e4m3(part / by) * by
            got.append(y.view(B * m, Hkv * D))
        return got
    lens = s["lens"].tolist()
    if c["op"] == "attend8":
        q = s["q"].double().view(B, Hkv, -1, D)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device=dev)
        for b in range(B):
            for h in range(Hkv):
                at = torch.arange(max(0, lens[b] - c["window"]) if c["window"] > 0 else 0, lens[b], device=dev)
                k, v = (_e4m3(code) * scale[:, None]
                        for code, scale in (_cached(s["cache"][b, :, h], at, D, c["block"], w) for w in ("k", "v")))
                x = (q[b, h] @ k.T) * (1.0 / math.sqrt(D))
                if c["softcap"] > 0:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                lse[b, h] = torch.logsumexp(x, -1)
                out[b, h] = torch.exp(x - lse[b, h][:, None]) @ v
        return out.view(B, -1), lse.view(B, -1)
    if c["op"] == "weigh":
        w, n, G = s["w"].double(), c["n_q"], c["Hq"] // Hkv
        for b, L in enumerate(lens):
            rows = torch.arange(max(0, n - L), n, device=dev)  # (a row before the first key is none)
            pos, at = (L - n + rows)[:, None], torch.arange(L, device=dev)
            seen = (at <= pos) & (at > pos - c["window"] if c["window"] > 0 else at >= 0)
            for h in range(Hkv * G):
                q = s["q"][b * n + rows, h * D:(h + 1) * D].double()
                x = (q @ s["k"][b, :L, h // G].double().T) * (1.0 / math.sqrt(D))
                if c["softcap"] > 0:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                x = torch.exp(x - s["lse"][b * n + rows, h].double()[:, None])
                w[b, h // G, :L] += torch.where(seen, x, torch.zeros_like(x)).sum(0)
        return w
    n, first = c["n_keep"], c["n_first"]
    k, v, w = s["k"].double(), s["v"].double(), torch.zeros_like(s["w"], dtype=torch.float64)
    for b, L in enumerate(lens):
        last = L - c["n_last"]
        for h in range(Hkv):
            at = np.arange(L)
            if L > n:
                x = s["w"][b, h, first:last].double().cpu().numpy()
                best = np.lexsort((np.arange(len(x)), -x))[:n - first - c["n_last"]] + first
                at = np.sort(np.concatenate([np.arange(first), best, np.arange(last, L)]))
            at = torch.from_numpy(at).cuda()
            w[b, h, :len(at)] = s["w"][b, h, at].double()
            k[b, :len(at), h], v[b, :len(at), h] = s["k"][b, at, h].double(), s["v"][b, at, h].double()
    return {"kept": None, "lens": None, "weights": w, "k": k, "v": v}
