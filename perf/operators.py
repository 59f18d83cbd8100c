"""The decode operators that read less of a long KV cache, as cases to be timed.

Five operators, each in a plain form (elementary torch operations in 32 bits; 64 for the
block scores, whose order is the answer) and as the library's calls:

  store   lat_kv_append_q4 + lat_kv_expand_q4: new K/V rows into the 4-bit cache, and the
          cached rows read back as K/V (what a chunked prefill over such a cache does)
  attend  lat_attn_decode_q4: one query token per sequence over the 4-bit cache
  bounds  lat_kv_block_bounds: channel maxima and minima of each block of cached keys
  select  lat_attn_select_blocks: the blocks each KV head keeps, by the bound of their scores
  blocks  lat_attn_decode_blocks: one query token per sequence over the kept blocks

The 4-bit row of one token and KV head.  Channels come in groups of 32 (head_dim 80 is
taken as 96 with zeros behind); with mn = min(0, x), mx = max(0, x) over the group,

  s = bf16((mx - mn) / 15),  z = clamp(rint(-mn / s), 0, 15),  c = clamp(rint(x / s) + z, 0, 15)

and the group reads back as s * (c - z).  s goes through fp32 (difference and quotient each
rounded once); the other two quotients round to the nearest whole number as they are, ties
to even.  Groups form sets of SG = 4 (2 at head_dim 64, 3
at 80); with channel d = 32 g + e and g = set * SG + j:
  K code: 32-bit word (set * 4 + e / 8) * SG + j, nibble (e % 8) / 2 + 4 * (e % 2)
  V code: 16-bit half (set * 8 + e % 8) * SG + j, nibble e / 8
and a row is the K words, the V halves, then a 32-bit parameter word per group of K and
per group of V (low half: bf16 s, high half: bf16 of 128 + z), padded to 16 bytes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HEAD_DIMS = (64, 80, 128, 256, 512)


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # a chat turn of one user on a small model: latency is all there is
        {"name": "attend_one_short", "op": "attend", "dt": "bf16", "B": 1, "Hq": 16, "Hkv": 8, "D": 64,
         "cap": 512, "ragged": False, "head_major": False, "window": 0, "softcap": 0.0},
        # continuous batching: 32 requests of every age over 4096-slot caches
        {"name": "attend_batch", "op": "attend", "dt": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "D": 128,
         "cap": 4096, "ragged": True, "head_major": False, "window": 0, "softcap": 0.0},
        # whole-repository contexts, eight at once
        {"name": "attend_128k", "op": "attend", "dt": "bf16", "B": 8, "Hq": 32, "Hkv": 8, "D": 128,
         "cap": 131072, "ragged": False, "head_major": True, "window": 0, "softcap": 0.0},
        # a 32-bit evaluation run: odd lengths, head_dim 80, a window and a score cap
        {"name": "attend_f32_capped", "op": "attend", "dt": "f32", "B": 9, "Hq": 10, "Hkv": 2, "D": 80,
         "cap": 5003, "ragged": True, "head_major": False, "window": 2500, "softcap": 30.0},
        # the next chunk of eight prompts enters the cache, read back for its prefill
        {"name": "store_chunk", "op": "store", "dt": "bf16", "B": 8, "Hkv": 8, "D": 128,
         "pos": 1536, "n_new": 512, "cap": 4096, "head_major": False},
        # the same for one sequence in 32 bits: odd sizes, heads apart
        {"name": "store_f32_odd", "op": "store", "dt": "f32", "B": 1, "Hkv": 3, "D": 256,
         "pos": 777, "n_new": 1023, "cap": 2001, "head_major": True},
        # one new token per request: the bounds of its block follow
        {"name": "bounds_step", "op": "bounds", "dt": "bf16", "B": 32, "Hkv": 8, "D": 128,
         "block": 64, "pos": 4000, "n_new": 1, "cap": 4096, "head_major": False},
        # whole prompts' bounds at once
        {"name": "bounds_prompt", "op": "bounds", "dt": "bf16", "B": 2, "Hkv": 8, "D": 128,
         "block": 64, "pos": 0, "n_new": 65536, "cap": 65536, "head_major": False},
        # a step over 128K contexts: 64 of up to 2048 blocks kept per KV head
        {"name": "select_128k", "op": "select", "dt": "bf16", "B": 8, "Hq": 32, "Hkv": 8, "D": 128,
         "block": 64, "cap": 131072, "n_sel": 64, "n_first": 1, "n_last": 4, "ragged": True, "head_major": False},
        # 32 bits, short and odd
        {"name": "select_f32", "op": "select", "dt": "f32", "B": 5, "Hq": 12, "Hkv": 4, "D": 64,
         "block": 32, "cap": 9000, "n_sel": 33, "n_first": 2, "n_last": 3, "ragged": True, "head_major": True},
        # the attention of the 128K step
        {"name": "blocks_128k", "op": "blocks", "dt": "bf16", "B": 8, "Hq": 32, "Hkv": 8, "D": 128,
         "block": 64, "cap": 131072, "n_sel": 64, "ragged": True, "head_major": False, "softcap": 0.0},
        # one user, wide heads, 32 bits, small blocks
        {"name": "blocks_one_f32", "op": "blocks", "dt": "f32", "B": 1, "Hq": 16, "Hkv": 2, "D": 256,
         "block": 16, "cap": 20011, "n_sel": 128, "ragged": False, "head_major": True, "softcap": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "store", "bounds", "select", "blocks"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    while True:
        D = rng.choice(HEAD_DIMS)
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 8, 12])
        B = _log(rng, 1, 48)
        cap = _log(rng, 64, 131072)
        block = rng.choice([16, 32, 48, 64, 128, 256])
        if B * cap * Hkv * D > (1 << 28):  # a quarter of the largest case's channels
            continue
        c = {"op": op, "dt": dt, "B": B, "Hkv": Hkv, "D": D, "cap": cap, "head_major": rng.random() < 0.5}
        if op == "store":
            n_new = _log(rng, 1, min(cap, 8192))
            return {**c, "n_new": n_new, "pos": rng.randint(0, cap - n_new)}
        if op == "bounds":
            n_new = _log(rng, 1, cap)
            return {**c, "block": block, "n_new": n_new, "pos": rng.randint(0, cap - n_new)}
        c = {**c, "Hq": Hkv * G, "ragged": rng.random() < 0.6}
        if op == "attend":
            return {**c, "window": rng.choice([0, 0, _log(rng, 1, 2 * cap)]), "softcap": rng.choice([0.0, 0.0, 30.0])}
        if op == "blocks":
            n_sel = _log(rng, 1, max(1, min(8192, cap) // block))
            return {**c, "block": block, "n_sel": n_sel, "softcap": rng.choice([0.0, 0.0, 30.0])}
        if cap < 48 * block:  # a choice among few is none
            continue
        n_sel = _log(rng, 2, max(2, min(8192 // block, cap // block // 2)))
        n_last = rng.randint(0, min(4, n_sel - 1))
        return {**c, "block": block, "n_sel": n_sel, "n_first": rng.randint(0, min(2, n_sel - 1 - n_last)),
                "n_last": n_last}


# --------------------------------------------------------------------------------- inputs
def _row_bytes(D):
    P = -(-D // 32) * 32
    return -(-(P + P // 4) // 16) * 16


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


def _quantise(x):
    """x [..., D] in 32 bits -> (codes [..., G, 32], s [..., G] as bf16, z [..., G])."""
    D = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -D % 32)).unflatten(-1, (-1, 32))
    mn, mx = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    s = ((mx - mn) / 15).bfloat16()
    f = torch.where(s == 0, torch.ones_like(s), s).double()  # in 64 bits: quotients next to a half
    z = torch.round(-mn / f).clamp(0, 15)
    c = (torch.round(x / f[..., None]) + z[..., None]).clamp(0, 15)
    return c.float(), s, z.float()


def _pack(k, v):
    """K and V rows [..., D] as the cache's bytes [..., row_bytes]."""
    D = k.shape[-1]
    (ck, sk, zk), (cv, sv, zv) = _quantise(k), _quantise(v)
    G = sk.shape[-1]
    SG = min(4, G)
    lead = ck.shape[:-2]
    n4 = torch.arange(8, device=k.device) * 4
    words = ck.to(torch.int64).view(*lead, G // SG, SG, 4, 4, 2).movedim(-4, -3)  # set, c, j, i, h
    words = (words.transpose(-1, -2).reshape(*lead, -1, 8) << n4).sum(-1)
    halves = cv.to(torch.int64).view(*lead, G // SG, SG, 4, 8)  # set, j, i, r
    halves = (halves.permute(*range(len(lead)), -4, -1, -3, -2).reshape(*lead, -1, 4) << n4[:4]).sum(-1)
    out = torch.zeros(*lead, _row_bytes(D), dtype=torch.uint8, device=k.device)
    P = 32 * G
    for j in range(4):
        out[..., j:P // 2:4] = (words >> (8 * j) & 255).to(torch.uint8)
    for j in range(2):
        out[..., P // 2 + j:P:2] = (halves >> (8 * j) & 255).to(torch.uint8)
    p = torch.stack([torch.cat([sk, sv], -1), (128 + torch.cat([zk, zv], -1)).bfloat16()], -1)
    out[..., P:P + 8 * G] = p.contiguous().view(torch.uint8).flatten(-2)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    dt = DTYPES[c["dt"]]
    B, Hkv, D, cap = c["B"], c["Hkv"], c["D"], c["cap"]
    s = {"case": c}
    if "Hq" in c:  # the queries sit in the rows of a fused projection
        qkv = torch.randn(B, (c["Hq"] + 2 * Hkv) * D, generator=g, device="cuda").to(dt)
        s["q"] = qkv[:, :c["Hq"] * D]
        s["lens"] = _lens(c, g)
    if c["op"] == "store":
        n = B * c["n_new"]
        new = torch.empty(n, 2 * Hkv * D, device="cuda", dtype=dt)
        new[:, :Hkv * D] = _keys_like(n, Hkv, D, g).flatten(1)
        new[:, Hkv * D:] = torch.randn(n, Hkv * D, generator=g, device="cuda")
        s["k_new"], s["v_new"] = new[:, :Hkv * D], new[:, Hkv * D:]
        s["pos"] = torch.full((B,), c["pos"], dtype=torch.int32, device="cuda")
    if c["op"] in ("store", "attend"):  # the packed cache, filled a sequence at a time
        rb = _row_bytes(D)
        shape = (B, Hkv, cap, rb) if c["head_major"] else (B, cap, Hkv, rb)
        cache = torch.empty(shape, dtype=torch.uint8, device="cuda")
        cache = cache.transpose(1, 2) if c["head_major"] else cache
        for b in range(B):
            for lo in range(0, cap, 32768):
                m = min(32768, cap - lo)
                cache[b, lo:lo + m] = _pack(_keys_like(m, Hkv, D, g).to(dt).float(),
                                            torch.randn(m, Hkv, D, generator=g, device="cuda").to(dt).float())
        s["cache"] = cache
    if c["op"] == "bounds":
        k = torch.empty(B, cap, Hkv, D, dtype=dt, device="cuda")
        for b in range(B):
            k[b] = _keys_like(cap, Hkv, D, g)
        s["k"] = _strided(k, c["head_major"])
        nb = -(-cap // c["block"])
        r = torch.randn(B, nb, Hkv, 2, D, generator=g, device="cuda")  # bounds of the rows before
        r[..., 0, :], r[..., 1, :] = r.amax(-2), r.amin(-2)
        s["bounds"] = _strided(r.to(dt).flatten(3), c["head_major"])
        s["pos"] = torch.full((B,), c["pos"], dtype=torch.int32, device="cuda")
    if c["op"] == "select":
        nb = -(-cap // c["block"])
        mid = _keys_like(B * nb, Hkv, D, g)
        off = 2.0 + 0.4 * torch.randn(2, B * nb, Hkv, D, generator=g, device="cuda").abs()
        r = torch.stack([mid + off[0], mid - off[1]], 2).to(dt)
        s["bounds"] = _strided(r.view(B, nb, Hkv, 2 * D), c["head_major"])
    if c["op"] == "blocks":
        kv = torch.empty(2, B, cap, Hkv, D, dtype=dt, device="cuda")
        for b in range(B):
            kv[0, b] = _keys_like(cap, Hkv, D, g)
            kv[1, b] = torch.randn(cap, Hkv, D, generator=g, device="cuda")
        s["k"], s["v"] = _strided(kv[0], c["head_major"]), _strided(kv[1], c["head_major"])
        nb = -(-cap // c["block"])
        have = (s["lens"] + c["block"] - 1) // c["block"]
        score = torch.rand(B, Hkv, nb, generator=g, device="cuda")
        at = torch.arange(nb, device="cuda")
        score = torch.where(at == have[:, None, None] - 1, torch.full_like(score, 2.0), score)
        score = torch.where(at < have[:, None, None], score, torch.full_like(score, -1.0))
        s["blocks"] = _ascending(score, have, c["n_sel"])
    return s


def _ascending(score, have, n_sel):
    """The n_sel best places of the last axis (ties to the lowest) in ascending order, as
    int32 with -1 behind; `have` [B] places of each are real, the rest score lowest."""
    nb = score.shape[-1]
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n_sel]
    best = torch.nn.functional.pad(best, (0, n_sel - best.shape[-1]), value=nb)
    best = torch.where(best < have[:, None, None], best, torch.full_like(best, nb)).sort(-1).values
    return torch.where(best < nb, best, torch.full_like(best, -1)).int()


# ------------------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return {"store": _own_store, "attend": _own_attend, "bounds": _own_bounds, "select": _own_select,
                "blocks": _own_blocks}[c["op"]](state, c)
    return {"store": _store, "attend": _attend, "bounds": _bounds, "select": _select,
            "blocks": _blocks}[c["op"]](state, c)


# the plain forms ------------------------------------------------------------------------
def _read_back(x):
    codes, s, z = _quantise(x)
    return (s.float()[..., None] * (codes - z[..., None])).flatten(-2)[..., :x.shape[-1]]


def _unpack(rows, D):
    """The cache's bytes [..., row_bytes] -> K and V values [..., D] in 32 bits."""
    G = -(-D // 32)
    SG, P, lead = min(4, G), 32 * G, rows.shape[:-1]
    rows = rows.contiguous()
    sh = torch.arange(8, device=rows.device, dtype=torch.int32) * 4
    k = rows[..., :P // 2].contiguous().view(torch.int32)[..., None] >> sh & 15
    k = k.view(*lead, G // SG, 4, SG, 2, 4).movedim(-3, -4).transpose(-1, -2).reshape(*lead, G, 32)
    v = rows[..., P // 2:P].contiguous().view(torch.int16).int()[..., None] >> sh[:4] & 15
    v = v.view(*lead, G // SG, 8, SG, 4)
    v = v.permute(*range(len(lead)), -4, -2, -1, -3).reshape(*lead, G, 32)
    p = rows[..., P:P + 8 * G].contiguous().view(torch.bfloat16).float().view(*lead, 2, G, 2)
    val = [(p[..., t, :, 0, None] * (x - (p[..., t, :, 1, None] - 128))).flatten(-2)[..., :D]
           for t, x in ((0, k), (1, v))]
    return val


def _softmax_rows(scores, seen, v, dt):
    """scores [B, Hkv, G, n], seen [B, 1 or Hkv, 1, n], v [B, n, Hkv, D] or [B, Hkv, n, D]."""
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m.clamp(min=-3e38))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l.clamp(min=1e-30)
    lse = (m + torch.log(l)).flatten(1)
    return o.flatten(1).to(dt), lse


def _scores(q, k, D, cap):
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    return cap * torch.tanh(s / cap) if cap > 0 else s


def _attend(s, c):
    B, Hkv, D, n = c["B"], c["Hkv"], c["D"], c["cap"]
    k, v = _unpack(s["cache"], D)
    q = s["q"].float().view(B, Hkv, -1, D)
    at = torch.arange(n, device="cuda")
    lens = s["lens"][:, None]
    seen = (at < lens) & (at >= (lens - c["window"] if c["window"] > 0 else 0 * lens))
    return _softmax_rows(_scores(q, k.transpose(1, 2), D, c["softcap"]), seen[:, None, None],
                         v.transpose(1, 2), DTYPES[c["dt"]])


def _store(s, c):
    B, Hkv, D, p, n = c["B"], c["Hkv"], c["D"], c["pos"], c["n_new"]
    k_new, v_new = (s[x].float().reshape(B, n, Hkv, D) for x in ("k_new", "v_new"))
    old = _unpack(s["cache"][:, :p], D)
    return [torch.cat([o, _read_back(x)], 1).to(DTYPES[c["dt"]]).view(B * (p + n), Hkv * D)
            for o, x in zip(old, (k_new, v_new))]


def _bounds(s, c):
    D, p, n, bs = c["D"], c["pos"], c["n_new"], c["block"]
    b0, b1 = p // bs, -(-(p + n) // bs)  # the blocks that hold new rows
    k = s["k"][:, p:p + n].float()
    front, back = p - b0 * bs, b1 * bs - p - n
    k = torch.nn.functional.pad(k, (0, 0, 0, 0, front, back), value=math.nan).unflatten(1, (b1 - b0, bs))
    gone = torch.isnan(k)
    hi = k.masked_fill(gone, -math.inf).amax(2)
    lo = k.masked_fill(gone, math.inf).amin(2)
    if front:  # the first block's earlier rows are in its stored bounds
        old = s["bounds"][:, b0].float()
        hi[:, 0] = torch.maximum(hi[:, 0], old[..., :D])
        lo[:, 0] = torch.minimum(lo[:, 0], old[..., D:])
    s["bounds"][:, b0:b1] = torch.cat([hi, lo], -1).to(DTYPES[c["dt"]])
    return s["bounds"]


def _select(s, c):
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    q = s["q"].double().view(B, Hkv, -1, D)
    r = s["bounds"].transpose(1, 2).double()  # B, Hkv, blocks, 2 D
    # max(q * hi, q * lo) is q * hi where q is positive and q * lo where it is negative
    score = torch.matmul(torch.cat([q.clamp(min=0), q.clamp(max=0)], -1), r.transpose(-1, -2)).amax(2)
    have = ((s["lens"] + c["block"] - 1) // c["block"])[:, None, None]
    at = torch.arange(r.shape[2], device="cuda")
    score = score.masked_fill((at < c["n_first"]) | (at >= have - c["n_last"]), math.inf)
    return _ascending(score.masked_fill(at >= have, -math.inf), have[:, 0, 0], c["n_sel"])


def _blocks(s, c):
    B, Hkv, D, bs = c["B"], c["Hkv"], c["D"], c["block"]
    row = s["blocks"].long()[..., None] * bs + torch.arange(bs, device="cuda")  # B, Hkv, n_sel, bs
    row = row.flatten(2)
    seen = (row >= 0) & (row < s["lens"][:, None, None])
    row = torch.where(seen, row, torch.zeros_like(row))
    b, h = torch.arange(B, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[:, None]
    k, v = s["k"][b, row, h].float(), s["v"][b, row, h].float()  # B, Hkv, n, D
    q = s["q"].float().view(B, Hkv, -1, D)
    return _softmax_rows(_scores(q, k, D, c["softcap"]), seen[:, :, None], v, DTYPES[c["dt"]])


# the library's calls -------------------------------------------------------------------
def _lib():
    from gqa_attention_lat_gb300 import binding
    return binding


def _dt(L, c):
    return L.LAT_BF16 if c["dt"] == "bf16" else L.LAT_F32


def _kept(s, n_bytes):
    """What a serving loop holds from step to step: the scratch and the status word."""
    if "scratch" not in s:
        s["scratch"] = torch.zeros(max(n_bytes, 256), dtype=torch.uint8, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s["scratch"], s["status"]


def _strides(x):
    return x.stride(1), x.stride(2), x.stride(0)


def _outputs(s, c):
    out = torch.empty(c["B"], c["Hq"] * c["D"], dtype=s["q"].dtype, device="cuda")
    return out, torch.empty(c["B"], c["Hq"], dtype=torch.float32, device="cuda")


def _own_attend(s, c):
    L = _lib()
    B, Hq, Hkv, D, cap, dt = c["B"], c["Hq"], c["Hkv"], c["D"], c["cap"], _dt(L, c)
    if "n_bytes" not in s:
        s["n_bytes"] = L.lat_attn_decode_q4_workspace_size(dt, B, Hq, Hkv, D, cap)
    ws, st = _kept(s, s["n_bytes"])
    out, lse = _outputs(s, c)
    L.lat_attn_decode_q4(dt, s["q"], s["q"].stride(0), s["cache"], *_strides(s["cache"]), s["lens"], cap, out,
                         out.stride(0), lse, B, Hq, Hkv, D, c["window"], 1.0 / math.sqrt(D), c["softcap"], ws,
                         s["n_bytes"], st)
    return out, lse


def _own_store(s, c):
    L = _lib()
    B, Hkv, D, n, m, dt = c["B"], c["Hkv"], c["D"], c["n_new"], c["pos"] + c["n_new"], _dt(L, c)
    _, st = _kept(s, 0)
    if "start" not in s:
        s["start"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    L.lat_kv_append_q4(dt, s["cache"], *_strides(s["cache"]), c["cap"], s["k_new"], s["v_new"],
                       s["k_new"].stride(0), s["pos"], n, B, Hkv, D, st)
    k, v = (torch.empty(B * m, Hkv * D, dtype=s["k_new"].dtype, device="cuda") for _ in range(2))
    L.lat_kv_expand_q4(dt, s["cache"], *_strides(s["cache"]), c["cap"], k, v, Hkv * D, s["start"], m, B, Hkv, D, st)
    return [k, v]


def _own_bounds(s, c):
    L = _lib()
    _, st = _kept(s, 0)
    L.lat_kv_block_bounds(_dt(L, c), s["k"], *_strides(s["k"]), c["cap"], s["bounds"], *_strides(s["bounds"]),
                          c["block"], s["pos"], c["n_new"], c["B"], c["Hkv"], c["D"], st)
    return s["bounds"]


def _own_select(s, c):
    L = _lib()
    B, Hq, Hkv, D, cap = c["B"], c["Hq"], c["Hkv"], c["D"], c["cap"]
    if "n_bytes" not in s:
        s["n_bytes"] = L.lat_attn_select_blocks_workspace_size(B, Hkv, c["block"], cap)
    ws, st = _kept(s, s["n_bytes"])
    blocks = torch.empty(B, Hkv, c["n_sel"], dtype=torch.int32, device="cuda")
    L.lat_attn_select_blocks(_dt(L, c), s["q"], s["q"].stride(0), s["bounds"], *_strides(s["bounds"]), c["block"],
                             s["lens"], cap, blocks, c["n_sel"], c["n_first"], c["n_last"], B, Hq, Hkv, D, ws,
                             s["n_bytes"], st)
    return blocks


def _own_blocks(s, c):
    L = _lib()
    B, Hq, Hkv, D, dt = c["B"], c["Hq"], c["Hkv"], c["D"], _dt(L, c)
    if "n_bytes" not in s:
        s["n_bytes"] = L.lat_attn_decode_blocks_workspace_size(dt, B, Hq, Hkv, D, c["block"], c["n_sel"])
    ws, st = _kept(s, s["n_bytes"])
    out, lse = _outputs(s, c)
    L.lat_attn_decode_blocks(dt, s["q"], s["q"].stride(0), s["k"], s["v"], *_strides(s["k"]), s["lens"], c["cap"],
                             c["block"], s["blocks"], c["n_sel"], out, out.stride(0), lse, B, Hq, Hkv, D,
                             1.0 / math.sqrt(D), c["softcap"], ws, s["n_bytes"], st)
    return out, lse


# --------------------------------------------------------------------- floors of one pass
def _mean_len(c):
    return (c["cap"] + 1) / 2 if c["ragged"] else c["cap"]


def work(case):
    c = case
    es = 2 if c["dt"] == "bf16" else 4
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    row4 = D + 8 * -(-D // 32)  # codes and parameters of one cached row, K and V
    if c["op"] == "store":
        n, m = c["n_new"], c["pos"] + c["n_new"]
        return {"bytes": B * Hkv * (n * (2 * D * es + row4) + m * 2 * D * es + c["pos"] * row4),
                "flops": B * Hkv * D * (12 * n + 4 * m)}
    if c["op"] == "bounds":
        b0, b1 = c["pos"] // c["block"], -(-(c["pos"] + c["n_new"]) // c["block"])
        return {"bytes": B * Hkv * D * es * (c["n_new"] + 2 * (b1 - b0) + (2 if c["pos"] % c["block"] else 0)),
                "flops": 2 * B * Hkv * D * c["n_new"]}
    io = B * c["Hq"] * (2 * D * es + 4)
    if c["op"] == "select":
        nb = _mean_len(c) / c["block"]
        return {"bytes": B * Hkv * (nb * 2 * D * es + 4 * c["n_sel"]) + B * c["Hq"] * D * es,
                "flops": 4 * B * c["Hq"] * D * nb}
    n = _mean_len(c)
    if c["op"] == "attend":
        n = min(n, c["window"]) if c["window"] > 0 else n
        return {"bytes": B * Hkv * n * row4 + io, "flops": 4 * B * c["Hq"] * D * n}
    n = min(n, c["n_sel"] * c["block"])
    return {"bytes": B * Hkv * (n * 2 * D * es + 4 * c["n_sel"]) + io, "flops": 4 * B * c["Hq"] * D * n}


# ------------------------------------------------------------ the definitions, in 64 bits
def _cached(rows, D, which):
    """Channel by channel: where the row's code lies, what its group's parameters say."""
    G = -(-D // 32)
    SG, P = min(4, G), 32 * G
    byte, shift, par = [], [], []
    for d in range(D):
        g, e = divmod(d, 32)
        st, j = divmod(g, SG)
        if which == "k":
            word, nib = (st * 4 + e // 8) * SG + j, e % 8 // 2 + 4 * (e % 2)
            byte.append(4 * word + nib // 2)
        else:
            half, nib = (st * 8 + e % 8) * SG + j, e // 8
            byte.append(P // 2 + 2 * half + nib // 2)
        shift.append(4 * (nib % 2))
        par.append(P + 4 * (g + (G if which == "v" else 0)))
    dev = rows.device
    byte, shift, par = (torch.tensor(x, device=dev) for x in (byte, shift, par))
    code = (rows[..., byte] >> shift.to(torch.uint8)) & 15

    def param(at):  # a bf16 from its two bytes
        bits = rows[..., par + at].int() | rows[..., par + at + 1].int() << 8
        return (bits << 16).view(torch.float32).double()

    return param(0) * (code.double() - (param(2) - 128))


def _attend64(q, k, v, lo, hi, D, cap):
    """One KV head group: q [G, D], k and v [n, D], keys lo .. hi-1."""
    if hi <= lo:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    x = (q @ k[lo:hi].T) * (1.0 / math.sqrt(D))
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]) @ v[lo:hi], lse


def exact(case, seed):
    c = case
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    if c["op"] == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    if c["op"] == "bounds":
        p, n, bs = c["pos"], c["n_new"], c["block"]
        k, out = s["k"].double(), s["bounds"].double().clone()
        edge = sorted({p, p + n} | {x * bs for x in range(p // bs + 1, (p + n - 1) // bs + 1)})
        for lo, hi in zip(edge, edge[1:]):
            up, dn = k[:, lo:hi].amax(1), k[:, lo:hi].amin(1)
            if lo % bs:
                up = torch.maximum(up, out[:, lo // bs, :, :D])
                dn = torch.minimum(dn, out[:, lo // bs, :, D:])
            out[:, lo // bs] = torch.cat([up, dn], -1)
        return out
    if c["op"] == "store":
        p, n = c["pos"], c["n_new"]
        got = []
        for which in ("k", "v"):
            x = s[which + "_new"].double().reshape(B, n, Hkv, D)
            y = torch.empty(B, p + n, Hkv, D, dtype=torch.float64, device="cuda")
            y[:, :p] = _cached(s["cache"][:, :p], D, which)
            for lo in range(0, D, 32):
                part = x[..., lo:lo + 32]
                low = torch.minimum(part.amin(-1, keepdim=True), torch.zeros((), dtype=torch.float64, device="cuda"))
                top = torch.maximum(part.amax(-1, keepdim=True), torch.zeros((), dtype=torch.float64, device="cuda"))
                step = ((top.float() - low.float()) / 15).bfloat16().double()
                div = torch.where(step > 0, step, torch.ones_like(step))
                z = torch.round(-low / div).clamp(0, 15)
                y[:, p:, :, lo:lo + 32] = step * ((torch.round(part / div) + z).clamp(0, 15) - z)
            got.append(y.view(B * (p + n), Hkv * D))
        return got
    q = s["q"].double().view(B, Hkv, -1, D)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(B):
        for h in range(Hkv):
            if c["op"] == "attend":
                rows = s["cache"][b, :lens[b], h]
                lo = max(0, lens[b] - c["window"]) if c["window"] > 0 else 0
                o = _attend64(q[b, h], _cached(rows, D, "k"), _cached(rows, D, "v"), lo, lens[b], D, c["softcap"])
            else:
                kept = [x for x in s["blocks"][b, h].tolist() if x >= 0]
                at = [x for n in kept for x in range(n * c["block"], min(lens[b], (n + 1) * c["block"]))]
                at = torch.tensor(at, dtype=torch.int64, device="cuda")
                o = _attend64(q[b, h], s["k"][b, at, h].double(), s["v"][b, at, h].double(), 0, len(at), D, c["softcap"])
            out[b, h], lse[b, h] = o
    return out.view(B, -1), lse.view(B, -1)
