"""The 8-bit KV cache: lat_kv_append_q8, lat_kv_expand_q8 and lat_attn_decode_q8.

Rows are compared bit for bit with the fp64 oracle's codes.  Decodes are compared with the fp64
attention oracle over the values that the rows read back as, so what 8 bits cost is no part of
the difference; bytes that no row was appended to are 0xff, a code of NaN.

Tolerances.  A decode's output is a mean of values |v| <= vmax under weights that sum to 1.  bf16:
the output is rounded once, 2^-8 vmax; each weight that meets a value is rounded to fp16, 2^-11 of
it; the scores are fp32 sums of exact products, whose error e moves every weight by a factor
e^(2e): with |q.k| sums below 64 in magnitude over 512 products e < 2^-12, 2^-11 vmax.  fp32: query
channels and weights are held to 2^-22 each, so scores of up to 64 in magnitude move by 2^-16 and
weights by 2^-15 (3.05e-5), fp32 sums and the weights' own 2^-22 by less than a third of that: 4e-5
vmax.  lse: the scores' error and its fp32 rounding, 1e-4.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import DT, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding
from oracle import q8

pytestmark = pytest.mark.gpu

HEAD_DIMS = (64, 80, 128, 256, 512)
REL = {"bf16": 2.0 ** -8 + 2.0 ** -10, "f32": 4e-5}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """An 8-bit cache [B, blocks, Hkv, record] (blocks or heads first), every byte 0xff at first."""

    def __init__(self, B, cap, Hkv, D, block=64, head_major=False, pad=0):
        self.B, self.cap, self.Hkv, self.D, self.block = B, cap, Hkv, D, block
        rb, nb = binding.lat_kv_q8_block_bytes(D, block) + pad, -(-cap // block)
        if head_major:
            t = torch.full((B, Hkv, nb, rb), 255, dtype=torch.uint8, device="cuda").transpose(1, 2)
        else:
            t = torch.full((B, nb, Hkv, rb), 255, dtype=torch.uint8, device="cuda")
        self.t = t
        self.strides = (t.stride(1), t.stride(2), t.stride(0))

    def append(self, k, v, pos, n, status=None, dt="bf16", rs=None, b0=0):
        """To sequences b0 .. b0 + len(pos) - 1."""
        st = status if status is not None else status_tensor()
        binding.lat_kv_append_q8(DT[dt], self.t[b0:], *self.strides, self.block, self.cap, k, v,
                                 self.Hkv * self.D if rs is None else rs, i32(pos), n, len(pos), self.Hkv, self.D, st)
        return st

    def expand(self, pos, n, dt="f32", status=None, pad=0):
        width = self.Hkv * self.D
        k = torch.full((self.B * n, width + pad), float("nan"), dtype=W.torch_dtype(dt), device="cuda")
        v = torch.full_like(k, float("nan"))
        st = status if status is not None else status_tensor()
        binding.lat_kv_expand_q8(DT[dt], self.t, *self.strides, self.block, self.cap, k, v, width + pad, i32(pos), n,
                                 self.B, self.Hkv, self.D, st)
        torch.cuda.synchronize()
        if pad:
            assert torch.isnan(k[:, width:].float()).all() and torch.isnan(v[:, width:].float()).all()
        return tuple(x[:, :width].reshape(self.B, n, self.Hkv, self.D) for x in (k, v))


def rows(B, n, Hkv, D, dt, seed, role):
    """Heads of unequal scale with a standing offset, as keys have."""
    x = W.normal((B, n, Hkv, D), dtype="f32", device="cuda", seed=seed, role=role)
    x = x * torch.linspace(0.3, 3.0, D, device="cuda") + torch.linspace(-1, 1, D, device="cuda")
    return x.to(W.torch_dtype(dt))


def f64(x):
    return x.float().cpu().numpy().astype(np.float64)


def held(x, block):
    """What the cache holds for rows [B, n, Hkv, D] appended in one call from row 0, by the oracle."""
    return np.stack([q8.readback(r, block) for r in f64(x)])


def assert_same(got, want, what):
    g, w = f64(got), np.asarray(want)
    assert np.array_equal(np.isnan(g), np.isnan(w)), what + ": NaN pattern"
    assert np.array_equal(g[~np.isnan(w)], w[~np.isnan(w)]), what


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,block,calls,head_major", [
    (1, 1, 16, [1], False), (2, 3, 16, [5, 1, 40], True), (2, 2, 32, [33, 31, 1, 1], False),
    (1, 5, 64, [130, 62, 3], True), (2, 1, 128, [100, 27, 1, 131], False)])
def test_rows_read_back_as_the_oracle_says(D, dt, B, Hkv, block, calls, head_major):
    """Several appends one after another, larger rows later, at other rows of each sequence."""
    n, start = sum(calls), [0, 2 * block][:B]
    cap = n + 2 * block + 5
    c = Cache(B, cap, Hkv, D, block, head_major, pad=32 if Hkv == 2 else 0)
    want = [[q8.Rows(cap, Hkv, D, block) for _ in range(2)] for _ in range(B)]
    st, at = status_tensor(), 0
    for i, m in enumerate(calls):
        k, v = (rows(B, m, Hkv, D, dt, 10 * D + i, r) * 2.0 ** (2 * i) for r in ("k", "v"))
        c.append(k.reshape(B * m, -1), v.reshape(B * m, -1), [s + at for s in start], m, st, dt)
        for b in range(B):
            for r, x in zip(want[b], (k, v)):
                r.append(f64(x[b]), start[b] + at)
        at += m
    for out in ("f32", "bf16"):
        gk, gv = c.expand(start, n, out, st, pad=0 if Hkv == 1 else 8)
        assert int(st.item()) == 0
        for b in range(B):
            assert_same(gk[b], want[b][0].value[start[b]:start[b] + n], "K")
            assert_same(gv[b], want[b][1].value[start[b]:start[b] + n], "V")
    # nothing in the blocks beside, behind the last row, nor between the records
    size = block * 2 * D
    for b in range(B):
        first, last = start[b] // block, (start[b] + n - 1) // block
        assert (c.t[b, :first] == 255).all() and (c.t[b, last + 1:] == 255).all()
        used = (start[b] + n - last * block) * 2 * D
        assert (c.t[b, last, :, used:size] == 255).all()
        assert (c.t[b, first:last + 1, :, size + 8:] == 255).all()


@pytest.mark.parametrize("dt,rs_pad,shift", [("bf16", 1, 0), ("bf16", 0, 1), ("f32", 3, 0), ("f32", 0, 1)])
def test_rows_at_odd_strides_and_addresses(dt, rs_pad, shift):
    B, n, Hkv, D = 2, 9, 3, 80
    rs = Hkv * D + rs_pad
    k, v = (rows(B, n, Hkv, D, dt, 5, r) for r in ("k", "v"))

    def odd(x):
        buf = torch.full((B * n * rs + 8,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf[shift:shift + B * n * rs].view(B * n, rs)
        view[:, :Hkv * D] = x.reshape(B * n, Hkv * D)
        return view

    c = Cache(B, 48, Hkv, D, 16)
    st = c.append(odd(k), odd(v), [0, 32], n, dt=dt, rs=rs)
    gk, gv = c.expand([0, 32], n, dt, st, pad=rs_pad)
    assert int(st.item()) == 0
    assert_same(gk, held(k, 16), "K")
    assert_same(gv, held(v, 16), "V")


def test_blocks_at_the_edges_of_the_numbers():
    """Zeros, tiny, subnormal and huge blocks, NaN and infinities among others, ties."""
    x = torch.zeros(13 * 16, 128)
    r = torch.randn(16, 128, generator=torch.Generator().manual_seed(3))
    fill = [0 * r, r.abs(), -r.abs(), 0 * r + 7.0, r * 2.0 ** -133, r * 2.0 ** -141, r * 2.0 ** 120, 0 * r + 3.3e38,
            r.clone(), r.clone(), r.clone(), 0 * r, torch.arange(16 * 128).view(16, 128) / 16.0]
    fill[8][3, 40] = float("nan")
    fill[9][5, 100] = float("inf")
    fill[10][0, 5], fill[10][0, 6] = float("-inf"), float("nan")
    fill[11][0, 0], fill[11][1, 1], fill[11][2, 2] = 1e-30, -1e30, 448.0
    for i, f in enumerate(fill):
        x[16 * i:16 * i + 16] = f
    for dt in ("f32", "bf16"):
        k = x.to(W.torch_dtype(dt)).cuda().view(1, -1, 1, 128)
        v = k.flip(-1).contiguous()
        c = Cache(1, len(x), 1, 128, 16)
        st = c.append(k, v, [0], len(x), dt=dt)
        gk, gv = c.expand([0], len(x), "f32", st)
        assert int(st.item()) == 0
        assert_same(gk, held(k, 16), "K " + dt)
        assert_same(gv, held(v, 16), "V " + dt)


def test_a_sequence_out_of_range_is_skipped_whole():
    B, n, Hkv, D, cap = 4, 5, 2, 64, 21
    pos = [16, 17, -1, 2 ** 31 - 3]  # only the first fits
    c = Cache(B, cap, Hkv, D, 16)
    k, v = rows(B, n, Hkv, D, "bf16", 1, "k"), rows(B, n, Hkv, D, "bf16", 1, "v")
    st = c.append(k, v, pos, n)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert (c.t[1:] == 255).all() and (c.t[0, 0] == 255).all()
    st = status_tensor()
    gk, gv = c.expand(pos, n, "f32", st)
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert_same(gk[:1], held(k[:1], 16), "K")
    assert torch.isnan(gk[1:]).all() and torch.isnan(gv[1:]).all()


def decode(c, q, lens, dt, Hq, window=0, softcap=0.0, scale=None, max_len=None, out_pad=0, stream=None,
           ws=None, status=None, out=None, lse=None):
    D = c.D
    mk = c.cap if max_len is None else max_len
    nb = binding.lat_attn_decode_q8_workspace_size(DT[dt], c.B, Hq, c.Hkv, D, mk)
    assert nb > 0
    if ws is None:
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((c.B, Hq * D + out_pad), float("nan"), dtype=q.dtype, device="cuda")
    if lse is None:
        lse = torch.full((c.B, Hq), float("nan"), device="cuda")
    st = status if status is not None else status_tensor()
    binding.lat_attn_decode_q8(DT[dt], q, q.stride(0), c.t, *c.strides, c.block, lens, mk, out, out.stride(0), lse,
                               c.B, Hq, c.Hkv, D, window, D ** -0.5 if scale is None else scale, softcap, ws, nb, st,
                               stream=stream)
    return out, lse, st


def check_decode(out, lse, q, kh, vh, lens, dt, Hq, D, window, softcap, what, scale=None, times=1):
    B = q.shape[0]
    ref, ref_lse = oracle.decode(q[:, :Hq * D].reshape(B, Hq, D), kh, vh, lens, window=window,
                                 scale=D ** -0.5 if scale is None else scale, softcap=softcap)
    got = out[:, :Hq * D].double().cpu().numpy().reshape(B, Hq, D)
    assert np.isfinite(got).all(), what
    vmax = max((np.abs(vh[b, :n]).max() for b, n in enumerate(lens) if n), default=0.0)
    err = np.abs(got - ref).max()
    assert err <= times * REL[dt] * vmax, "%s: %.3e of %.3e" % (what, err, REL[dt] * vmax)
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l), np.isneginf(ref_lse)), what
    fin = np.isfinite(ref_lse)
    assert not fin.any() or np.abs(l[fin] - ref_lse[fin]).max() <= times * 1e-4, what


def filled(B, cap, Hkv, D, lens, dt, seed, block=64, head_major=False):
    """A cache with lens[b] rows a sequence, and what it holds (zeros behind them)."""
    c = Cache(B, cap, Hkv, D, block, head_major)
    k, v = rows(B, cap, Hkv, D, dt, seed, "k"), rows(B, cap, Hkv, D, dt, seed, "v")
    kh, vh = np.zeros((2, B, cap, Hkv, D))
    for b, n in enumerate(lens):
        if n:
            c.append(k[b, :n].contiguous(), v[b, :n].contiguous(), [0], n, dt=dt, b0=b)
            kh[b, :n], vh[b, :n] = held(k[b:b + 1, :n], block)[0], held(v[b:b + 1, :n], block)[0]
    return c, kh, vh


# (B, Hq, Hkv, D, cap, lens, window, softcap, block, head_major)
SHAPES = [
    (1, 1, 1, 64, 1, [1], 0, 0.0, 16, False),
    (6, 4, 2, 64, 300, [0, 1, 15, 16, 17, 300], 0, 0.0, 32, False),
    (5, 16, 2, 128, 700, [31, 32, 33, 129, 700], 0, 0.0, 64, True),
    (3, 10, 2, 80, 515, [515, 128, 511], 200, 0.0, 16, False),
    (3, 12, 1, 128, 400, [400, 399, 7], 0, 30.0, 16, False),   # 12 heads: two blocks of a unit
    (2, 24, 2, 256, 333, [333, 100], 65, 50.0, 128, True),
    (2, 16, 2, 512, 260, [260, 63], 0, 0.0, 32, False),
    (2, 3, 1, 512, 129, [129, 65], 1, 0.0, 64, True),          # a window of one key
    (40, 8, 8, 64, 90, [1 + (37 * b) % 90 for b in range(40)], 0, 0.0, 128, False),
    (2, 8, 2, 128, 800, [800, 799], 129, 0.0, 128, False),     # windows that begin inside a copy
    (1, 8, 1, 128, 9000, [8999], 0, 0.0, 64, False),           # one unit over every CTA
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dH%d-%dD%dL%dW%dC%gb%d%s" % (
    s[0], s[1], s[2], s[3], s[4], s[6], s[7], s[8], "h" if s[9] else ""))
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_matches_the_oracle(shape, dt):
    B, Hq, Hkv, D, cap, lens, window, softcap, block, hm = shape
    c, kh, vh = filled(B, cap, Hkv, D, lens, dt, 100 + D, block, hm)
    full = W.normal((B, Hq * D + 16), dtype=dt, device="cuda", seed=D, role="q")
    q = full[:, :Hq * D]
    out, lse, st = decode(c, q, i32(lens), dt, Hq, window, softcap, out_pad=16)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(out[:, Hq * D:].float()).all()
    check_decode(out, lse, q, kh, vh, lens, dt, Hq, D, window, softcap, str(shape))


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("G,block,window", [(1, 16, 0), (5, 64, 0), (8, 128, 33)])
def test_every_length_around_a_tile(D, G, block, window):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 95, 96, 97, 127, 128, 129, 130, 255, 256, 257]
    B, Hkv, cap = len(lens), 1, 257
    c, kh, vh = filled(B, cap, Hkv, D, lens, "bf16", 7 * D, block)
    q = W.normal((B, G * D), dtype="bf16", device="cuda", seed=G, role="q")
    out, lse, st = decode(c, q, i32(lens), "bf16", G, window)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, kh, vh, lens, "bf16", G, D, window, 0.0, "D%d G%d" % (D, G))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_sequences_most_of_them_empty(dt):
    """More sequences than a CTA has threads, zero to 70 keys each, over a capacity above
    max_kv_len: the shares cross many short units."""
    B, Hq, Hkv, D, cap = 700, 4, 2, 64, 96
    g = torch.Generator().manual_seed(11)
    lens = (torch.randint(0, 71, (B,), generator=g) * (torch.rand(B, generator=g) < 0.4)).tolist()
    c = Cache(B, cap, Hkv, D, 32)
    k, v = rows(B, cap, Hkv, D, dt, 1, "k"), rows(B, cap, Hkv, D, dt, 1, "v")
    c.append(k, v, [0] * B, cap, dt=dt)
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q")
    out, lse, st = decode(c, q, i32(lens), dt, Hq, max_len=71)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, held(k, 32), held(v, 32), lens, dt, Hq, D, 0, 0.0, "many")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("q_mul,k_mul,scale", [(1.0, 1.0, 0.0), (1.0, 1.0, -0.1), (2.0 ** 110, 2.0 ** -90, 2.0 ** -23),
                                               (2.0 ** -112, 2.0 ** 112, 0.4), (2.0 ** -9, 1.0, 50.0)])
def test_scales_at_the_edges_of_the_numbers(dt, q_mul, k_mul, scale):
    """Scale zero and below; queries and keys far from 1 whose products are not."""
    B, Hq, Hkv, D, cap = 2, 4, 1, 128, 200
    k, v = rows(B, cap, Hkv, D, "f32", 1, "k") * k_mul, rows(B, cap, Hkv, D, "f32", 1, "v")
    q = W.normal((B, Hq * D), dtype="f32", device="cuda", seed=2, role="q") * q_mul
    k, v, q = (x.to(W.torch_dtype(dt)) for x in (k, v, q))
    c = Cache(B, cap, Hkv, D, 64)
    c.append(k, v, [0] * B, cap, dt=dt)
    lens = [200, 3]
    out, lse, st = decode(c, q, i32(lens), dt, Hq, scale=scale)
    torch.cuda.synchronize()
    # (a larger scale magnifies the scores' error: their magnitude stays below 2^7 here)
    check_decode(out, lse, q, held(k, 64), held(v, 64), lens, dt, Hq, D, 0, 0.0, "edges", scale=scale, times=2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_blocks_of_very_different_size(dt):
    """Values that differ by 2^60 from block to block, and keys whose scores hide either.  The error
    is measured against what the weights leave of each sequence's values."""
    B, Hq, Hkv, D, cap, block = 4, 4, 1, 128, 512, 16
    k, v = rows(B, cap, Hkv, D, "f32", 1, "k"), rows(B, cap, Hkv, D, "f32", 1, "v")
    v = v * torch.where(torch.arange(cap, device="cuda") // 16 % 2 == 0, 2.0 ** -30, 2.0 ** 30).view(1, cap, 1, 1)
    k[1] = k[1] * 0.01
    q = W.normal((B, Hq * D), dtype="f32", device="cuda", seed=2, role="q")
    # sequence 2: the large blocks lie 50 below in score, so that the small ones are all of it
    direction = torch.randn(D, generator=torch.Generator().manual_seed(1)).cuda()
    direction = direction / direction.norm()
    q[2:] = (8.0 * direction).repeat(2, Hq)
    even = (torch.arange(cap, device="cuda") // 16 % 2 == 0).float().view(cap, 1, 1)
    k[2] = even * (50.0 * direction * D ** 0.5 / 8)
    v[3, 16:] = 0.0  # all but the first block (of small values) nothing at all
    k, v, q = (x.to(W.torch_dtype(dt)) for x in (k, v, q))
    c = Cache(B, cap, Hkv, D, block)
    c.append(k, v, [0] * B, cap, dt=dt)
    lens = [cap] * B
    out, lse, st = decode(c, q, i32(lens), dt, Hq)
    torch.cuda.synchronize()
    kh, vh = held(k, block), held(v, block)
    ref, ref_lse = oracle.decode(q.view(B, Hq, D), kh, vh, lens, window=0, scale=D ** -0.5)
    mag, _ = oracle.decode(q.view(B, Hq, D), kh, np.abs(vh), lens, window=0, scale=D ** -0.5)
    got = out.double().cpu().numpy().reshape(B, Hq, D)
    # relative to the mean of the values' magnitudes under the same weights
    assert (np.abs(got - ref) <= 2 * REL[dt] * mag).all()
    assert np.abs(lse.double().cpu().numpy() - ref_lse).max() <= 1e-4


def test_nan_in_a_visible_row_and_in_the_query():
    """A NaN value makes its channel NaN and no other; a NaN key or query, the head."""
    B, Hq, Hkv, D, cap = 3, 2, 1, 128, 64
    k, v = rows(B, cap, Hkv, D, "bf16", 1, "k"), rows(B, cap, Hkv, D, "bf16", 1, "v")
    v[0, 5, 0, 40] = float("nan")
    k[1, 7, 0, 3] = float("inf")
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=2, role="q")
    q[2, 3] = float("nan")  # head 0
    c = Cache(B, cap, Hkv, D, 32)
    c.append(k, v, [0] * B, cap)
    out, lse, st = decode(c, q, torch.full((B,), cap, dtype=torch.int32, device="cuda"), "bf16", Hq)
    bad = torch.isnan(out.view(B, Hq, D))
    assert bad[0, :, 40].all() and int(bad[0].sum()) == Hq
    assert bad[1].all() and bad[2, 0].all() and not bad[2, 1].any()


def test_nan_before_the_window_does_not_show():
    B, Hq, Hkv, D, cap, window = 2, 4, 1, 128, 300, 150
    k, v = rows(B, cap, Hkv, D, "bf16", 1, "k"), rows(B, cap, Hkv, D, "bf16", 1, "v")
    lens = [300, 291]
    for b, n in enumerate(lens):
        k[b, :n - window] = float("nan")
        v[b, :n - window] = float("nan")
    c = Cache(B, cap, Hkv, D, 64)
    c.append(k, v, [0] * B, cap)
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=2, role="q")
    out, lse, st = decode(c, q, i32(lens), "bf16", Hq, window)
    torch.cuda.synchronize()
    kh, vh = np.nan_to_num(held(k, 64)), np.nan_to_num(held(v, 64))
    check_decode(out, lse, q, kh, vh, lens, "bf16", Hq, D, window, 0.0, "window")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [300, 9000])
def test_scores_below_the_least_float_weigh_nothing(dt, cap):
    """Whole pieces of a sequence whose scores leave fp32's range on the low side."""
    B, Hq, Hkv, D = 3, 4, 1, 128
    k, v = rows(B, cap, Hkv, D, dt, 1, "k"), rows(B, cap, Hkv, D, dt, 1, "v")
    k[0, :cap - 44] = -2.9e38  # (blocks of 16 rows: the others keep their scale)
    k[1, 48:] = -2.9e38
    k[2, 96:cap - 92] = -2.9e38
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q").abs()  # sums of 128 terms near -3e38
    c = Cache(B, cap, Hkv, D, 16)
    c.append(k, v, [0] * B, cap, dt=dt)
    lens = [cap] * B
    out, lse, st = decode(c, q, i32(lens), dt, Hq)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, held(k, 16), held(v, 16), lens, dt, Hq, D, 0, 0.0, "low scores")


def test_lengths_out_of_range_leave_their_rows_alone():
    B, Hq, Hkv, D, cap = 4, 4, 2, 128, 64
    lens = [64, 65, -1, 10]
    c, kh, vh = filled(B, cap, Hkv, D, [64, 64, 64, 10], "bf16", 3)
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=9, role="q")
    out, lse, st = decode(c, q, i32(lens), "bf16", Hq)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert torch.isnan(out[1:3].float()).all() and torch.isnan(lse[1:3]).all()
    keep = [0, 3]
    check_decode(out[keep], lse[keep], q[keep], kh[keep], vh[keep], [64, 10], "bf16", Hq, D, 0, 0.0, "kept")


def test_a_long_cache_past_32_bit_offsets():
    """Two sequences of 2.2e9 bytes, written and read at their far ends."""
    B, Hq, Hkv, D, cap = 2, 8, 1, 512, 2_200_000  # 1024 bytes a row
    c = Cache(B, cap, Hkv, D, 32)
    n = 288
    at = cap // 32 * 32 - n
    k, v = rows(B, n, Hkv, D, "bf16", 1, "k"), rows(B, n, Hkv, D, "bf16", 1, "v")
    st = c.append(k, v, [at, at], n)
    gk, gv = c.expand([at, at], n, "f32", st)
    kh, vh = held(k, 32), held(v, 32)
    assert_same(gk, kh, "K")
    assert_same(gv, vh, "V")
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=9, role="q")
    out, lse, st = decode(c, q, i32([at + n] * B), "bf16", Hq, window=n, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, kh, vh, [n, n], "bf16", Hq, D, 0, 0.0, "far end")


def test_chunks_prefill_and_steps_together():
    """As a server uses it: two chunks of a prompt (append, read back, prefill), then steps
    (append one token, decode), on a stream of its own, the step captured and replayed."""
    B, Hq, Hkv, D, cap, chunk, steps, block = 2, 8, 2, 128, 256, 96, 5, 64
    total = 2 * chunk + steps
    k, v = rows(B, total, Hkv, D, "bf16", 21, "k"), rows(B, total, Hkv, D, "bf16", 21, "v")
    k[:, -2:] *= 4  # the last tokens raise their block's scale
    q = W.normal((B, total, Hq * D), dtype="bf16", device="cuda", seed=21, role="q")
    want = [[q8.Rows(cap, Hkv, D, block) for _ in range(2)] for _ in range(B)]

    def note(p0, n):
        for b in range(B):
            want[b][0].append(f64(k[b, p0:p0 + n]), p0)
            want[b][1].append(f64(v[b, p0:p0 + n]), p0)

    def now(i):
        return np.nan_to_num(np.stack([w[i].value for w in want]))

    c = Cache(B, cap, Hkv, D, block)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st = status_tensor()
        for p0 in (0, chunk):
            c.append(k[:, p0:p0 + chunk].contiguous(), v[:, p0:p0 + chunk].contiguous(), [p0] * B, chunk, st)
            note(p0, chunk)
            n = p0 + chunk
            gk, gv = c.expand([0] * B, n, "bf16", st)
            assert_same(gk, now(0)[:, :n], "K")
            gk, gv = gk.reshape(B * n, Hkv * D), gv.reshape(B * n, Hkv * D)
            qc = q[:, p0:n].reshape(B * chunk, Hq * D)
            out = torch.empty_like(qc)
            binding.lat_attn_prefill(binding.LAT_BF16, qc, Hq * D, gk, Hkv * D, gv, Hkv * D, out, Hq * D, None, B,
                                     chunk, n, Hq, Hkv, D, 1, 0, D ** -0.5, st)
            s.synchronize()
            ref, _ = oracle.prefill(qc.view(B, chunk, Hq, D), gk.view(B, n, Hkv, D), gv.view(B, n, Hkv, D),
                                    causal=True, window=0, scale=D ** -0.5)
            assert np.abs(out.float().cpu().numpy().reshape(ref.shape) - ref).max() <= 2.0 ** -7 * np.abs(now(1)).max()
        qs, lens = torch.empty(B, Hq * D, dtype=q.dtype, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        nb = binding.lat_attn_decode_q8_workspace_size(binding.LAT_BF16, B, Hq, Hkv, D, cap)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        out = torch.empty(B, Hq * D, dtype=q.dtype, device="cuda")
        lse = torch.empty(B, Hq, device="cuda")
        pos = torch.zeros(B, dtype=torch.int32, device="cuda")
        kn, vn = (torch.empty(B, Hkv * D, dtype=q.dtype, device="cuda") for _ in range(2))

        def step():
            binding.lat_kv_append_q8(binding.LAT_BF16, c.t, *c.strides, block, cap, kn, vn, Hkv * D, pos, 1, B, Hkv, D,
                                     st)
            decode(c, qs, lens, "bf16", Hq, ws=ws, status=st, out=out, lse=lse)

        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            step()
        for t in range(2 * chunk, total):
            kn.copy_(k[:, t].reshape(B, -1))
            vn.copy_(v[:, t].reshape(B, -1))
            qs.copy_(q[:, t])
            pos.fill_(t)
            lens.fill_(t + 1)
            note(t, 1)
            graph.replay()
            s.synchronize()
            check_decode(out, lse, qs, now(0), now(1), [t + 1] * B, "bf16", Hq, D, 0, 0.0, "step %d" % t)
        assert int(st.item()) == 0


def test_two_streams_with_a_workspace_each():
    B, Hq, Hkv, D, cap = 3, 16, 4, 128, 5000
    lens = [5000, 1, 2777]
    c, kh, vh = filled(B, cap, Hkv, D, lens, "bf16", 33)
    lt = i32(lens)
    qs = [W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=i, role="q") for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[] for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(decode(c, qs[i], lt, "bf16", Hq, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse, st in got[i]:
            assert int(st.item()) == 0
            assert torch.equal(out, got[i][0][0]) and torch.equal(lse, got[i][0][1])  # no order of joins shows
        check_decode(got[i][0][0], got[i][0][1], qs[i], kh, vh, lens, "bf16", Hq, D, 0, 0.0, "stream %d" % i)


@pytest.mark.parametrize("D", HEAD_DIMS)
def test_32_bit_sums_lean_to_no_side(D):
    """Long shares of values around 0, in LAT_F32: the root mean square of the output's error.

    A weight's error: four roundings of a score below 16 in magnitude (its sum, its scale, its
    distance from the reference, what the exponential takes), each at most 2^-21, root mean square
    2^-21 / sqrt(3), 3.8e-7 of the weight in all; the exponential's own 2^-22 and the two fp16 terms'
    2^-23, 2.7e-7 together at their most.  Errors of the weights that have no common sign move a sum of
    values around 0 by as much of itself: 4.7e-7 (the squares add up).  Each rounded add of the sum moves it by 2^-24 /
    sqrt(3) at most, 128 of them by 3.9e-7.  6.1e-7 in all, and 1e-6 leaves room for the output's
    being smaller than its share of the weights says.  (Sums cut off toward zero lose 128 * 2^-24 =
    7.6e-6.)"""
    B, Hkv, G, n = (76, 2, 1, 8192) if D < 512 else (38, 2, 1, 4096)
    c = Cache(B, n, Hkv, D, 64)
    for b in range(B):
        kb, vb = (W.normal((1, n, Hkv, D), dtype="f32", device="cuda", seed=900 + b, role=r) for r in ("k", "v"))
        c.append(kb, vb, [0], n, dt="f32", b0=b)
    k, v = c.expand([0] * B, n)
    q = W.normal((B, Hkv * G * D), dtype="f32", device="cuda", seed=77, role="q")
    out = decode(c, q, i32([n] * B), "f32", Hkv * G)[0]
    got, q = out.reshape(B, Hkv, D).double(), q.reshape(B, Hkv, D).double()
    wrong = size = 0.0
    for b in range(B):
        s = torch.einsum("hd,nhd->hn", q[b], k[b].double()) / math.sqrt(D)
        want = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), v[b].double())
        assert s.abs().max().item() * math.log2(math.e) < 16
        wrong, size = wrong + (got[b] - want).square().sum().item(), size + want.square().sum().item()
    assert math.sqrt(wrong / size) <= 1e-6


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nothing_cached_anywhere(dt):
    """max_kv_len 0, and caches of every length 0: zeros and -inf, no read of the cache."""
    B, Hq, Hkv, D, cap = 3, 4, 2, 64, 16
    c = Cache(B, cap, Hkv, D, 16)
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=1, role="q")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for mk in (0, cap):
        out, lse, st = decode(c, q, lens, dt, Hq, max_len=mk)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and (out == 0).all() and torch.isneginf(lse).all()


# (B, Hq, Hkv, D, cap): units joined by tickets, whole, and joined by a second kernel
@pytest.mark.parametrize("shape", [(40, 8, 2, 64, 3000), (3, 8, 2, 80, 700), (1, 8, 1, 128, 9000),
                                   (2, 16, 1, 512, 4000), (4, 4, 4, 64, 200)], ids=lambda s: "B%dH%d-%dD%dL%d" % s)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_the_waits_run_out(shape, dt):
    """A hook never brings a CTA's first rows: every CTA records LAT_ERR_TIMEOUT, drains its copies
    and exits.  Then the same buffers, a re-zeroed workspace and the regular call are right."""
    B, Hq, Hkv, D, cap = shape
    lens = [cap - 7 * (b % 3) for b in range(B)]
    c, kh, vh = filled(B, cap, Hkv, D, lens, dt, 3)
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q")
    nb = binding.lat_attn_decode_q8_workspace_size(DT[dt], B, Hq, Hkv, D, cap)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    out = torch.zeros(B, Hq * D, dtype=q.dtype, device="cuda")
    st, lt = status_tensor(), i32(lens)
    binding.lat_test_decode_q8_timeout(DT[dt], q, q.stride(0), c.t, *c.strides, c.block, lt, cap, out, out.stride(0),
                                       B, Hq, Hkv, D, ws, nb, 20_000_000, st)
    torch.cuda.synchronize()  # the kernels end by themselves: no fault, no hang
    assert int(st.item()) == binding.LAT_ERR_TIMEOUT
    ws.zero_()
    out, lse, st = decode(c, q, lt, dt, Hq, ws=ws)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, kh, vh, lens, dt, Hq, D, 0, 0.0, "after a timeout")
