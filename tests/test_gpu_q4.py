"""The 4-bit KV cache: lat_kv_append_q4, lat_kv_expand_q4 and lat_attn_decode_q4.

Rows are compared bit for bit with the fp64 oracle's quantisation.  Decodes are compared
with the fp64 attention oracle over the values that the rows read back as, so what 4 bits
cost is no part of the difference; slots past a sequence's length hold bytes of 0xff.

Tolerances.  A decode's output is a mean of values |v| <= vmax under weights that sum to 1.
bf16: each weight is rounded once to bf16 (2^-9 relative, half a step of 8 bits), which moves
the mean by at most 2^-8 vmax / 2, and the output once more: together 2^-8 vmax.  The scores
are fp32 sums of exact products: their error e moves every weight by a factor e^(2e); with
|q.k| sums below 64 in magnitude over 512 products, e < 2^-12, 2^-11 vmax in all.  fp32: no
rounding to bf16 remains, the same score error alone, which at the sizes here (terms below
2^6, products summed in fp32) stays under 2e-5 vmax.  lse: the score error and its fp32
rounding, 1e-4.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import DT, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding
from oracle import q4

pytestmark = pytest.mark.gpu

HEAD_DIMS = (64, 80, 128, 256, 512)
REL = {"bf16": 2.0 ** -8 + 2.0 ** -11, "f32": 2e-5}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


class Cache:
    """A 4-bit cache [B, cap, Hkv, row] (token- or head-major), every byte 0xff at first."""

    def __init__(self, B, cap, Hkv, D, head_major=False, pad=0):
        self.B, self.cap, self.Hkv, self.D = B, cap, Hkv, D
        rb = binding.lat_kv_q4_row_bytes(D) + pad
        if head_major:
            t = torch.full((B, Hkv, cap, rb), 255, dtype=torch.uint8, device="cuda").transpose(1, 2)
        else:
            t = torch.full((B, cap, Hkv, rb), 255, dtype=torch.uint8, device="cuda")
        self.t = t
        self.strides = (t.stride(1), t.stride(2), t.stride(0))

    def append(self, k, v, pos, n, status=None, stream=None, dt="bf16", rs=None):
        st = status if status is not None else status_tensor()
        p = torch.tensor(pos, dtype=torch.int32, device="cuda")
        binding.lat_kv_append_q4(DT[dt], self.t, *self.strides, self.cap, k, v,
                                 self.Hkv * self.D if rs is None else rs, p, n, self.B, self.Hkv, self.D,
                                 st, stream=stream)
        return st

    def expand(self, pos, n, dt="f32", status=None, pad=0):
        tdt = W.torch_dtype(dt)
        width = self.Hkv * self.D
        k = torch.full((self.B * n, width + pad), float("nan"), dtype=tdt, device="cuda")
        v = torch.full_like(k, float("nan"))
        st = status if status is not None else status_tensor()
        p = torch.tensor(pos, dtype=torch.int32, device="cuda")
        binding.lat_kv_expand_q4(DT[dt], self.t, *self.strides, self.cap, k, v, width + pad, p, n, self.B,
                                 self.Hkv, self.D, st)
        torch.cuda.synchronize()
        if pad:
            assert torch.isnan(k[:, width:].float()).all() and torch.isnan(v[:, width:].float()).all()
        return tuple(x[:, :width].reshape(self.B, n, self.Hkv, self.D) for x in (k, v))


def rows(B, n, Hkv, D, dt, seed, role):
    """Heads of unequal scale with a standing offset, as keys have."""
    x = W.normal((B, n, Hkv, D), dtype="f32", device="cuda", seed=seed, role=role)
    x = x * torch.linspace(0.3, 3.0, D, device="cuda") + torch.linspace(-1, 1, D, device="cuda")
    return x.to(W.torch_dtype(dt))


def held(x):
    """What the cache holds for the rows x, by the oracle."""
    return q4.readback(x.float().cpu().numpy())


def assert_held(got, x, what):
    want = torch.from_numpy(held(x)).to(got.dtype)  # one rounding to the output's type
    g = got.cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what + ": NaN pattern"
    assert torch.equal(g[~torch.isnan(g)], want[~torch.isnan(want)]), what


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,n,head_major", [(1, 1, 1, False), (3, 2, 37, True), (2, 5, 64, False)])
def test_rows_read_back_as_the_oracle_says(D, dt, B, Hkv, n, head_major):
    cap = n + 11
    pos = [min(11, 3 * b) for b in range(B)]
    c = Cache(B, cap, Hkv, D, head_major, pad=16 if Hkv == 2 else 0)
    k, v = rows(B, n, Hkv, D, dt, D, "k"), rows(B, n, Hkv, D, dt, D + 1, "v")
    st = c.append(k, v, pos, n, dt=dt)
    for out in ("f32", dt):
        gk, gv = c.expand(pos, n, out, st, pad=0 if Hkv == 1 else 8)
        assert int(st.item()) == 0
        assert_held(gk, k, "K")
        assert_held(gv, v, "V")
    # nothing outside the appended rows, nor between the rows
    rb = binding.lat_kv_q4_row_bytes(D)
    for b in range(B):
        assert (c.t[b, :pos[b]] == 255).all() and (c.t[b, pos[b] + n:] == 255).all()
    assert (c.t[..., rb:] == 255).all()


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

    c = Cache(B, 16, Hkv, D)
    st = c.append(odd(k), odd(v), [0, 7], n, dt=dt, rs=rs)
    gk, gv = c.expand([0, 7], n, dt, st, pad=rs_pad)
    assert int(st.item()) == 0
    assert_held(gk, k, "K")
    assert_held(gv, v, "V")


def test_groups_at_the_edges_of_the_numbers():
    """Zero, one-sided, constant, tiny (subnormal), huge, over-ranged, NaN and infinite groups,
    one beside another; each in K and in V."""
    x = torch.zeros(12, 128)
    r = torch.randn(128, generator=torch.Generator().manual_seed(3))
    x[1] = r.abs()
    x[2] = -r.abs()
    x[3] = 7.0
    x[4] = r * 2.0 ** -133
    x[5] = r * 2.0 ** -141
    x[6] = r * 2.0 ** 120
    x[7, 0], x[7, 1] = 3e38, -3e38        # finite, but its range is not
    x[8] = r
    x[8, 40] = float("nan")
    x[9] = r
    x[9, 100] = float("inf")
    x[10] = r
    x[10, 5], x[10, 6] = float("-inf"), float("nan")
    x[11, 31], x[11, 32] = 1e-30, -1e30
    for dt in ("f32", "bf16"):
        k = x.to(W.torch_dtype(dt)).cuda().view(1, 12, 1, 128)
        v = k.flip(-1).contiguous()
        c = Cache(1, 12, 1, 128)
        st = c.append(k, v, [0], 12, dt=dt)
        gk, gv = c.expand([0], 12, "f32", st)
        assert int(st.item()) == 0
        assert_held(gk, k, "K " + dt)
        assert_held(gv, v, "V " + dt)


def test_a_sequence_out_of_range_is_skipped_whole():
    B, n, Hkv, D, cap = 4, 5, 2, 64, 12
    pos = [7, 8, -1, 2 ** 31 - 3]  # only the first fits
    c = Cache(B, cap, Hkv, D)
    k, v = rows(B, n, Hkv, D, "bf16", 1, "k"), rows(B, n, Hkv, D, "bf16", 1, "v")
    st = c.append(k, v, pos, n)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert (c.t[1:] == 255).all() and (c.t[0, :7] == 255).all()
    st = status_tensor()
    gk, gv = c.expand(pos, n, "f32", st)
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert_held(gk[:1], k[:1], "K")
    assert torch.isnan(gk[1:]).all() and torch.isnan(gv[1:]).all()


def decode(c, q, lens, dt, Hq, window=0, softcap=0.0, scale=None, max_len=None, out_pad=0, stream=None,
           ws=None, status=None, out=None, lse=None):
    D = c.D
    mk = c.cap if max_len is None else max_len
    nb = binding.lat_attn_decode_q4_workspace_size(DT[dt], c.B, Hq, c.Hkv, D, mk)
    assert nb > 0
    if ws is None:
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((c.B, Hq * D + out_pad), float("nan"), dtype=q.dtype, device="cuda")
    if lse is None:
        lse = torch.full((c.B, Hq), float("nan"), device="cuda")
    st = status if status is not None else status_tensor()
    binding.lat_attn_decode_q4(DT[dt], q, q.stride(0), c.t, *c.strides, lens, mk, out, out.stride(0), lse, c.B,
                               Hq, c.Hkv, D, window, D ** -0.5 if scale is None else scale, softcap, ws, nb, st,
                               stream=stream)
    return out, lse, st


def check_decode(out, lse, q, kh, vh, lens, dt, Hq, D, window, softcap, what):
    B = q.shape[0]
    ref, ref_lse = oracle.decode(q[:, :Hq * D].reshape(B, Hq, D), kh, vh, lens, window=window, scale=D ** -0.5,
                                 softcap=softcap)
    got = out[:, :Hq * D].double().cpu().numpy().reshape(B, Hq, D)
    assert np.isfinite(got).all(), what
    vmax = np.abs(vh).max()
    err = np.abs(got - ref).max()
    assert err <= REL[dt] * vmax, "%s: %.3e of %.3e" % (what, err, REL[dt] * vmax)
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l), np.isneginf(ref_lse)), what
    fin = np.isfinite(ref_lse)
    assert not fin.any() or np.abs(l[fin] - ref_lse[fin]).max() <= 1e-4, what


def filled(B, cap, Hkv, D, lens, dt, seed, head_major=False):
    c = Cache(B, cap, Hkv, D, head_major)
    k, v = rows(B, cap, Hkv, D, dt, seed, "k"), rows(B, cap, Hkv, D, dt, seed, "v")
    for b, n in enumerate(lens):
        if n:
            one = Cache.__new__(Cache)
            one.B, one.cap, one.Hkv, one.D, one.t, one.strides = 1, cap, Hkv, D, c.t[b:b + 1], c.strides
            one.append(k[b:b + 1, :n].contiguous(), v[b:b + 1, :n].contiguous(), [0], n, dt=dt)
    return c, held(k), held(v)


# (B, Hq, Hkv, D, cap, lens, window, softcap, head_major)
SHAPES = [
    (1, 1, 1, 64, 1, [1], 0, 0.0, False),
    (6, 4, 2, 64, 300, [0, 1, 15, 16, 17, 300], 0, 0.0, False),
    (5, 16, 2, 128, 700, [31, 32, 33, 129, 700], 0, 0.0, True),
    (3, 10, 2, 80, 515, [515, 128, 511], 200, 0.0, False),
    (3, 12, 1, 128, 400, [400, 399, 7], 0, 30.0, False),   # 12 heads: two blocks of a unit
    (2, 24, 2, 256, 333, [333, 100], 65, 50.0, True),
    (2, 16, 2, 512, 260, [260, 63], 0, 0.0, False),
    (2, 3, 1, 512, 129, [129, 65], 1, 0.0, True),          # a window of one key
    (40, 8, 8, 64, 90, [1 + (37 * b) % 90 for b in range(40)], 0, 0.0, False),
    (1, 8, 1, 128, 9000, [8999], 0, 0.0, False),           # one unit over every CTA
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dH%d-%dD%dL%dW%dC%g%s" % (
    s[0], s[1], s[2], s[3], s[4], s[6], s[7], "h" if s[8] else ""))
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_matches_the_oracle(shape, dt):
    B, Hq, Hkv, D, cap, lens, window, softcap, hm = shape
    c, kh, vh = filled(B, cap, Hkv, D, lens, dt, 100 + D, hm)
    full = W.normal((B, Hq * D + 16), dtype=dt, device="cuda", seed=D, role="q")
    q = full[:, :Hq * D]
    out, lse, st = decode(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), dt, Hq, window, softcap,
                          out_pad=16)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(out[:, Hq * D:].float()).all()
    check_decode(out, lse, q, kh, vh, lens, dt, Hq, D, window, softcap, str(shape))


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("G", [1, 5, 8])
def test_every_length_around_a_tile(D, G):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 95, 96, 97, 127, 128, 129, 130, 255, 256, 257]
    B, Hkv, cap = len(lens), 1, 257
    c, kh, vh = filled(B, cap, Hkv, D, lens, "bf16", 7 * D)
    q = W.normal((B, G * D), dtype="bf16", device="cuda", seed=G, role="q")
    out, lse, st = decode(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), "bf16", G)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, kh, vh, lens, "bf16", G, D, 0, 0.0, "D%d G%d" % (D, G))


@pytest.mark.parametrize("window,softcap", [(0, 0.0), (130, 20.0)])
def test_short_sequences_in_long_caches(window, softcap):
    """Caches long enough for the form of head_dim 128 that takes 64 keys a warp at once."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 511, 513, 600]
    B, Hq, Hkv, D, cap, n = len(lens), 40, 8, 128, 10240, 600
    c = Cache(B, cap, Hkv, D)
    k, v = rows(B, n, Hkv, D, "bf16", 3, "k"), rows(B, n, Hkv, D, "bf16", 3, "v")
    c.append(k, v, [0] * B, n)
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=4, role="q")
    for b, x in enumerate(lens):
        c.t[b, x:n] = 255
    out, lse, st = decode(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), "bf16", Hq, window, softcap)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, held(k), held(v), lens, "bf16", Hq, D, window, softcap, "long caches")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_sequences_most_of_them_empty(dt):
    """More sequences than a CTA has threads, zero to 70 keys each, over a capacity above
    max_kv_len: the shares cross many short units."""
    B, Hq, Hkv, D, cap = 700, 4, 2, 64, 96
    g = torch.Generator().manual_seed(11)
    lens = (torch.randint(0, 71, (B,), generator=g) * (torch.rand(B, generator=g) < 0.4)).tolist()
    c = Cache(B, cap, Hkv, D)
    k, v = rows(B, cap, Hkv, D, dt, 1, "k"), rows(B, cap, Hkv, D, dt, 1, "v")
    c.append(k, v, [0] * B, cap, dt=dt)
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q")
    out, lse, st = decode(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), dt, Hq, max_len=71)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, held(k), held(v), lens, dt, Hq, D, 0, 0.0, "many")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("q_mul,k_mul,scale", [(1.0, 1.0, 0.0), (1.0, 1.0, -0.1), (2.0 ** 118, 2.0 ** -118, 0.1),
                                               (2.0 ** -120, 2.0 ** 118, 0.4), (2.0 ** -9, 1.0, 50.0)])
def test_scales_at_the_edges_of_the_numbers(dt, q_mul, k_mul, scale):
    """Scale zero and below; queries and keys far from 1 whose products are not."""
    B, Hq, Hkv, D, cap = 2, 4, 1, 128, 200
    k, v = rows(B, cap, Hkv, D, "f32", 1, "k") * k_mul, rows(B, cap, Hkv, D, "f32", 1, "v")
    q = W.normal((B, Hq * D), dtype="f32", device="cuda", seed=2, role="q") * q_mul
    k, v, q = (x.to(W.torch_dtype(dt)) for x in (k, v, q))
    c = Cache(B, cap, Hkv, D)
    c.append(k, v, [0] * B, cap, dt=dt)
    lens = [200, 3]
    out, lse, st = decode(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), dt, Hq, scale=scale)
    torch.cuda.synchronize()
    kh, vh = held(k), held(v)
    ref, ref_lse = oracle.decode(q.view(B, Hq, D), kh, vh, lens, window=0, scale=scale)
    got = out.double().cpu().numpy().reshape(B, Hq, D)
    assert np.isfinite(got).all()
    # (a larger scale magnifies the scores' error: their magnitude stays below 2^7 here)
    assert np.abs(got - ref).max() <= 2 * REL[dt] * np.abs(vh).max()
    assert np.abs(lse.double().cpu().numpy() - ref_lse).max() <= 2e-4


def test_nan_in_a_visible_row_and_in_the_query():
    """A NaN value makes its group's 32 channels NaN and no others; a NaN key or query, the head."""
    B, Hq, Hkv, D, cap = 3, 2, 1, 128, 64
    k, v = rows(B, cap, Hkv, D, "bf16", 1, "k"), rows(B, cap, Hkv, D, "bf16", 1, "v")
    v[0, 5, 0, 40] = float("nan")
    k[1, 7, 0, 3] = float("inf")
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=2, role="q")
    q[2, 3] = float("nan")  # head 0
    c = Cache(B, cap, Hkv, D)
    c.append(k, v, [0] * B, cap)
    out, lse, st = decode(c, q, torch.full((B,), cap, dtype=torch.int32, device="cuda"), "bf16", Hq)
    bad = torch.isnan(out.view(B, Hq, D))
    assert bad[0, :, 32:64].all() and int(bad[0].sum()) == Hq * 32
    assert bad[1].all() and bad[2, 0].all() and not bad[2, 1].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [300, 9000])
def test_scores_below_the_least_float_weigh_nothing(dt, cap):
    """Whole pieces of a sequence whose scores leave fp32's range on the low side."""
    B, Hq, Hkv, D = 3, 4, 1, 128
    k, v = rows(B, cap, Hkv, D, dt, 1, "k"), rows(B, cap, Hkv, D, dt, 1, "v")
    k[0, :cap - 40] = -3e38
    k[1, 40:] = -3e38
    k[2, 100:cap - 100] = -3e38
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q").abs()  # sums of 128 terms near -3e38
    c = Cache(B, cap, Hkv, D)
    c.append(k, v, [0] * B, cap, dt=dt)
    lens = [cap] * B
    out, lse, st = decode(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), dt, Hq)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, held(k), held(v), lens, dt, Hq, D, 0, 0.0, "low scores")


def test_lengths_out_of_range_leave_their_rows_alone():
    B, Hq, Hkv, D, cap = 4, 4, 2, 128, 64
    lens = [64, 65, -1, 10]
    c, kh, vh = filled(B, cap, Hkv, D, [64, 64, 64, 10], "bf16", 3)
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=9, role="q")
    out, lse, st = decode(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), "bf16", Hq)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert torch.isnan(out[1:3].float()).all() and torch.isnan(lse[1:3]).all()
    keep = [0, 3]
    check_decode(out[keep], lse[keep], q[keep], kh[keep], vh[keep], [64, 10], "bf16", Hq, D, 0, 0.0, "kept")


def test_a_long_cache_past_32_bit_offsets():
    """Two sequences of 2.2e9 bytes, written and read at their far ends."""
    B, Hq, Hkv, D, cap = 2, 8, 1, 512, 3_500_000  # 640 bytes a row: 2.2e9 bytes a sequence
    c = Cache(B, cap, Hkv, D)
    n, at = 300, cap - 300
    k, v = rows(B, n, Hkv, D, "bf16", 1, "k"), rows(B, n, Hkv, D, "bf16", 1, "v")
    st = c.append(k, v, [at, at], n)
    gk, gv = c.expand([at, at], n, "f32", st)
    assert_held(gk, k, "K")
    assert_held(gv, v, "V")
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=9, role="q")
    lens = torch.tensor([cap, cap], dtype=torch.int32, device="cuda")
    out, lse, st = decode(c, q, lens, "bf16", Hq, window=n, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, held(k), held(v), [n, n], "bf16", Hq, D, 0, 0.0, "far end")


def test_chunks_prefill_and_steps_together():
    """As a server uses it: two chunks of a prompt (append, read back, prefill), then steps
    (append one token, decode), on a stream of its own, the decode captured and replayed."""
    B, Hq, Hkv, D, cap, chunk, steps = 2, 8, 2, 128, 256, 96, 4
    total = 2 * chunk + steps
    k, v = rows(B, total, Hkv, D, "bf16", 21, "k"), rows(B, total, Hkv, D, "bf16", 21, "v")
    q = W.normal((B, total, Hq * D), dtype="bf16", device="cuda", seed=21, role="q")
    kh, vh = held(k), held(v)
    vmax = np.abs(vh).max()
    c = Cache(B, cap, Hkv, D)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st = status_tensor()
        for p0 in (0, chunk):
            kn, vn = (x[:, p0:p0 + chunk].contiguous() for x in (k, v))
            c.append(kn, vn, [p0] * B, chunk, st)
            n = p0 + chunk
            gk, gv = c.expand([0] * B, n, "bf16", st)
            gk, gv = gk.reshape(B * n, Hkv * D), gv.reshape(B * n, Hkv * D)
            qc = q[:, p0:n].reshape(B * chunk, Hq * D)
            out = torch.empty_like(qc)
            binding.lat_attn_prefill(binding.LAT_BF16, qc, Hq * D, gk, Hkv * D, gv, Hkv * D, out, Hq * D, None, B,
                                     chunk, n, Hq, Hkv, D, 1, 0, D ** -0.5, st)
            s.synchronize()
            ref, _ = oracle.prefill(qc.view(B, chunk, Hq, D), gk.view(B, n, Hkv, D), gv.view(B, n, Hkv, D),
                                    causal=True, window=0, scale=D ** -0.5)
            assert np.abs(out.float().cpu().numpy().reshape(ref.shape) - ref).max() <= 2.0 ** -7 * vmax
        qs, lens = torch.empty(B, Hq * D, dtype=q.dtype, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        nb = binding.lat_attn_decode_q4_workspace_size(binding.LAT_BF16, B, Hq, Hkv, D, cap)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        out = torch.empty(B, Hq * D, dtype=q.dtype, device="cuda")
        lse = torch.empty(B, Hq, device="cuda")
        pos = torch.zeros(B, dtype=torch.int32, device="cuda")
        kn, vn = (torch.empty(B, Hkv * D, dtype=q.dtype, device="cuda") for _ in range(2))

        def step():
            binding.lat_kv_append_q4(binding.LAT_BF16, c.t, *c.strides, cap, kn, vn, Hkv * D, pos, 1, B, Hkv, D, st)
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
            graph.replay()
            s.synchronize()
            check_decode(out, lse, qs, kh, vh, [t + 1] * B, "bf16", Hq, D, 0, 0.0, "step %d" % t)
        assert int(st.item()) == 0


def test_two_streams_with_a_workspace_each():
    B, Hq, Hkv, D, cap = 3, 16, 4, 128, 5000
    lens = [5000, 1, 2777]
    c, kh, vh = filled(B, cap, Hkv, D, lens, "bf16", 33)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
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


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nothing_cached_anywhere(dt):
    """max_kv_len 0, and caches of every length 0: zeros and -inf, no read of the cache."""
    B, Hq, Hkv, D, cap = 3, 4, 2, 64, 16
    c = Cache(B, cap, Hkv, D)
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=1, role="q")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for mk in (0, cap):
        out, lse, st = decode(c, q, lens, dt, Hq, max_len=mk)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and (out == 0).all() and torch.isneginf(lse).all()
