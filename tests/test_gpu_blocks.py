"""Decode over chosen blocks: lat_kv_block_bounds, lat_attn_select_blocks and
lat_attn_decode_blocks.

Bounds and choices are exact.  Decodes are compared with the fp64 attention oracle over the
listed keys; every other cache row holds NaN.  Tolerances: a bf16 output is a mean of |v| <= vmax
under weights rounded once to bf16 (2^-9 relative each), rounded once more itself, 2^-8 vmax, and
the scores' fp32 sums add at most 2^-11 vmax; in fp32 the sums alone remain, 2e-5 vmax at these
sizes (products of magnitude below 2^6).  lse 1e-4.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import DT, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding
from oracle import blocks as ob

pytestmark = pytest.mark.gpu

HEAD_DIMS = (64, 80, 128, 256, 512)
REL = {"bf16": 2.0 ** -8 + 2.0 ** -11, "f32": 2e-5}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def room(B, n, H, D, dt, head_major=False, pad=0):
    """[B, n, H, D + pad] of NaN, token- or head-major."""
    shape = (B, H, n, D + pad) if head_major else (B, n, H, D + pad)
    t = torch.full(shape, float("nan"), dtype=W.torch_dtype(dt), device="cuda")
    return t.transpose(1, 2) if head_major else t


def strides(t):
    return t.stride(1), t.stride(2), t.stride(0)


def make_bounds(k, bounds, block, pos, n, D, dt, status=None):
    B, cap, H = k.shape[:3]
    st = status if status is not None else status_tensor()
    binding.lat_kv_block_bounds(DT[dt], k, *strides(k), cap, bounds, *strides(bounds), block, i32(pos), n, B, H, D, st)
    return st


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------------- bounds
@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("block,hm", [(16, False), (48, True), (64, False)])
def test_bounds_are_the_blocks_extremes(D, dt, block, hm):
    B, H, cap = 2, 3, 5 * block + 7
    k = room(B, cap, H, D, dt, hm, pad=16)
    k[..., :D] = W.normal((B, cap, H, D), dtype=dt, device="cuda", seed=D, role="k")
    nb = -(-cap // block)
    bd = room(B, nb, H, 2 * D, dt, hm, pad=16)
    st = make_bounds(k, bd, block, [0, 0], cap, D, dt)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(B):
        for h in range(H):
            hi, lo = ob.bounds(f64(k[b, :, h, :D]), block)
            assert np.array_equal(f64(bd[b, :, h, :D]), hi) and np.array_equal(f64(bd[b, :, h, D:2 * D]), lo)
    assert torch.isnan(bd[..., 2 * D:]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bounds_grow_with_the_cache(dt):
    """Pieces of 1, 5, 16, 37, ... rows, each sequence at its own place: after every piece the
    bounds are those of all rows so far, and no other row of them is touched."""
    B, H, D, block, cap = 3, 2, 128, 32, 300
    start = [0, 32, 64]  # whole blocks in
    k = room(B, cap, H, D, dt)
    bd = room(B, -(-cap // block), H, 2 * D, dt)
    new = W.normal((B, cap, H, D), dtype=dt, device="cuda", seed=4, role="new")
    at = list(start)
    for n in (1, 1, 5, 16, 37, 2, 64, 3):
        for b in range(B):
            k[b, at[b]:at[b] + n] = new[b, at[b]:at[b] + n]
        st = make_bounds(k, bd, block, at, n, D, dt)
        at = [x + n for x in at]
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        for b in range(B):
            n0, n1 = start[b] // block, -(-at[b] // block)
            assert torch.isnan(bd[b, :n0]).all() and torch.isnan(bd[b, n1:]).all()
            for h in range(H):
                hi, lo = ob.bounds(f64(k[b, start[b]:at[b], h]), block)
                assert np.array_equal(f64(bd[b, n0:n1, h, :D]), hi)
                assert np.array_equal(f64(bd[b, n0:n1, h, D:]), lo)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bounds_keep_nan_and_infinities(dt):
    D, block = 64, 16
    k = W.normal((1, 48, 1, D), dtype=dt, device="cuda", seed=1, role="k")
    k[0, 3, 0, 5], k[0, 20, 0, 6], k[0, 21, 0, 7] = float("nan"), float("inf"), float("-inf")
    bd = room(1, 3, 1, 2 * D, dt)
    make_bounds(k, bd, block, [0], 48, D, dt)
    got = f64(bd[0, :, 0])
    assert np.isnan(got[0, 5]) and np.isnan(got[0, D + 5]) and np.isnan(got).sum() == 2
    assert got[1, 6] == np.inf and got[1, D + 7] == -np.inf
    # a later row of the same block keeps it
    make_bounds(k, bd, block, [4], 12, D, dt)
    assert np.isnan(f64(bd[0, 0, 0])).sum() == 2


def test_bounds_out_of_range_skip_the_sequence():
    k = W.normal((3, 40, 1, 64), dtype="bf16", device="cuda", seed=1, role="k")
    bd = room(3, 3, 1, 128, "bf16")
    st = make_bounds(k, bd, 16, [31, 35, -1], 9, 64, "bf16")
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert torch.isnan(bd[1:]).all() and torch.isnan(bd[0, 0]).all() and not torch.isnan(bd[0, 2]).any()


# ---------------------------------------------------------------------------------- select
def select(q, bd, lens, block, Hq, H, D, dt, n_sel, n_first, n_last, max_len=None, out=None, ws=None, st=None):
    B = q.shape[0]
    mk = max(max(lens), 1) if max_len is None else max_len
    nb = binding.lat_attn_select_blocks_workspace_size(B, H, block, mk)
    if ws is None:  # needs no clearing
        ws = torch.full((max(nb, 256),), 255, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((B, H, n_sel), -7, dtype=torch.int32, device="cuda")
    st = st if st is not None else status_tensor()
    binding.lat_attn_select_blocks(DT[dt], q, q.stride(0), bd, *strides(bd), block, i32(lens), mk, out, n_sel,
                                   n_first, n_last, B, Hq, H, D, ws, nb, st)
    return out, st


def check_select(got, q, bd, lens, block, Hq, H, D, n_sel, n_first, n_last):
    G = Hq // H
    for b, n in enumerate(lens):
        nb = -(-n // block)
        for h in range(H):
            r = f64(bd[b, :nb, h])
            s = ob.scores(f64(q[b, h * G * D:(h + 1) * G * D]).reshape(G, D), r[:, :D], r[:, D:2 * D])
            want = ob.choose(s, n_sel, n_first, n_last)
            assert np.array_equal(got[b, h].cpu().numpy(), want), (b, h, n)


# (Hq, H, D, block, lens, n_sel, n_first, n_last, head_major)
SELECT = [
    (4, 2, 64, 16, [1, 16, 17, 500, 3000, 0], 8, 1, 2, False),
    (8, 1, 128, 64, [9000, 4096, 70], 20, 0, 0, True),
    (24, 2, 80, 32, [2000, 1999], 7, 2, 3, False),      # 12 heads a group
    (3, 3, 256, 48, [3000, 48 * 40], 40, 0, 1, True),   # exactly as many as are kept
    (10, 1, 512, 128, [6000], 5, 5, 0, False),          # nothing left to choose
    (2, 2, 64, 1024, [50000, 1024], 3, 0, 1, False),
    (16, 2, 128, 16, [2500], 1, 0, 0, False),
]


@pytest.mark.parametrize("case", SELECT, ids=lambda c: "H%d-%dD%db%dn%d" % (c[0], c[1], c[2], c[3], c[5]))
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_select_is_the_oracles_choice(case, dt):
    Hq, H, D, block, lens, n_sel, n_first, n_last, hm = case
    B, nb = len(lens), -(-max(lens) // block)
    bd = room(B, nb, H, 2 * D, dt, hm)
    mid = W.normal((B, nb, H, D), dtype="f32", device="cuda", seed=D, role="k")
    half = W.normal((B, nb, H, D), dtype="f32", device="cuda", seed=D, role="v").abs()
    bd[..., :D], bd[..., D:] = mid + half, mid - half
    for b, n in enumerate(lens):  # blocks past the length hold anything
        bd[b, -(-n // block):] = float("nan")
    q = W.normal((B, Hq * D + 16), dtype=dt, device="cuda", seed=D, role="q")[:, :Hq * D]
    got, st = select(q, bd, lens, block, Hq, H, D, dt, n_sel, n_first, n_last)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_select(got, q, bd, lens, block, Hq, H, D, n_sel, n_first, n_last)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_select_between_equal_and_nearly_equal_scores(dt):
    """Blocks with the same products in another order (their fp32 sums differ, their exact scores
    do not) and blocks ahead of them by a part in 2^30: ties go to the lowest, the least bit more
    decides."""
    D, nb, n_sel, block = 128, 300, 40, 16
    g = torch.Generator().manual_seed(5)
    x = torch.randn(D, generator=g).bfloat16().float()
    x[-1] = 0.0
    r = torch.empty(1, nb, 1, 2 * D)
    for n in range(nb):
        y = x[torch.cat([torch.randperm(D - 1, generator=g), torch.tensor([D - 1])])]
        r[0, n, 0, :D], r[0, n, 0, D:] = y, y
    for n in (299, 150, 31):  # the last channel's product adds 2^-30
        r[0, n, 0, D - 1] = r[0, n, 0, 2 * D - 1] = 2.0 ** -30
    r[0, 7, 0, D - 1] = r[0, 7, 0, 2 * D - 1] = -2.0 ** -30  # and takes it away: not among the lowest
    q = torch.ones(1, D, dtype=W.torch_dtype(dt), device="cuda")
    got, st = select(q, r.to(W.torch_dtype(dt)).cuda(), [nb * block], block, 1, 1, D, dt, n_sel, 0, 0)
    want = sorted([31, 150, 299] + [n for n in range(nb) if n not in (7, 31, 150, 299)][:n_sel - 3])
    assert got[0, 0].tolist() == want and int(st.item()) == 0
    zero = torch.zeros_like(q)  # every score 0
    got, _ = select(zero, r.to(W.torch_dtype(dt)).cuda(), [nb * block], block, 1, 1, D, dt, n_sel, 2, 3)
    assert got[0, 0].tolist() == list(range(n_sel - 3)) + [nb - 3, nb - 2, nb - 1]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nb", [300, 2000])
@pytest.mark.parametrize("q_mul,k_mul", [(2.0 ** 60, 2.0 ** 50), (2.0 ** -40, 2.0 ** -30)])
def test_select_between_near_scores_far_from_one(dt, nb, q_mul, k_mul):
    """The same at the ends of the range, where a pair of floats cannot hold the sums: every sum
    of these products is exact in fp64 (terms of 8 bits from 2^-30 to 2^3 of the scale)."""
    D, n_sel, block = 128, 40, 16
    g = torch.Generator().manual_seed(6)
    x = torch.randn(D, generator=g).bfloat16().float()
    x[-1] = 0.0
    r = torch.empty(1, nb, 1, 2 * D)
    for n in range(nb):
        y = x[torch.cat([torch.randperm(D - 1, generator=g), torch.tensor([D - 1])])]
        r[0, n, 0, :D], r[0, n, 0, D:] = y, y
    for n in (nb - 1, 150, 31):
        r[0, n, 0, D - 1] = r[0, n, 0, 2 * D - 1] = 2.0 ** -30
    r[0, 7, 0, D - 1] = r[0, 7, 0, 2 * D - 1] = -2.0 ** -30
    q = torch.full((2, D), q_mul, dtype=W.torch_dtype(dt), device="cuda")
    q[1] = 1.0  # and a sequence whose scores lie elsewhere
    rr = (r * k_mul).to(W.torch_dtype(dt)).cuda().expand(2, -1, -1, -1).contiguous()
    got, st = select(q, rr, [nb * block] * 2, block, 1, 1, D, dt, n_sel, 0, 0)
    want = sorted([31, 150, nb - 1] + [n for n in range(nb) if n not in (7, 31, 150, nb - 1)][:n_sel - 3])
    assert got[0, 0].tolist() == want and got[1, 0].tolist() == want and int(st.item()) == 0


@pytest.mark.parametrize("dt,nb,n_sel", [("bf16", 2000, 700), ("f32", 2000, 1), ("bf16", 9000, 4000)])
def test_select_among_many_equal_scores(dt, nb, n_sel):
    """Thousands of exact ties: the lowest, beside one block ahead and one behind."""
    D, block = 64, 16
    bd = torch.ones(1, nb, 1, 2 * D, dtype=W.torch_dtype(dt), device="cuda")
    bd[0, nb - 7, 0, 3] = 1.5
    bd[0, 5, 0, 9] = 0.5
    q = torch.ones(1, D, dtype=W.torch_dtype(dt), device="cuda")
    got, st = select(q, bd, [nb * block], block, 1, 1, D, dt, n_sel, 0, 0)
    assert int(st.item()) == 0
    want = sorted([nb - 7] + [n for n in range(nb) if n not in (5, nb - 7)][:n_sel - 1])
    assert got[0, 0].tolist() == want


@pytest.mark.parametrize("nb,n_sel", [(6200, 100), (65536, 2000)])
def test_select_among_many_blocks(nb, n_sel):
    """More than the keys that shared memory holds, up to the most blocks a sequence may have."""
    D, block, H = 64, 16, 2
    bd = W.normal((1, nb, H, 2 * D), dtype="bf16", device="cuda", seed=nb, role="k")
    q = W.normal((1, 4 * D), dtype="bf16", device="cuda", seed=nb, role="q")
    got, st = select(q, bd, [nb * block], block, 4, H, D, "bf16", n_sel, 3, 5)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    qd = q.double().view(H, 2, D)
    r = bd[0].double()
    s = (torch.einsum("hgd,nhd->hgn", qd.clamp(min=0), r[..., :D]) +
         torch.einsum("hgd,nhd->hgn", qd.clamp(max=0), r[..., D:])).amax(1).cpu().numpy()
    for h in range(H):
        assert np.array_equal(got[0, h].cpu().numpy(), ob.choose(s[h], n_sel, 3, 5))


def test_select_puts_nan_first_and_takes_infinities():
    D, nb, block = 64, 50, 16
    bd = W.normal((1, nb, 1, 2 * D), dtype="bf16", device="cuda", seed=2, role="k").abs()
    q = W.normal((1, D), dtype="bf16", device="cuda", seed=2, role="q").abs() + 0.5
    bd[0, 40, 0, 3] = float("nan")
    bd[0, 30, 0, 4] = float("inf")
    bd[0, 20, 0, 5] = float("-inf")
    got, _ = select(q, bd, [nb * block], block, 1, 1, D, "bf16", 2, 0, 0)
    assert got[0, 0].tolist() == [30, 40]
    got, _ = select(q, bd, [nb * block], block, 1, 1, D, "bf16", 1, 0, 0)
    assert got[0, 0].tolist() == [40]
    got, _ = select(q, bd, [nb * block], block, 1, 1, D, "bf16", nb - 1, 0, 0)
    assert got[0, 0].tolist() == [n for n in range(nb) if n != 20]


def test_select_out_of_range_leaves_the_lists():
    D = 64
    bd = W.normal((3, 10, 1, 2 * D), dtype="f32", device="cuda", seed=2, role="k")
    q = W.normal((3, D), dtype="f32", device="cuda", seed=2, role="q")
    got, st = select(q, bd, [100, -1, 161], 16, 1, 1, D, "f32", 3, 0, 0, max_len=160)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert (got[1:] == -7).all() and (got[0] >= 0).all()


# ---------------------------------------------------------------------------------- decode
def decode(q, k, v, lens, block, lists, Hq, D, dt, softcap=0.0, max_len=None, out_pad=0, ws=None, st=None, out=None,
           lse=None, stream=None):
    B, cap, H = k.shape[:3]
    n_sel = lists.shape[2]
    nb = binding.lat_attn_decode_blocks_workspace_size(DT[dt], B, Hq, H, D, block, n_sel)
    assert nb > 0
    if ws is None:
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        if dt == "f32":
            ws.fill_(255)  # needs no clearing
    if out is None:
        out = torch.full((B, Hq * D + out_pad), float("nan"), dtype=q.dtype, device="cuda")
    if lse is None:
        lse = torch.full((B, Hq), float("nan"), device="cuda")
    st = st if st is not None else status_tensor()
    lens_t = lens if torch.is_tensor(lens) else i32(lens)
    binding.lat_attn_decode_blocks(DT[dt], q, q.stride(0), k, v, *strides(k), lens_t, cap if max_len is None else max_len,
                                   block, lists, n_sel, out, out.stride(0), lse, B, Hq, H, D, D ** -0.5, softcap, ws,
                                   nb, st, stream=stream)
    return out, lse, st


def check_decode(out, lse, q, k, v, lens, block, lists, Hq, D, dt, softcap=0.0):
    B, _, H = k.shape[:3]
    G = Hq // H
    got, gl = f64(out[:, :Hq * D]).reshape(B, Hq, D), f64(lse)
    for b in range(B):
        for h in range(H):
            at = ob.rows_of(lists[b, h].tolist(), block, lens[b])
            hs = slice(h * G, (h + 1) * G)
            if not at:
                assert (got[b, hs] == 0).all() and np.isneginf(gl[b, hs]).all()
                continue
            kk, vv = f64(k[b, at, h, :D])[None, :, None], f64(v[b, at, h, :D])[None, :, None]
            qq = f64(q[b, h * G * D:(h + 1) * G * D]).reshape(1, G, D)
            ref, rl = oracle.decode(qq, kk, vv, [len(at)], window=0, scale=D ** -0.5, softcap=softcap)
            assert np.isfinite(got[b, hs]).all()
            err = np.abs(got[b, hs] - ref[0]).max()
            assert err <= REL[dt] * np.abs(vv).max(), (b, h, err)
            assert np.abs(gl[b, hs] - rl[0]).max() <= 1e-4, (b, h)


def lists_for(lens, H, block, n_sel, seed, pad=True):
    """Random ascending lists, the last block among some; shorter ones padded."""
    r = np.random.default_rng(seed)
    out = np.full((len(lens), H, n_sel), -1, dtype=np.int64)
    for b, n in enumerate(lens):
        nb = -(-n // block)
        for h in range(H):
            m = int(r.integers(0, min(nb, n_sel) + 1)) if pad else min(nb, n_sel)
            pick = sorted(r.permutation(nb)[:m].tolist())
            if m and r.random() < 0.7 and pick[-1] != nb - 1:
                pick[-1] = nb - 1
            out[b, h, :m] = pick
    return out


def cache_for(lists, lens, cap, block, D, dt, hm, seed):
    B, H = lists.shape[:2]
    k, v = room(B, cap, H, D, dt, hm), room(B, cap, H, D, dt, hm)
    for b in range(B):
        for h in range(H):
            at = ob.rows_of(lists[b, h].tolist(), block, lens[b])
            if at:
                k[b, at, h] = W.normal((len(at), D), dtype=dt, device="cuda", seed=seed + 7 * b + h, role="k")
                v[b, at, h] = W.normal((len(at), D), dtype=dt, device="cuda", seed=seed + 7 * b + h, role="v")
    return k, v


# (Hq, H, D, block, lens, n_sel, softcap, head_major)
DECODE = [
    (2, 1, 64, 16, [1, 15, 16, 17, 200, 0], 6, 0.0, False),
    (8, 2, 128, 64, [4000, 64, 65, 3999], 20, 0.0, True),
    (10, 2, 80, 32, [1000, 333], 9, 30.0, False),
    (24, 2, 128, 48, [700, 1500], 11, 0.0, False),   # 12 heads a group; a tile spans blocks
    (16, 2, 256, 16, [900, 64], 30, 50.0, True),
    (16, 2, 512, 128, [2000, 1], 6, 0.0, False),
    (4, 4, 64, 1024, [5000, 1024], 2, 0.0, False),
    (8, 8, 128, 16, [300 + 11 * b for b in range(24)], 10, 0.0, False),
    (16, 1, 128, 64, [30000], 200, 0.0, False),      # one unit over every CTA
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "H%d-%dD%db%dn%d" % (c[0], c[1], c[2], c[3], c[5]))
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [False, True])
def test_decode_over_listed_blocks(case, dt, pad):
    Hq, H, D, block, lens, n_sel, softcap, hm = case
    cap = max(lens) + 5
    lists = lists_for(lens, H, block, n_sel, D + block, pad)
    k, v = cache_for(lists, lens, cap, block, D, dt, hm, D)
    q = W.normal((len(lens), Hq * D + 16), dtype=dt, device="cuda", seed=D, role="q")[:, :Hq * D]
    out, lse, st = decode(q, k, v, lens, block, i32(lists), Hq, D, dt, softcap, out_pad=16)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(out[:, Hq * D:].float()).all()
    check_decode(out, lse, q, k, v, lens, block, lists, Hq, D, dt, softcap)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_all_blocks_is_the_whole_cache(dt):
    """A list of every block gives lat_attn_decode's answer."""
    B, Hq, H, D, block = 3, 8, 2, 128, 32
    lens = [500, 77, 1]
    di = W.decode_inputs(B, Hq, H, D, 512, kv_lens=lens, dtype=dt, device="cuda")
    lists = np.full((B, H, 16), -1)
    for b, n in enumerate(lens):
        lists[b, :, :-(-n // block)] = np.arange(-(-n // block))
    k, v = di.k_cache.view(B, 512, H, D), di.v_cache.view(B, 512, H, D)
    out, lse, st = decode(di.q, k, v, lens, block, i32(lists), Hq, D, dt)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, di.q, k, v, lens, block, lists, Hq, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [[3, 3, 5], [5, 3, -1], [-1, 2, -1], [0, 1, 10], [-2, 1, 2]])
def test_a_list_out_of_order_or_range_is_reported(dt, bad):
    """The same block twice, descending, an entry behind padding, past the blocks there are,
    below -1: the status says so; the other sequence's answer stands."""
    Hq, H, D, block, lens = 4, 1, 64, 16, [160, 160]
    lists = np.array([[bad], [[0, 4, 9]]])
    k = W.normal((2, 160, H, D), dtype=dt, device="cuda", seed=1, role="k")
    v = W.normal((2, 160, H, D), dtype=dt, device="cuda", seed=1, role="v")
    q = W.normal((2, Hq * D), dtype=dt, device="cuda", seed=1, role="q")
    out, lse, st = decode(q, k, v, lens, block, i32(lists), Hq, D, dt)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    check_decode(out[1:], lse[1:], q[1:], k[1:], v[1:], lens[1:], block, lists[1:], Hq, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_lengths_out_of_range_leave_their_rows_alone(dt):
    Hq, H, D, block = 4, 2, 128, 16
    lens = [64, 65, -1, 10]
    lists = np.tile(np.array([0, -1, -1, -1]), (4, H, 1))
    k = W.normal((4, 64, H, D), dtype=dt, device="cuda", seed=1, role="k")
    v = W.normal((4, 64, H, D), dtype=dt, device="cuda", seed=1, role="v")
    q = W.normal((4, Hq * D), dtype=dt, device="cuda", seed=1, role="q")
    out, lse, st = decode(q, k, v, lens, block, i32(lists), Hq, D, dt)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert torch.isnan(out[1:3].float()).all() and torch.isnan(lse[1:3]).all()
    keep = [0, 3]
    check_decode(out[keep], lse[keep], q[keep], k[keep], v[keep], [64, 10], block, lists[keep], Hq, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_steps_together(dt):
    """As a server uses it: a prompt's keys appended and bounded, then steps, each an append, its
    block's bounds, the choice and the attention, captured once and replayed on a stream of its
    own.  Every step is checked against the oracle's bounds, choice and attention."""
    B, Hq, H, D, block, cap, prompt, n_sel = 2, 8, 2, 128, 16, 256, 150, 5
    k = room(B, cap, H, D, dt)
    v = room(B, cap, H, D, dt)
    bd = room(B, cap // block, H, 2 * D, dt)
    steps = 4
    kn = W.normal((B, prompt + steps, H, D), dtype=dt, device="cuda", seed=3, role="k")
    vn = W.normal((B, prompt + steps, H, D), dtype=dt, device="cuda", seed=3, role="v")
    q = W.normal((B, prompt + steps, Hq * D), dtype=dt, device="cuda", seed=3, role="q")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st = status_tensor()
        qs = torch.empty(B, Hq * D, dtype=q.dtype, device="cuda")
        k1, v1 = (torch.empty(B, H * D, dtype=q.dtype, device="cuda") for _ in range(2))
        pos, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        lists = torch.empty(B, H, n_sel, dtype=torch.int32, device="cuda")
        out, lse = torch.empty_like(qs), torch.empty(B, Hq, device="cuda")
        nb1 = binding.lat_attn_select_blocks_workspace_size(B, H, block, cap)
        ws1 = torch.empty(nb1, dtype=torch.uint8, device="cuda")
        nb2 = binding.lat_attn_decode_blocks_workspace_size(DT[dt], B, Hq, H, D, block, n_sel)
        ws2 = torch.zeros(nb2, dtype=torch.uint8, device="cuda")

        def put(kx, vx, n):
            binding.lat_kv_append(DT[dt], k, v, *strides(k), cap, kx, vx, H * D, pos, n, B, H, D, st)
            binding.lat_kv_block_bounds(DT[dt], k, *strides(k), cap, bd, *strides(bd), block, pos, n, B, H, D, st)

        def step():
            put(k1, v1, 1)
            binding.lat_attn_select_blocks(DT[dt], qs, Hq * D, bd, *strides(bd), block, lens, cap, lists, n_sel, 1, 2,
                                           B, Hq, H, D, ws1, nb1, st)
            decode(qs, k, v, lens, block, lists, Hq, D, dt, ws=ws2, st=st, out=out, lse=lse)

        put(kn[:, :prompt].contiguous(), vn[:, :prompt].contiguous(), prompt)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for t in range(prompt, prompt + steps):
            k1.copy_(kn[:, t].reshape(B, -1))
            v1.copy_(vn[:, t].reshape(B, -1))
            qs.copy_(q[:, t])
            pos.fill_(t)
            lens.fill_(t + 1)
            graph.replay()
            s.synchronize()
            assert int(st.item()) == 0
            n = t + 1
            for b in range(B):
                for h in range(H):
                    hi, lo = ob.bounds(f64(k[b, :n, h]), block)
                    r = f64(bd[b, :len(hi), h])
                    assert np.array_equal(r[:, :D], hi) and np.array_equal(r[:, D:], lo)
            check_select(lists, qs, bd, [n] * B, block, Hq, H, D, n_sel, 1, 2)
            check_decode(out, lse, qs, k, v, [n] * B, block, lists.cpu().numpy(), Hq, D, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nothing_cached_anywhere(dt):
    """max_kv_len 0, and caches of every length 0: empty lists, zeros and -inf."""
    B, Hq, H, D, cap, block, n_sel = 3, 4, 2, 64, 32, 16, 2
    k = W.normal((B, cap, H, D), dtype=dt, device="cuda", seed=1, role="k")
    bd = W.normal((B, cap // block, H, 2 * D), dtype=dt, device="cuda", seed=1, role="v")
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=1, role="q")
    for mk in (0, cap):
        got, st = select(q, bd, [0] * B, block, Hq, H, D, dt, n_sel, 1, 1, max_len=mk)
        out, lse, st2 = decode(q, k, k, [0] * B, block, got, Hq, D, dt, max_len=mk)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(st2.item()) == 0 and (got == -1).all()
        assert (out == 0).all() and torch.isneginf(lse).all()
