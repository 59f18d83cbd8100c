"""How near a bf16 decode over the 8-bit cache comes: to the rounding of its output.

Tolerance.  y = sum_j w_j v_j, the w_j positive and of sum 1, |v| <= vmax; the kernel returns
bf16(y + e), so with |e| <= E it lies between bf16(y - E) and bf16(y + E).  E, in parts of vmax:
  * Scores.  Only the query's channels that are not zero add any error, three here; a product of a
    bf16 channel and a code is exact, and with M the largest scale * log2(e) * sum |q k| a score's
    three sums are cut off by 2^-22 M each at most, its three factors and its distance from the
    reference round by 2^-24 M each: 4 * 2^-22 M.  M <= 12 here: 1.15e-5 in the exponent of 2, 8e-6
    of a weight, and a mean of weights moves by twice that: 1.6e-5.
  * The exponential, twice (2^-22 each); the two fp16 terms of a weight, 2^-22.
  * Sums of positive weights: a lane adds 2^-24 a weight to its own, at most 5 (of 300 keys, 64 a tile of
    four warps), then eight of them and four warps; the values' sums are cut off by 2^-22 an MMA, two
    terms a 16-key tile, 10 in a warp.  5 * 2^-24 + 12 * 2^-24 + 10 * 2^-22 = 3.4e-6.
1.6e-5 + 7.2e-7 + 3.4e-6 < 2.1e-5 <= 2^-15 (3.05e-5), which has room for longer pieces, too: a fp16 term
alone is 2^-12 off (2.4e-4).
"""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import ensure_library
from test_gpu_q8 import HEAD_DIMS, Cache, decode, f64, filled, held, i32, rows

pytestmark = pytest.mark.gpu

SCALE = 0.15


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def queries(B, Hq, D, seed):
    """Three channels of each head of magnitude 0.5 to 1 and either sign, the rest zero."""
    g = np.random.default_rng(seed)
    q = np.zeros((B, Hq, D), np.float32)
    for b in range(B):
        for h in range(Hq):
            for d in g.choice(D, 3, replace=False):
                q[b, h, d] = g.uniform(0.5, 1) * g.choice([-1, 1])
    return torch.from_numpy(q.reshape(B, Hq * D)).to(torch.bfloat16).cuda()


def to_bf16(x):
    return f64(torch.from_numpy(x).to(torch.float32).to(torch.bfloat16))


def check(c, q, lens, Hq, kh, vh, window, what):
    B, D = c.B, c.D
    assert SCALE * math.log2(math.e) * 3 * np.abs(kh).max() <= 12  # the docstring's M
    out, lse, st = decode(c, q, i32(lens), "bf16", Hq, window, scale=SCALE)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, _ = oracle.decode(q.view(B, Hq, D), kh, vh, lens, window=window, scale=SCALE)
    got = out.double().cpu().numpy().reshape(B, Hq, D)
    # (the reference itself is rounded to fp32 on the way to bf16)
    E = 2.0 ** -15 * np.abs(vh).max() + 2.0 ** -24 * np.abs(ref)
    out_of = (got < to_bf16(ref - E)) | (got > to_bf16(ref + E))
    assert not out_of.any(), "%s: %d of %d" % (what, out_of.sum(), out_of.size)


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("G", [1, 4, 8, 12])
def test_weights_add_no_rounding_that_shows(D, G):
    lens = [1, 2, 3, 5, 8, 16, 17, 40, 65, 130, 300]
    B, Hkv, cap = len(lens), 2, 300
    c, kh, vh = filled(B, cap, Hkv, D, lens, "bf16", 5 * D + G, block=32)
    check(c, queries(B, G * Hkv, D, G), lens, G * Hkv, kh, vh, 0, "D%d G%d" % (D, G))


@pytest.mark.parametrize("D", [64, 128, 512])
@pytest.mark.parametrize("v_mul", [2.0 ** -90, 2.0 ** 100])
def test_values_far_from_one(D, v_mul):
    lens = [2, 3, 5, 17, 40, 130, 300]
    B, Hkv, cap, G = len(lens), 2, 300, 4
    c = Cache(B, cap, Hkv, D, 64)
    k, v = rows(B, cap, Hkv, D, "bf16", 8, "k"), rows(B, cap, Hkv, D, "bf16", 8, "v") * v_mul
    c.append(k, v, [0] * B, cap)
    check(c, queries(B, G * Hkv, D, G), lens, G * Hkv, held(k, 64), held(v, 64), 0, "D%d" % D)


@pytest.mark.parametrize("G", [4, 8])
def test_one_unit_over_every_cta(G):
    B, Hkv, D, cap = 1, 1, 128, 9000
    c, kh, vh = filled(B, cap, Hkv, D, [8999], "bf16", 17)
    check(c, queries(B, G, D, 5), [8999], G, kh, vh, 0, "one unit, G%d" % G)
    check(c, queries(B, G, D, 6), [8999], G, kh, vh, 3, "three keys, G%d" % G)


@pytest.mark.parametrize("D", [64, 80, 128])
def test_sums_over_long_shares_lean_to_no_side(D):
    """Outputs around 0 over 32768 keys a CTA, against the exact ones rounded to bf16.

    Scores are small (queries of a tenth), so that a score's D / 16 cuts of 2^-22 of at most 1.6 (the
    exponents of 2) are below 3e-6, 2.1e-6 of a weight; its other roundings, the exponential and the
    weight's two terms 2^-22 each at most, 5e-7 together.  These have no sign in common with the values, so
    they move a sum of values around 0 by as much of its own size; and 512 rounded adds by sqrt(512) *
    2^-24 / sqrt(3), 7.8e-7.  2.3e-6 of the outputs' root mean square in all (squares added): six times that,
    1.5e-5, is what no output passes.  Sums cut off toward zero 1024 times by 2^-24 of what they have come to,
    two thirds of it in the mean, are 4e-5 off.  (A number is not between two that are rounded to
    bf16 only if it has gone over a border between them.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, Hkv, n = sms, 2, 32768  # a unit a CTA
    c = Cache(B, n, Hkv, D, 64, head_major=True)
    q = (torch.randn(B, Hkv * D, generator=torch.Generator().manual_seed(3)) * 0.1).cuda().bfloat16()
    want = torch.empty(B, Hkv, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        g = torch.Generator(device="cuda").manual_seed(500 + b)
        k, v = (torch.randn(1, n, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        c.append(k, v, [0], n, b0=b)
        one = Cache(1, n, Hkv, D, 64)
        one.append(k, v, [0], n)
        k, v = (x[0].double() for x in one.expand([0], n))
        s = torch.einsum("hd,nhd->hn", q[b].view(Hkv, D).double(), k) / math.sqrt(D)
        assert s.abs().max().item() * math.log2(math.e) < 1.6
        want[b] = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), v)
    out, _, st = decode(c, q, i32([n] * B), "bf16", Hkv)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got, E = out.view(B, Hkv, D).double(), 1.5e-5 * want.square().mean().sqrt()
    over = (got < (want - E).bfloat16().double()) | (got > (want + E).bfloat16().double())
    assert int(over.sum()) == 0, "%d of %d" % (over.sum(), over.numel())
