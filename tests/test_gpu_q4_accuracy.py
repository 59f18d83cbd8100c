"""How near a bf16 decode over the 4-bit cache comes: to the rounding of its output.

Tolerance.  y = sum_j w_j v_j, the w_j positive and of sum 1, |v| <= vmax.  The kernel returns
bf16(y + e), which is off by at most 2^-8 |y| and a little more than |e|.  A weight times a scale
of V is held in two bf16 terms, 2^-16 of it, which moves the mean by 2^-16 vmax.  A score is a
fp32 sum of products of which only the query's channels that are not zero add any error: three
here, one a group, with codes of up to 79 (64 and a nibble) times V's scale s, so that a group's
numbers stay below M = 79 s |q| scale <= 16; four operations a group on them, each off by 2^-22 M
at most (an MMA lines up and truncates), are off by 3 * 4 * 2^-22 * 16 < 2^-14 together, and move
a mean of weights e^x by 2 * 2^-14 vmax.  |e| <= (2^-13 + 2^-16) vmax: with the exponentials' and
the joins' 2^-20, below 1.25 * 2^-13 vmax.  One bf16 term a weight alone is 2^-9 off.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import ensure_library
from test_gpu_q4 import HEAD_DIMS, Cache, decode, filled, held, rows

pytestmark = pytest.mark.gpu

SCALE = 0.05


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def queries(B, Hq, D, seed):
    """Three channels of each head in 1 .. 2 and of either sign, in as many groups of 32 as there
    are; the rest zero."""
    g = np.random.default_rng(seed)
    q = np.zeros((B, Hq, D), np.float32)
    for b in range(B):
        for h in range(Hq):
            for i in range(3):
                d = min(32 * (i % (D // 32)) + int(g.integers(0, 32)), D - 1)
                q[b, h, d] = g.uniform(1, 2) * g.choice([-1, 1])
    return torch.from_numpy(q.reshape(B, Hq * D)).to(torch.bfloat16).cuda()


def check(c, q, lens, Hq, kh, vh, window, what):
    B, D = c.B, c.D
    for d in range(0, D, 32):  # the docstring's M: the 16 codes of a group span its range
        g = kh[..., d:d + 32]
        assert 79 * (np.maximum(g.max(-1), 0) - np.minimum(g.min(-1), 0)).max() / 15 * 2 * SCALE <= 16
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse, st = decode(c, q, lt, "bf16", Hq, window, scale=SCALE)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, _ = oracle.decode(q.view(B, Hq, D), kh, vh, lens, window=window, scale=SCALE)
    got = out.double().cpu().numpy().reshape(B, Hq, D)
    vmax = np.abs(vh).max()
    over = (np.abs(got - ref) - 2.0 ** -8 * np.abs(ref)) / vmax
    assert over.max() <= 1.25 * 2.0 ** -13, "%s: %.2e" % (what, over.max())


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8, 12])
def test_weights_add_no_rounding_that_shows(D, G):
    lens = [1, 2, 3, 5, 8, 16, 17, 40, 65, 130, 300]
    B, Hkv, cap = len(lens), 2, 300
    c, kh, vh = filled(B, cap, Hkv, D, lens, "bf16", 5 * D + G)
    check(c, queries(B, G * Hkv, D, G), lens, G * Hkv, kh, vh, 0, "D%d G%d" % (D, G))


@pytest.mark.parametrize("D", [64, 128, 512])
@pytest.mark.parametrize("G", [4, 6])
@pytest.mark.parametrize("v_mul", [2.0 ** -110, 2.0 ** -60, 2.0 ** 100])
def test_values_far_from_one(D, G, v_mul):
    lens = [2, 3, 5, 17, 40, 130, 300]
    B, Hkv, cap = len(lens), 2, 300
    c = Cache(B, cap, Hkv, D)
    k, v = rows(B, cap, Hkv, D, "bf16", 8, "k"), rows(B, cap, Hkv, D, "bf16", 8, "v") * v_mul
    c.append(k, v, [0] * B, cap)
    check(c, queries(B, G * Hkv, D, G), lens, G * Hkv, held(k), held(v), 0, "D%d G%d" % (D, G))


@pytest.mark.parametrize("G", [2, 4, 7])
def test_long_caches_too(G):
    """The form of head_dim 128 that takes 64 keys a warp at once, units cut and whole."""
    lens = [1, 2, 4, 9, 33, 64, 65, 129, 200, 257, 400, 600] * 2
    B, Hkv, D, cap, n = len(lens), 8, 128, 10240, 600
    c = Cache(B, cap, Hkv, D)
    k, v = rows(B, n, Hkv, D, "bf16", 3, "k"), rows(B, n, Hkv, D, "bf16", 3, "v")
    c.append(k, v, [0] * B, n)
    check(c, queries(B, G * Hkv, D, 3), lens, G * Hkv, held(k), held(v), 0, "long caches, G%d" % G)


@pytest.mark.parametrize("G", [4, 8])
def test_one_unit_over_every_cta(G):
    B, Hkv, D, cap = 1, 1, 128, 9000
    c, kh, vh = filled(B, cap, Hkv, D, [8999], "bf16", 17)
    check(c, queries(B, G, D, 5), [8999], G, kh, vh, 0, "one unit, G%d" % G)
    check(c, queries(B, G, D, 6), [8999], G, kh, vh, 3, "three keys, G%d" % G)
