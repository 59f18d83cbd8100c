"""lat_attn_key_weights against its definition in 64 bits.

Tolerance.  A weight e^(s - lse) moves by a factor e^d when its exponent is off by d.  The score is
an fp32 sum of D products (exact for bf16, rounded for fp32) whose error is at most D * 2^-23 *
scale * sum |q_d k_d| (D additions and D products of half a step each); a cap only shrinks it.  The
log-sum-exp and the factors of log2(e) round to 2^-24 of |s| + |lse| each, the exponential to
2^-22 of itself.  Sums of positive terms add 2^-22.  TOL computes that bound from the
inputs of each test; the sum that was there before adds its own rounding, 2^-24 of the result.
"""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DT, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(x):
    return x.double().cpu().numpy()


def definition(q, k, lens, n_q, causal, window, scale, cap, lse=None):
    """q [B, n_q, Hq, D], k [B, cap, Hkv, D] -> (added weights [B, Hkv, cap], lse [B, n_q, Hq] as
    fp32, the largest error of an exponent).  The log-sum-exp is the rows' own unless given."""
    q, k = f64(q), f64(k)
    B, _, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    added = np.zeros((B, Hkv, k.shape[1]))
    out = np.full((B, n_q, Hq), -np.inf, dtype=np.float32) if lse is None else lse
    worst = 0.0
    for b, L in enumerate(lens):
        if L < 1:
            continue
        pos = (L - n_q + np.arange(n_q))[:, None]
        j = np.arange(L)[None, :]
        seen = (pos >= 0) & (j <= pos if causal else j >= 0)
        if window > 0:
            seen &= pos - j < window
        for h in range(Hq):
            kk = k[b, :L, h // G]
            s = scale * (q[b, :, h] @ kk.T)
            mag = abs(scale) * (np.abs(q[b, :, h]) @ np.abs(kk).T)
            if cap > 0:
                s = cap * np.tanh(s / cap)
            s = np.where(seen, s, -np.inf)
            if lse is None:
                m = s.max(-1)
                m = np.where(np.isfinite(m), m, 0)
                with np.errstate(divide="ignore"):
                    out[b, :, h] = (m + np.log(np.exp(s - m[:, None]).sum(-1))).astype(np.float32)
            l = out[b, :, h].astype(np.float64)
            live = seen & np.isfinite(l)[:, None]
            x = np.where(live, s - np.where(np.isfinite(l), l, 0)[:, None], -np.inf)
            added[b, h // G, :L] += np.exp(x).sum(0)
            if live.any():
                near = live & (x > -40)  # (what is left of others is nothing)
                if near.any():
                    a = np.where(near, D * 2.0 ** -23 * mag + 2.0 ** -23 * (np.abs(np.where(near, s, 0)) + np.abs(np.where(np.isfinite(l), l, 0))[:, None]), 0)
                    worst = max(worst, a.max())
    return added, out, worst


def run(q, k, lens, dt, Hq, Hkv, D, n_q, lse, w, causal=1, window=0, scale=None, cap=0.0, max_len=None, status=None,
        stream=None):
    st = status if status is not None else status_tensor()
    binding.lat_attn_key_weights(DT[dt], q, q.stride(0), n_q, k, k.stride(1), k.stride(2), k.stride(0),
                                 lens if torch.is_tensor(lens) else i32(lens), k.shape[1] if max_len is None else max_len,
                                 lse, w, w.stride(1), w.stride(0), k.shape[0], Hq, Hkv, D, causal, window,
                                 D ** -0.5 if scale is None else scale, cap, st, stream=stream)
    return st


def inputs(B, Hq, Hkv, D, cap, n_q, dt, seed, head_major=False, pad=16):
    """Queries in padded rows, keys of unequal channels, rows at and past the lengths to be set NaN."""
    full = W.normal((B * n_q, Hq * D + pad), dtype=dt, device="cuda", seed=seed, role="q")
    k = W.normal((B, cap, Hkv, D), dtype="f32", device="cuda", seed=seed, role="k")
    k = (k * torch.linspace(0.3, 2.0, D, device="cuda") + 0.3).to(W.torch_dtype(dt))
    if head_major:
        k = k.transpose(1, 2).contiguous().transpose(1, 2)
    return full[:, :Hq * D], k


def check(got, was, added, worst, lens, what):
    g, w = got.double().cpu().numpy(), was.double().cpu().numpy()
    want = w + added
    tol = added * (np.expm1(worst) + 2.0 ** -20) + want * 2.0 ** -23
    for b, n in enumerate(lens):
        n = max(n, 0)
        assert np.isfinite(g[b, :, :n]).all(), what
        off = np.abs(g[b, :, :n] - want[b, :, :n]) - tol[b, :, :n]
        assert off.max(initial=-1.0) <= 0, "%s: sequence %d, %.3e over" % (what, b, off.max())
        assert np.array_equal(g[b, :, n:], w[b, :, n:]), what + ": entries behind"


def start(B, Hkv, cap, seed, pad=0):
    w = torch.rand(B, Hkv, cap + pad, generator=torch.Generator().manual_seed(seed)).cuda() * 0.1
    return w[:, :, :cap]


# (B, Hq, Hkv, D, cap, n_q, lens, causal, window, softcap, head_major)
SHAPES = [
    (1, 1, 1, 64, 1, 1, [1], 1, 0, 0.0, False),
    (6, 8, 2, 64, 300, 1, [0, 1, 127, 128, 129, 300], 1, 0, 0.0, False),
    (3, 32, 8, 128, 700, 1, [700, 33, 256], 1, 0, 0.0, True),
    (3, 12, 2, 80, 515, 1, [515, 1, 400], 1, 100, 30.0, False),
    (2, 16, 2, 256, 400, 3, [400, 2], 1, 0, 0.0, False),         # more rows than a sequence has
    (2, 16, 2, 512, 300, 4, [300, 129], 1, 0, 0.0, True),
    (2, 20, 4, 128, 600, 25, [600, 311], 1, 0, 0.0, False),      # 125 columns: the last 16 are not whole
    (2, 8, 2, 128, 900, 64, [900, 70], 1, 0, 0.0, False),        # 256 columns, all in one tile
    (2, 8, 2, 128, 900, 65, [900, 64], 1, 0, 0.0, False),        # 260: keys stay
    (1, 8, 4, 64, 1000, 1000, [1000], 1, 0, 0.0, False),         # a whole prompt
    (2, 6, 2, 80, 500, 500, [500, 260], 1, 130, 0.0, True),      # one, and more rows than the other has
    (1, 4, 2, 256, 700, 600, [700], 1, 0, 20.0, False),
    (1, 4, 1, 512, 400, 333, [400], 1, 50, 0.0, False),
    (2, 4, 2, 128, 400, 90, [400, 399], 0, 0, 0.0, False),       # not causal
    (2, 4, 2, 128, 400, 90, [400, 399], 0, 33, 0.0, False),
    (2, 300, 1, 64, 200, 2, [200, 1], 1, 0, 0.0, False),         # more heads than a tile has columns
    (1, 200, 1, 128, 260, 1, [260], 1, 0, 0.0, False),
    (40, 4, 4, 64, 90, 1, [1 + (37 * b) % 90 for b in range(40)], 1, 0, 0.0, False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%dH%d-%dD%dL%dq%d%sW%dC%g%s" % (
    s[0], s[1], s[2], s[3], s[4], s[5], "" if s[7] else "n", s[8], s[9], "h" if s[10] else ""))
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_matches_the_definition(shape, dt):
    B, Hq, Hkv, D, cap, n_q, lens, causal, window, softcap, hm = shape
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, dt, 31 + D, hm)
    added, lse, worst = definition(q.reshape(B, n_q, Hq, D), k, lens, n_q, causal, window, D ** -0.5, softcap)
    for b, n in enumerate(lens):
        k[b, n:] = float("nan")
    w = start(B, Hkv, cap, 5, pad=3)
    was = w.clone()
    st = run(q, k, lens, dt, Hq, Hkv, D, n_q, torch.from_numpy(lse).cuda(), w, causal, window, cap=softcap)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check(w, was, added, worst, lens, str(shape))
    # every row's weights sum to one: so do all of a sequence's
    for b, n in enumerate(lens):
        rows = min(n, n_q) * Hq
        total = float((w[b] - was[b]).double().sum())
        assert abs(total - rows) <= rows * (np.expm1(worst) + 1e-4) + 1e-9


@pytest.mark.parametrize("D,n_q", [(64, 1), (128, 1), (128, 40), (256, 200)])
def test_every_length_around_a_tile(D, n_q):
    lens = [0, 1, 2, 15, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 383, 384, 385]
    B, Hq, Hkv, cap = len(lens), 6, 2, 385
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, "bf16", D)
    added, lse, worst = definition(q.reshape(B, n_q, Hq, D), k, lens, n_q, 1, 0, D ** -0.5, 0.0)
    w = start(B, Hkv, cap, 6)
    was = w.clone()
    st = run(q, k, lens, "bf16", Hq, Hkv, D, n_q, torch.from_numpy(lse).cuda(), w)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check(w, was, added, worst, lens, "D%d q%d" % (D, n_q))


@pytest.mark.parametrize("D,n_q,window", [(64, 1, 0), (80, 2, 50), (128, 1, 0), (128, 5, 140), (256, 1, 0), (256, 20, 0),
                                          (512, 1, 0), (512, 9, 0)])
def test_many_short_sequences(D, n_q, window):
    """A CTA's share is a dozen or more (sequence, head)s of one or two tiles, empty ones between."""
    B, Hq, Hkv, cap = 900, 4, 2, 200
    lens = [(b * 89) % 201 if b % 7 else 0 for b in range(B)]
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, "bf16", 17 + D)
    added, lse, worst = definition(q.reshape(B, n_q, Hq, D), k, lens, n_q, 1, window, D ** -0.5, 0.0)
    w = start(B, Hkv, cap, 7)
    was = w.clone()
    st = run(q, k, lens, "bf16", Hq, Hkv, D, n_q, torch.from_numpy(lse).cuda(), w, window=window)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check(w, was, added, worst, lens, "D%d q%d" % (D, n_q))


@pytest.mark.parametrize("D", [64, 80, 128, 256, 512])
@pytest.mark.parametrize("Hq,Hkv,n_q", [(2, 2, 1), (6, 2, 1), (6, 1, 1), (4, 2, 3), (6, 2, 9)])
@pytest.mark.parametrize("odd", [False, True])
def test_32_bit_rows_at_any_stride_and_address(D, Hq, Hkv, n_q, odd):
    """One column to 27, whole stretches of keys and what is left of one, a window that begins in either."""
    B, cap, lens, window = 3, 1100, [1100, 517, 2], 900
    q0, k0 = inputs(B, Hq, Hkv, D, cap, n_q, "f32", 5 + D, pad=0)
    pad = 3 if odd else 4
    q = torch.full((B * n_q, Hq * D + 2 * pad), float("nan"), device="cuda")[:, pad:pad + Hq * D]
    k = torch.full((B, cap, Hkv, D + 2 * pad), float("nan"), device="cuda")[..., pad:pad + D]
    q.copy_(q0), k.copy_(k0)
    added, lse, worst = definition(q.reshape(B, n_q, Hq, D), k, lens, n_q, 1, window, D ** -0.5, 30.0)
    for b, n in enumerate(lens):
        k[b, n:] = float("nan")
    w = start(B, Hkv, cap, 8, pad=5)
    was = w.clone()
    st = run(q, k, lens, "f32", Hq, Hkv, D, n_q, torch.from_numpy(lse).cuda(), w, window=window, cap=30.0)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check(w, was, added, worst, lens, "D%d q%d" % (D, n_q))


@pytest.mark.parametrize("B,Hq,Hkv,D,cap,n_q,window", [(1, 12, 1, 64, 200, 200, 0), (1, 12, 1, 80, 200, 3, 0),
                                                       (3, 10, 2, 128, 150, 90, 0), (1, 3, 3, 256, 513, 333, 40),
                                                       (2, 9, 1, 512, 70, 70, 0), (2, 6, 2, 64, 1000, 11, 0)])
def test_32_bit_columns_shared_by_ctas(B, Hq, Hkv, D, cap, n_q, window):
    """Few keys and many columns: 2, 4 or 8 CTAs share a key's, some of them without any."""
    lens = [cap, 1, cap // 2][:B]
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, "f32", 3 + D)
    added, lse, worst = definition(q.reshape(B, n_q, Hq, D), k, lens, n_q, 1, window, D ** -0.5, 0.0)
    for b, n in enumerate(lens):
        k[b, n:] = float("nan")
    w = start(B, Hkv, cap, 9, pad=1)
    was, again = w.clone(), w.clone()
    lse = torch.from_numpy(lse).cuda()
    st = run(q, k, lens, "f32", Hq, Hkv, D, n_q, lse, w, window=window)
    run(q, k, lens, "f32", Hq, Hkv, D, n_q, lse, again, window=window, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(w, again)
    check(w, was, added, worst, lens, "D%d q%d" % (D, n_q))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [1, 300])
def test_rows_without_a_log_sum_exp_give_nothing(dt, n_q):
    """-inf among the rows' log-sum-exps, and rows whose weights leave fp32 on the low side."""
    B, Hq, Hkv, D, cap = 2, 4, 2, 128, 300
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, dt, 3)
    _, lse, _ = definition(q.reshape(B, n_q, Hq, D), k, [cap] * B, n_q, 1, 0, D ** -0.5, 0.0)
    lse[0, ::2, 1] = -np.inf
    lse[1, 0, 2] = 3e38
    added, _, worst = definition(q.reshape(B, n_q, Hq, D), k, [cap] * B, n_q, 1, 0, D ** -0.5, 0.0, lse)
    w = start(B, Hkv, cap, 6)
    was = w.clone()
    run(q, k, [cap] * B, dt, Hq, Hkv, D, n_q, torch.from_numpy(lse).cuda(), w)
    torch.cuda.synchronize()
    check(w, was, added, worst, [cap] * B, "no log-sum-exp")


def test_nan_stays_with_its_key_or_its_head():
    """A NaN key makes its own weight NaN; a NaN query every key's of its head that it sees."""
    B, Hq, Hkv, D, cap, n_q = 2, 4, 2, 64, 200, 2
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, "bf16", 3)
    lse = torch.full((B, n_q, Hq), 5.0, device="cuda")
    k[0, 7, 1, 3] = float("nan")
    q[3, 2 * D] = float("nan")  # sequence 1, row 1, head 2
    w = torch.zeros(B, Hkv, cap, device="cuda")
    run(q, k, [cap, 150], "bf16", Hq, Hkv, D, n_q, lse, w)
    bad = torch.isnan(w)
    assert bad[0, 1, 7] and int(bad[0].sum()) == 1
    assert bad[1, 1, :150].all() and int(bad[1].sum()) == 150


def test_lengths_out_of_range_leave_their_weights_alone():
    B, Hq, Hkv, D, cap = 4, 4, 2, 128, 200
    for dt in ("bf16", "f32"):
        q, k = inputs(B, Hq, Hkv, D, cap, 1, dt, 3)
        lens = [200, 201, -1, 10]
        added, lse, worst = definition(q.reshape(B, 1, Hq, D), k, [200, 0, 0, 10], 1, 1, 0, D ** -0.5, 0.0)
        w = start(B, Hkv, cap, 6)
        was = w.clone()
        st = run(q, k, lens, dt, Hq, Hkv, D, 1, torch.from_numpy(lse).cuda(), w)
        torch.cuda.synchronize()
        assert int(st.item()) == binding.LAT_ERR_BOUNDS
        check(w, was, added, worst, [200, 0, 0, 10], dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nothing_cached_anywhere(dt):
    B, Hq, Hkv, D = 2, 4, 2, 64
    q, k = inputs(B, Hq, Hkv, D, 16, 1, dt, 3)
    w = start(B, Hkv, 16, 6)
    was = w.clone()
    for mk in (0, 16):
        st = run(q, k, [0, 0], dt, Hq, Hkv, D, 1, torch.zeros(B, Hq, device="cuda"), w, max_len=mk)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.equal(w, was)


def test_the_same_call_gives_the_same_bits():
    """Two streams at once and a replayed graph, few columns and many."""
    B, Hq, Hkv, D, cap = 3, 8, 2, 128, 3000
    for n_q in (1, 700):
        q, k = inputs(B, Hq, Hkv, D, cap, n_q, "bf16", 3)
        lens = i32([3000, 1, 2049])
        lse = torch.full((B, n_q, Hq), 9.0, device="cuda")
        first = torch.zeros(B, Hkv, cap, device="cuda")
        run(q, k, lens, "bf16", Hq, Hkv, D, n_q, lse, first)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for _ in range(4):
            for s in streams:
                with torch.cuda.stream(s):
                    w = torch.zeros(B, Hkv, cap, device="cuda")
                    run(q, k, lens, "bf16", Hq, Hkv, D, n_q, lse, w, stream=s)
                    got.append(w)
        torch.cuda.synchronize()
        w = torch.zeros(B, Hkv, cap, device="cuda")
        st = status_tensor()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(q, k, lens, "bf16", Hq, Hkv, D, n_q, lse, w, status=st)
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, first) for x in got + [w]) and int(st.item()) == 0


def test_after_the_librarys_own_attention():
    """The log-sum-exps of a prefill and of a decode step, as they come."""
    B, Hq, Hkv, D, cap, S = 2, 8, 2, 128, 512, 400
    q, k = inputs(B, Hq, Hkv, D, cap, S, "bf16", 9, pad=0)
    v = torch.randn_like(k)
    st = status_tensor()
    out, lse = torch.empty_like(q), torch.empty(B, S, Hq, device="cuda")
    binding.lat_attn_prefill_cached(binding.LAT_BF16, q, q.stride(0), k, v, k.stride(1), k.stride(2), k.stride(0), out,
                                    out.stride(0), lse, B, S, S, Hq, Hkv, D, 1, 0, D ** -0.5, st)
    w = torch.zeros(B, Hkv, cap, device="cuda")
    run(q, k, [S] * B, "bf16", Hq, Hkv, D, S, lse, w, status=st)
    q1 = q[:B].contiguous()
    nb = binding.lat_attn_decode_workspace_size(binding.LAT_BF16, B, Hq, Hkv, D, cap)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    out1, lse1 = torch.empty(B, Hq * D, dtype=q.dtype, device="cuda"), torch.empty(B, Hq, device="cuda")
    lens = i32([S, S])
    binding.lat_attn_decode(binding.LAT_BF16, q1, q1.stride(0), k, v, k.stride(1), k.stride(2), k.stride(0), lens, cap,
                            out1, out1.stride(0), lse1, B, Hq, Hkv, D, 0, D ** -0.5, ws, nb, st)
    w1 = torch.zeros(B, Hkv, cap, device="cuda")
    run(q1, k, lens, "bf16", Hq, Hkv, D, 1, lse1, w1, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, qq, n in ((w, q, S), (w1, q1, 1)):
        added, _, worst = definition(qq.reshape(B, n, Hq, D), k, [S] * B, n, 1, 0, D ** -0.5, 0.0)
        # (the library's log-sum-exp is held to 1e-3 by its own tests)
        assert (np.abs(f64(x) - added) <= added * (np.expm1(worst) + 1.001e-3) + 1e-9).all()


@pytest.mark.parametrize("n_q", [1, 300])
def test_the_waits_run_out(n_q):
    """A hook never brings a CTA's first rows: LAT_ERR_TIMEOUT, and the next call is right."""
    B, Hq, Hkv, D, cap = 3, 8, 2, 128, 2000
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, "bf16", 3)
    lens = [2000, 1500, 300]
    added, lse, worst = definition(q.reshape(B, n_q, Hq, D), k, lens, n_q, 1, 0, D ** -0.5, 0.0)
    lse = torch.from_numpy(lse).cuda()
    w, st = start(B, Hkv, cap, 6), status_tensor()
    was = w.clone()
    binding.lat_test_key_weights_timeout(q, q.stride(0), n_q, k, k.stride(1), k.stride(2), k.stride(0), i32(lens), cap,
                                         lse, w, w.stride(1), w.stride(0), B, Hq, Hkv, D, 20_000_000, st)
    torch.cuda.synchronize()  # the kernel ends by itself: no fault, no hang
    assert int(st.item()) == binding.LAT_ERR_TIMEOUT
    w.copy_(was)
    st = run(q, k, lens, "bf16", Hq, Hkv, D, n_q, lse, w)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check(w, was, added, worst, lens, "after a timeout")
