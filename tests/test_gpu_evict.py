"""lat_kv_evict_choose and lat_kv_evict_rows: everything they write is exact.

The choice is compared with a stable sort of each head's weights, the moved rows with the rows that
the lists name, bit for bit, and every byte that is not to change with what it was.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import DT, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def the_choice(w, n, n_keep, n_first, n_last):
    """Kept keys of one head, ascending: w numpy, n its length."""
    if n <= n_keep:
        return np.arange(n)
    mid = w[n_first:n - n_last].astype(np.float64)
    mid = np.where(np.isnan(mid), np.inf, mid)  # (no infinity among the tests' weights)
    best = np.argsort(-mid, kind="stable")[:n_keep - n_first - n_last] + n_first
    return np.sort(np.concatenate([np.arange(n_first), best, np.arange(n - n_last, n)]))


def choose(w, lens, n_keep, n_first, n_last, out="new", max_len=None, kept=None, new=None, status=None, stream=None):
    B, H, cap = w.shape
    kept = torch.full((B, H, n_keep), -7, dtype=torch.int32, device="cuda") if kept is None else kept
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda") if new is None else new
    o = torch.full_like(w, -7.0) if out == "new" else w if out == "same" else None
    st = status if status is not None else status_tensor()
    binding.lat_kv_evict_choose(w, w.stride(1), w.stride(0), lens if torch.is_tensor(lens) else i32(lens),
                                cap if max_len is None else max_len, kept, n_keep, n_first, n_last, o,
                                0 if o is None else o.stride(1), 0 if o is None else o.stride(0), new, B, H, st,
                                stream=stream)
    return kept, o, new, st


def check_choice(w, lens, n_keep, n_first, n_last, got, what, behind=-7.0):
    kept, o, new, st = (x.cpu().numpy() if x is not None else None for x in got)
    assert st[0] == 0
    wn = w.cpu().numpy()
    for b, n in enumerate(lens):
        assert new[b] == min(n, n_keep), what
        for h in range(w.shape[1]):
            at = the_choice(wn[b, h], n, n_keep, n_first, n_last)
            want = np.full(n_keep, -1)
            want[:len(at)] = at
            assert np.array_equal(kept[b, h], want), "%s: sequence %d head %d" % (what, b, h)
            if o is not None:
                row = np.concatenate([wn[b, h][at], np.zeros(n - len(at), np.float32)])
                assert np.array_equal(o[b, h, :n], row, equal_nan=True), what
                rest = wn[b, h, n:] if behind is None else np.full(w.shape[2] - n, behind, np.float32)
                assert np.array_equal(o[b, h, n:], rest, equal_nan=True), what


def weights(B, H, cap, seed, kind="spread", pad=0):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(3 * torch.randn(B, H, cap + pad, generator=g))
    if kind == "ties":
        w = torch.randint(0, 4, (B, H, cap + pad), generator=g).float()
    elif kind == "equal":
        w = torch.zeros(B, H, cap + pad)
    elif kind == "signed":
        w = torch.randn(B, H, cap + pad, generator=g) * torch.exp(10 * torch.randn(B, H, cap + pad, generator=g))
    elif kind == "near":  # differ in the last places alone
        w = 1.0 + torch.randint(0, 50, (B, H, cap + pad), generator=g) * 2.0 ** -23
    elif kind == "odd":
        w[..., ::5] = 0.0
        w[..., 1::5] = -0.0
        w[..., 2::97] = float("nan")
        w[..., 3::7] = 2.0 ** -140
    return w.cuda()[:, :, :cap]


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "signed", "near", "odd"])
@pytest.mark.parametrize("B,H,cap,lens,n_keep,n_first,n_last", [
    (3, 2, 100, [100, 57, 41], 40, 3, 7),
    (4, 1, 33, [0, 1, 32, 33], 32, 0, 0),
    (2, 3, 5000, [5000, 4097], 1, 0, 0),
    (2, 3, 5000, [5000, 4097], 4096, 4, 64),
    (1, 2, 20000, [19999], 777, 0, 777),        # none is chosen
    (1, 1, 70001, [70001], 33333, 11, 0),
    (5, 1, 9000, [9000, 8999, 1, 4500, 0], 4500, 4500, 0),
])
def test_choice_matches_a_sort(kind, B, H, cap, lens, n_keep, n_first, n_last):
    w = weights(B, H, cap, 3, kind, pad=5)
    was = w.clone()
    got = choose(w, lens, n_keep, n_first, n_last)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(w), torch.nan_to_num(was))
    check_choice(was, lens, n_keep, n_first, n_last, got, kind)
    got = choose(w, lens, n_keep, n_first, n_last, out=None)
    torch.cuda.synchronize()
    check_choice(was, lens, n_keep, n_first, n_last, got, kind + ", no weights")
    got = choose(w, lens, n_keep, n_first, n_last, out="same")  # written over
    torch.cuda.synchronize()
    check_choice(was, lens, n_keep, n_first, n_last, got, kind + ", in place", behind=None)


def test_choice_at_the_largest_length():
    cap = 425984
    w = weights(1, 1, cap, 5)
    got = choose(w, [cap], cap // 3, 4, 64)
    torch.cuda.synchronize()
    check_choice(w, [cap], cap // 3, 4, 64, got, "largest")


def test_lengths_out_of_range_are_left_alone():
    w = weights(4, 2, 64, 5)
    kept, o, new, st = choose(w, [64, 65, -1, 10], 16, 1, 1)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    assert (kept[1:3] == -7).all() and (o[1:3] == -7).all() and (new[1:3] == -7).all()
    st.zero_()
    keep = [0, 3]
    check_choice(w[keep], [64, 10], 16, 1, 1, (kept[keep], o[keep], new[keep], st), "kept")


def caches(B, cap, H, D, dt, seed, head_major=False, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2):
        x = torch.randn(B, cap, H, D + pad, generator=g, device="cuda").to(W.torch_dtype(dt))
        if head_major:
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        out.append(x)
    return out


def move(k, v, kept, dt, D, capacity=None, status=None, stream=None):
    st = status if status is not None else status_tensor()
    B, cap, H, _ = k.shape
    binding.lat_kv_evict_rows(DT[dt], k, v, k.stride(1), k.stride(2), k.stride(0), cap if capacity is None else capacity,
                              kept, kept.shape[2], B, H, D, st, stream=stream)
    return st


def bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 80), ("bf16", 128), ("f32", 80), ("bf16", 512), ("f32", 512)])
@pytest.mark.parametrize("B,H,cap,n_keep,how,head_major", [
    (1, 1, 1, 1, "all", False), (2, 3, 300, 299, "one", False), (3, 2, 700, 233, "some", True),
    (1, 1, 5000, 2500, "some", False), (1, 2, 4100, 4000, "late", False), (2, 1, 900, 640, "last", True),
    (40, 8, 64, 40, "some", False)])
def test_rows_are_the_lists(dt, D, B, H, cap, n_keep, how, head_major):
    pad = 16 if D == 80 else 0
    k, v = caches(B, cap, H, D, dt, D, head_major, pad)
    g = torch.Generator().manual_seed(cap)
    kept = torch.full((B, H, n_keep), -1, dtype=torch.int32)
    for b in range(B):
        for h in range(H):
            n = n_keep - (b % 3)  # lists that end early, too
            at = torch.arange(cap)
            if how == "one":
                at = torch.cat([at[:7], at[8:]])[:n]
            elif how == "some":
                at = torch.randperm(cap, generator=g)[:n].sort().values
            elif how == "late":
                at = at[cap - n:]
            elif how == "last":
                at = torch.cat([at[:n - 1], at[-1:]])
            kept[b, h, :len(at)] = at.int()
    want = []
    for x in (k, v):
        y = x.clone()
        for b in range(B):
            for h in range(H):
                at = kept[b, h][kept[b, h] >= 0].long().cuda()
                y[b, :len(at), h, :D] = x[b, at, h, :D]
        want.append(y)
    st = move(k, v, kept.cuda(), dt, D)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, y in zip((k, v), want):
        assert torch.equal(bits(x.contiguous()), bits(y.contiguous()))


@pytest.mark.parametrize("bad", [[0, 2, 2, 5], [0, 3, 1, 5], [0, 1, 2, 8], [0, 1, -2, 5], [0, 1, -1, 5], [3, 4, 5, 2 ** 31 - 1]])
def test_a_list_that_is_none_is_reported(bad):
    """And no other head is touched by it, nor a row at or past the capacity."""
    B, H, cap, D = 1, 2, 12, 64
    k, v = caches(B, cap, H, D, "bf16", 1)
    was = [k.clone(), v.clone()]
    kept = i32([[[1, 3, 5, 7], bad]])
    st = move(k, v, kept, "bf16", D, capacity=8)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    for x, y in zip((k, v), was):
        assert torch.equal(x[0, :4, 0], y[0, [1, 3, 5, 7], 0]) and torch.equal(x[0, 4:, 0], y[0, 4:, 0])
        assert torch.equal(x[0, 8:], y[0, 8:])


@pytest.mark.parametrize("D", [64, 256])
def test_lists_that_begin_again_stay_below_the_capacity(D):
    """Lists longer than the cache that count up several times: a stretch of rows of its own ends at each."""
    B, H, cap = 1, 2, 700
    k, v = caches(B, 1500, H, D, "bf16", 2)
    was = [k.clone(), v.clone()]
    kept = torch.arange(1300, dtype=torch.int32).remainder(cap)
    kept = torch.stack([kept, torch.arange(1300, dtype=torch.int32) // 2])[None].cuda()
    st = move(k, v, kept, "bf16", D, capacity=cap)
    torch.cuda.synchronize()
    assert int(st.item()) == binding.LAT_ERR_BOUNDS
    for x, y in zip((k, v), was):
        assert torch.equal(x[:, cap:], y[:, cap:])


def test_a_long_cache_past_32_bit_offsets():
    """Rows that come from beyond 2^32 bytes behind the cache's begin."""
    cap, D, n = 4_300_000, 512, 3000
    x = torch.zeros(1, cap, 1, D, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    src = torch.randn(n, D, device="cuda").bfloat16()
    x[0, cap - n:, 0], y[0, cap - n:, 0] = src, -src
    kept = torch.cat([torch.arange(5), torch.arange(cap - n, cap)]).int().cuda().view(1, 1, -1)
    st = move(x, y, kept, "bf16", D)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(x[0, 5:5 + n, 0], src) and torch.equal(y[0, 5:5 + n, 0], -src) and (x[0, :5] == 0).all()


def test_a_prompt_is_cut_down_and_decoded_from():
    """As a server uses it, on one stream: prefill a prompt, sum up what its last rows looked at,
    choose and move, then steps over what is left (append, decode, sum up) that evict again when
    the budget is passed.  Every step's attention is compared with the oracle's over the rows that
    the lists say are there; the kept keys' weights with a sum in 64 bits."""
    B, Hq, Hkv, D, S, cap, budget, steps = 2, 8, 2, 64, 300, 320, 96, 6
    G, scale = Hq // Hkv, D ** -0.5
    g = torch.Generator(device="cuda").manual_seed(4)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    q, kn, vn = rnd(B, S, Hq * D), rnd(B, S, Hkv * D), rnd(B, S, Hkv * D)
    kc, vc = (torch.full((B, cap, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    strides = (kc.stride(1), kc.stride(2), kc.stride(0))
    st, BF = status_tensor(), binding.LAT_BF16
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lens = i32([S] * B)
        binding.lat_kv_append(BF, kc, vc, *strides, cap, kn, vn, Hkv * D, i32([0] * B), S, B, Hkv, D, st)
        out, lse = torch.empty(B * S, Hq * D, dtype=q.dtype, device="cuda"), torch.empty(B, S, Hq, device="cuda")
        binding.lat_attn_prefill(BF, q, Hq * D, kn, Hkv * D, vn, Hkv * D, out, Hq * D, lse, B, S, S, Hq, Hkv, D, 1, 0,
                                 scale, st)
        n_q = 32  # an observation window at the prompt's end
        w = torch.zeros(B, Hkv, cap, device="cuda")
        qw = q[:, S - n_q:].reshape(B * n_q, Hq * D).contiguous()
        lw = lse[:, S - n_q:].contiguous()
        binding.lat_attn_key_weights(BF, qw, Hq * D, n_q, kc, *strides, lens, cap, lw, w, w.stride(1), w.stride(0), B, Hq,
                                     Hkv, D, 1, 0, scale, 0.0, st)
        nb = binding.lat_attn_decode_workspace_size(BF, B, Hq, Hkv, D, cap)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        total = torch.zeros(B, Hkv, cap, dtype=torch.float64)  # the same sums in 64 bits
        k64, v64 = (x.double().cpu() for x in (kc, vc))

        def add(qq, n):  # what n rows' softmaxes give, onto total
            L = int(lens[0])
            for h in range(Hq):
                x = scale * qq[:, :, h] @ k64[:, :L, h // G].transpose(1, 2)
                if n > 1:
                    x = x.masked_fill(torch.arange(L) > (L - n + torch.arange(n))[:, None], -math.inf)
                total[:, h // G, :L] += torch.softmax(x, -1).sum(1)

        add(qw.double().cpu().view(B, n_q, Hq, D), n_q)
        s.synchronize()
        for step in range(steps + 1):
            # over the budget: choose, move, and follow with the copies
            before = [x.cpu() for x in (w, lens)]
            kept, _, new, _ = choose(w, lens, budget, 4, 16, out="same", status=st)
            move(kc, vc, kept, "bf16", D, status=st)
            s.synchronize()
            for b in range(B):
                n = int(before[1][b])
                for h in range(Hkv):
                    at = the_choice(before[0][b, h].numpy(), n, budget, 4, 16)
                    assert np.array_equal(kept[b, h].cpu().numpy()[:len(at)], at)
                    at = torch.from_numpy(at)
                    t = total[b, h, at].clone()
                    total[b, h] = 0
                    total[b, h, :len(at)] = t
                    k64[b, :len(at), h], v64[b, :len(at), h] = k64[b, at, h].clone(), v64[b, at, h].clone()
            lens = new
            # (lse to 1e-3, each weight then to as much; 40 or fewer rows)
            assert (w.double().cpu() - total).abs().max() <= 2e-3 * total.max()
            pos = lens.clone()
            kt, vt, qt = rnd(B, Hkv * D), rnd(B, Hkv * D), rnd(B, Hq * D)
            binding.lat_kv_append(BF, kc, vc, *strides, cap, kt, vt, Hkv * D, pos, 1, B, Hkv, D, st)
            L = int(pos[0])
            k64[:, L], v64[:, L] = kt.double().cpu().view(B, Hkv, D), vt.double().cpu().view(B, Hkv, D)
            lens = lens + 1
            out, lse = torch.empty(B, Hq * D, dtype=q.dtype, device="cuda"), torch.empty(B, Hq, device="cuda")
            binding.lat_attn_decode(BF, qt, Hq * D, kc, vc, *strides, lens, cap, out, Hq * D, lse, B, Hq, Hkv, D, 0, scale,
                                    ws, nb, st)
            binding.lat_attn_key_weights(BF, qt, Hq * D, 1, kc, *strides, lens, cap, lse, w, w.stride(1), w.stride(0), B,
                                         Hq, Hkv, D, 1, 0, scale, 0.0, st)
            s.synchronize()
            add(qt.double().cpu().view(B, 1, Hq, D), 1)
            ref, _ = oracle.decode(qt.view(B, Hq, D), k64.nan_to_num().numpy(), v64.nan_to_num().numpy(), [L + 1] * B,
                                   window=0, scale=scale)
            err = np.abs(out.double().cpu().numpy().reshape(B, Hq, D) - ref).max()
            assert err <= 2.0 ** -7 * float(v64.nan_to_num().abs().max())
        assert int(st.item()) == 0


def test_kept_rows_enter_the_8_bit_cache():
    """A prompt's kept rows quantised and decoded from: what the two caches have in common."""
    Hq, Hkv, D, S, n_keep, block = 8, 2, 128, 200, 70, 32
    k, v = caches(1, S, Hkv, D, "bf16", 8)
    kept, _, new, st = choose(weights(1, Hkv, S, 2), [S], n_keep, 2, 8)
    want = [x[0, kept[0, h].long(), h] for x in (k, v) for h in range(Hkv)]
    move(k, v, kept, "bf16", D, status=st)
    rb = binding.lat_kv_q8_block_bytes(D, block)
    c = torch.zeros(1, 3, Hkv, rb, dtype=torch.uint8, device="cuda")
    strides = (c.stride(1), c.stride(2), c.stride(0))
    binding.lat_kv_append_q8(binding.LAT_BF16, c, *strides, block, 96, k, v, Hkv * D, i32([0]), n_keep, 1, Hkv, D, st)
    gk, gv = (torch.empty(n_keep, Hkv * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    binding.lat_kv_expand_q8(binding.LAT_BF16, c, *strides, block, 96, gk, gv, Hkv * D, i32([0]), n_keep, 1, Hkv, D, st)
    q = W.normal((1, Hq * D), dtype="bf16", device="cuda", seed=2, role="q")
    nb = binding.lat_attn_decode_q8_workspace_size(binding.LAT_BF16, 1, Hq, Hkv, D, 96)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    out = torch.empty(1, Hq * D, dtype=torch.bfloat16, device="cuda")
    binding.lat_attn_decode_q8(binding.LAT_BF16, q, Hq * D, c, *strides, block, new, 96, out, Hq * D, None, 1, Hq, Hkv, D,
                               0, D ** -0.5, 0.0, ws, nb, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, w in zip([y.view(n_keep, Hkv, D)[:, h] for y in (gk, gv) for h in range(Hkv)], want):
        assert ((x.float() - w.float()).abs() <= 2.0 ** -4 * w.float().abs() + 2.0 ** -9 * w.float().abs().max() / 224).all()
    ref, _ = oracle.decode(q.view(1, Hq, D), gk.double().cpu().view(1, n_keep, Hkv, D).numpy(),
                           gv.double().cpu().view(1, n_keep, Hkv, D).numpy(), [n_keep], window=0, scale=D ** -0.5)
    err = np.abs(out.double().cpu().numpy().reshape(1, Hq, D) - ref).max()
    assert err <= (2.0 ** -8 + 2.0 ** -10) * float(gv.abs().max())


def test_choice_and_rows_in_a_graph_and_on_two_streams():
    B, H, cap, D, n_keep = 3, 2, 6000, 64, 1500
    w = weights(B, H, cap, 9)
    lens = i32([6000, 1500, 4000])
    k, v = caches(B, cap, H, D, "bf16", 5)
    ref = choose(w, lens, n_keep, 4, 32)
    rk, rv = k.clone(), v.clone()
    move(rk, rv, ref[0], "bf16", D)
    torch.cuda.synchronize()
    got = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                a, b = k.clone(), v.clone()
                c = choose(w, lens, n_keep, 4, 32, stream=s)
                move(a, b, c[0], "bf16", D, stream=s)
                got.append((a, b, c))
    torch.cuda.synchronize()
    a, b = k.clone(), v.clone()
    st = status_tensor()
    kept, new = torch.zeros(B, H, n_keep, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = choose(w, lens, n_keep, 4, 32, out=None, kept=kept, new=new, status=st)
        move(a, b, kept, "bf16", D, status=st)
    a.copy_(k)
    b.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, y, z in got + [(a, b, (kept, None, new))]:
        assert torch.equal(x, rk) and torch.equal(y, rv) and torch.equal(z[0], ref[0]) and torch.equal(z[2], ref[2])


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f32", 512)])
def test_the_waits_of_the_rows_run_out(dt, D):
    """A hook keeps one CTA of each cluster silent: LAT_ERR_TIMEOUT, and the next call is right."""
    B, H, cap, n = 2, 2, 3000, 2000
    k, v = caches(B, cap, H, D, dt, 3)
    kept = torch.arange(0, 2 * n, 2, dtype=torch.int32)[:n].clamp(max=cap - 1)
    kept = torch.unique(kept)
    kept = torch.cat([kept, torch.full((n - len(kept),), -1, dtype=torch.int32)]).expand(B, H, n).contiguous().cuda()
    was = [k.clone(), v.clone()]
    st = status_tensor()
    binding.lat_test_evict_rows_timeout(DT[dt], k, v, k.stride(1), k.stride(2), k.stride(0), cap, kept, n, B, H, D,
                                        20_000_000, st)
    torch.cuda.synchronize()  # the kernel ends by itself: no fault, no hang
    assert int(st.item()) == binding.LAT_ERR_TIMEOUT
    assert torch.equal(k, was[0]) and torch.equal(v, was[1])
    st = move(k, v, kept, dt, D)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    m = int((kept[0, 0] >= 0).sum())
    at = kept[0, 0, :m].long()
    for x, y in zip((k, v), was):
        assert torch.equal(x[:, :m], y[:, at]) and torch.equal(x[:, m:], y[:, m:])
