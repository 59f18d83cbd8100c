"""lat_attn_key_weights: what may lie around its inputs, and the ends of its arguments' ranges."""
import pytest
import torch

import workloads as W
from gpu_helpers import ensure_library
from test_gpu_key_weights import check, definition, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("n_q", [9, 150])
def test_capped_weights_of_a_padded_batch(n_q, window):
    """Queries of rows that see nothing (before a sequence's first position, or of no log-sum-exp), and keys
    that no row sees: whatever they hold, the bits of all others stay."""
    B, Hq, Hkv, D, cap, softcap = 4, 12, 2, 128, 300, 50.0
    lens = [300, 5, 131, 140]
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, "bf16", 4)
    lse = torch.full((B, n_q, Hq), 7.0, device="cuda")
    lse[3, ::2] = float("-inf")
    got = []
    for fill in (0.0, 1.0, 3e4, float("inf"), float("nan")):
        for b, n in enumerate(lens):
            k[b, n:] = fill
            if window > 0:
                k[b, :max(0, n - n_q - window + 1)] = fill
            q[b * n_q:b * n_q + max(0, n_q - n)] = fill
        q[3 * n_q:4 * n_q:2] = fill
        w = torch.zeros(B, Hkv, cap, device="cuda")
        st = run(q, k, lens, "bf16", Hq, Hkv, D, n_q, lse, w, window=window, cap=softcap)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        got.append(w)
    assert all(torch.equal(w, got[0]) for w in got) and bool((got[0] != 0).any())


@pytest.mark.parametrize("D", [64, 80, 128, 256, 512])
@pytest.mark.parametrize("Hq,n_q", [(2, 1), (8, 1), (10, 3), (10, 80), (300, 2)])
def test_capped_weights_hang_on_nothing_else(D, Hq, n_q):
    """The bits stay as they are whatever lies behind the lengths, and whatever an earlier kernel left in
    shared memory, where the columns are no multiple of 16.  Most scores here lie far below the cap,
    what lies around far above."""
    B, Hkv, cap, softcap = 6, 2, 700, 50.0
    lens = [700, 1, 33, 130, 301, 515]
    q, k = inputs(B, Hq, Hkv, D, cap, n_q, "bf16", 3 + D)
    lse = torch.full((B, n_q, Hq), 7.0, device="cuda")
    dirt = [inputs(B, 128, 1, D, cap, n, "bf16", 5) for n in (1, 2, 5)]
    got = []
    for fill in (0.0, 1.0, 3e4, float("inf"), float("nan")):
        for b, n in enumerate(lens):
            k[b, n:] = fill
        for mul in (0.0, 1e4):
            for dq, dk in dirt:  # one tile of columns or more, whole, of zeros or of large queries
                n = dq.shape[0] // B
                run(dq * mul, dk, [cap] * B, "bf16", 128, 1, D, n, torch.full((B, n, 128), 7.0, device="cuda"),
                    torch.zeros(B, 1, cap, device="cuda"))
            w = torch.zeros(B, Hkv, cap, device="cuda")
            st = run(q, k, lens, "bf16", Hq, Hkv, D, n_q, lse, w, cap=softcap)
            torch.cuda.synchronize()
            assert int(st.item()) == 0
            got.append(w)
    assert all(torch.equal(w, got[0]) for w in got)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("Hq,n_q", [(2, 1), (6, 9), (2, 300)])
def test_the_last_keys_that_are_taken(dt, causal, Hq, n_q):
    """A sequence of 2^31 - 128 keys, of which the last are seen.  (Rows begin 16 bytes apart, so each shares all
    but 16 bytes with the next: 34 GB.)"""
    L, D, window, n = 2 ** 31 - 128, 64, 500, 2000
    step = 8 if dt == "bf16" else 4
    q, _ = inputs(1, Hq, 1, D, 1, n_q, dt, 8)
    buf = torch.empty(L * step + D, dtype=q.dtype, device="cuda")
    buf[-n * step - D:] = W.normal((n * step + D,), dtype=dt, device="cuda", seed=4, role="k")
    k = buf.as_strided((1, n, 1, D), (buf.numel() // 8 * 8, step, step, 1), (L - n) * step)
    added, lse, worst = definition(q.reshape(1, n_q, Hq, D), k, [n], n_q, causal, window, D ** -0.5, 0.0)
    w = torch.zeros(1, 1, L, device="cuda")
    whole = buf.as_strided((1, L, 1, D), k.stride())
    st = run(q, whole, [L], dt, Hq, 1, D, n_q, torch.from_numpy(lse).cuda(), w, causal, window)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check(w[:, :, L - n:], torch.zeros(1, 1, n), added, worst, [n], "last keys")
    assert all(int(x.count_nonzero()) == 0 for x in w[0, 0, :L - n].split(1 << 28))
