"""The bounded waits of the decodes over a 4-bit cache and over chosen blocks run out.

As for the dense decode: a hook never brings a CTA's first rows, so the waits for them must run
out.  Every CTA records LAT_ERR_TIMEOUT, drains its copies and exits; a kernel that joins the
pieces, where the shape has one, still runs and ends.  Then the same buffers, a re-zeroed
workspace and the regular calls give correct results.
"""
import time

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import DT, compare, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding
from test_gpu_blocks import f64, i32, room, strides
from test_gpu_q4 import REL, decode, filled

pytestmark = pytest.mark.gpu

BUDGET_NS = 20_000_000


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def runs_out(call, st):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()  # the kernels end by themselves: no fault, no hang
    assert st.item() == binding.LAT_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 2.0


# (B, Hq, Hkv, D, cap): units joined by tickets, whole, wide, and joined by a second kernel
@pytest.mark.parametrize("shape", [(40, 8, 2, 64, 3000), (3, 8, 2, 80, 700), (9, 20, 2, 128, 2000),
                                   (32, 32, 8, 128, 8192), (1, 8, 1, 128, 9000), (2, 16, 1, 512, 4000),
                                   (4, 4, 4, 64, 200)], ids=lambda s: "B%dH%d-%dD%dL%d" % s)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_over_a_4_bit_cache(shape, dt):
    B, Hq, Hkv, D, cap = shape
    lens = [cap - 7 * (b % 3) for b in range(B)]
    if B * cap > 100000:  # (one sequence's rows for all: what is read does not matter here)
        c, kh, vh = filled(1, cap, Hkv, D, lens[:1], dt, 3)
        c.t, c.B = c.t.expand(B, -1, -1, -1).contiguous(), B
        c.strides = (c.t.stride(1), c.t.stride(2), c.t.stride(0))
    else:
        c, kh, vh = filled(B, cap, Hkv, D, lens, dt, 3)
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q")
    nb = binding.lat_attn_decode_q4_workspace_size(DT[dt], B, Hq, Hkv, D, cap)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    out = torch.zeros(B, Hq * D, dtype=q.dtype, device="cuda")
    st, lt = status_tensor(), i32(lens)
    runs_out(lambda: binding.lat_test_decode_q4_timeout(
        DT[dt], q, q.stride(0), c.t, *c.strides, lt, cap, out, out.stride(0), B, Hq, Hkv, D, ws, nb,
        BUDGET_NS, st), st)

    ws.zero_()
    out, lse, st = decode(c, q, lt, dt, Hq, ws=ws)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    n = min(B, kh.shape[0])
    ref, ref_lse = oracle.decode(q[:n].view(n, Hq, D), kh, vh, lens[:n], window=0, scale=D ** -0.5)
    got = out[:n].double().cpu().numpy().reshape(n, Hq, D)
    assert np.abs(got - ref).max() <= REL[dt] * np.abs(vh).max()
    assert np.abs(lse[:n].double().cpu().numpy() - ref_lse).max() <= 1e-4


# (B, Hq, Hkv, D, blocks there are, block, chosen): cut units joined in the kernel, and by another
@pytest.mark.parametrize("shape", [(40, 8, 2, 128, 40, 64, 24), (3, 8, 1, 80, 60, 48, 31), (2, 8, 1, 512, 300, 64, 256),
                                   (5, 12, 3, 64, 30, 16, 9)], ids=lambda s: "B%dH%d-%dD%dn%dx%dof%d" % s)
def test_decode_over_chosen_blocks(shape):
    B, Hq, Hkv, D, have, block, n_sel = shape
    cap = have * block
    lens = [cap - 5 * (b % 3) for b in range(B)]
    k, v = (room(B, cap, Hkv, D, "bf16") for _ in range(2))
    g = np.random.default_rng(5)
    lists = np.stack([np.stack([np.sort(g.choice(have, n_sel, replace=False)) for _ in range(Hkv)])
                      for _ in range(B)]).astype(np.int32)
    for x, role in ((k, "k"), (v, "v")):
        x[:] = W.normal((B, cap, Hkv, D), dtype="bf16", device="cuda", seed=D, role=role)
    q = W.normal((B, Hq * D), dtype="bf16", device="cuda", seed=D, role="q")
    lt, blocks = i32(lens), torch.from_numpy(lists).cuda()
    bf16 = binding.LAT_BF16
    nb = binding.lat_attn_decode_blocks_workspace_size(bf16, B, Hq, Hkv, D, block, n_sel)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    out = torch.zeros(B, Hq * D, dtype=q.dtype, device="cuda")
    st = status_tensor()
    runs_out(lambda: binding.lat_test_decode_blocks_timeout(
        q, q.stride(0), k, v, *strides(k), lt, cap, block, blocks, n_sel, out, out.stride(0), B, Hq, Hkv, D,
        ws, nb, BUDGET_NS, st), st)

    ws.zero_()
    st = status_tensor()
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    binding.lat_attn_decode_blocks(bf16, q, q.stride(0), k, v, *strides(k), lt, cap, block, blocks, n_sel, out,
                                   out.stride(0), lse, B, Hq, Hkv, D, D ** -0.5, 0.0, ws, nb, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in (0, B - 1):
        for h in range(Hkv):
            keys = np.concatenate([np.arange(i * block, min((i + 1) * block, lens[b])) for i in lists[b, h]])
            rows = torch.from_numpy(keys).cuda()
            hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            ref, ref_lse = oracle.decode(f64(q[b].view(Hq, D)[hs])[None], f64(k[b, rows, h])[None, :, None],
                                         f64(v[b, rows, h])[None, :, None], [len(keys)], window=0,
                                         scale=D ** -0.5)
            compare(out[b].view(Hq, D)[hs][None], ref, "bf16", "after a timeout", lse[b, hs][None], ref_lse)
