"""Score caps down to the least float: capped scores are as good as 0, and a softmax of them a mean.

Tolerance: with every score within 2^-100 of 0 the output is the mean of the visible values; the
bounds of the decodes' own tests hold (one rounding to bf16 and 2^-11 of the largest value, or
2e-5 of it in fp32), and lse is log n within 1e-4.
"""
import math

import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DT, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding
from test_gpu_blocks import i32, strides
from test_gpu_q4 import REL, decode, filled

pytestmark = pytest.mark.gpu

CAPS = [2.0 ** -149, 1e-40, 1e-38, 1e-30]


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def half_zero(B, Hq, D, dt):
    q = W.normal((B, Hq, D), dtype=dt, device="cuda", seed=2, role="q")
    q[:, ::2] = 0.0
    return q.view(B, Hq * D)


def is_mean(out, lse, vh, n, dt, Hq, D):
    """vh [B, n, Hkv, D]"""
    mean = vh[:, :n].mean(1)
    got = out.double().cpu().numpy().reshape(-1, Hq, D)
    ref = np.repeat(mean, Hq // mean.shape[1], axis=1)
    assert np.abs(got - ref).max() <= REL[dt] * np.abs(vh).max()
    assert np.abs(lse.double().cpu().numpy() - math.log(n)).max() <= 1e-4


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 512])
def test_a_4_bit_cache(cap, dt, D):
    B, Hq, Hkv, n = 2, 8, 2, 150
    c, kh, vh = filled(B, n, Hkv, D, [n] * B, dt, 3)
    out, lse, st = decode(c, half_zero(B, Hq, D, dt), i32([n] * B), dt, Hq, softcap=cap, scale=1.0)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    is_mean(out, lse, vh, n, dt, Hq, D)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("listed", [True, False])
def test_a_cache_and_chosen_blocks_of_it(cap, dt, listed):
    B, Hq, Hkv, D, n, block = 2, 8, 2, 128, 160, 32
    k, v = (W.normal((B, n, Hkv, D), dtype=dt, device="cuda", seed=4, role=r) for r in "kv")
    q, lens, st = half_zero(B, Hq, D, dt), i32([n] * B), status_tensor()
    out, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    if listed:
        lists = i32([[[0, 2, 3]] * Hkv] * B)
        nb = binding.lat_attn_decode_blocks_workspace_size(DT[dt], B, Hq, Hkv, D, block, 3)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        binding.lat_attn_decode_blocks(DT[dt], q, Hq * D, k, v, *strides(k), lens, n, block, lists, 3, out, Hq * D,
                                       lse, B, Hq, Hkv, D, 1.0, cap, ws, nb, st)
        v, n = torch.cat([v[:, :32], v[:, 64:128]], 1), 96
    else:
        nb = binding.lat_attn_decode_workspace_size(DT[dt], B, Hq, Hkv, D, n)
        ws = torch.zeros(max(nb, 256), dtype=torch.uint8, device="cuda")
        binding.lat_attn_decode_softcap(DT[dt], q, Hq * D, k, v, *strides(k), lens, n, out, Hq * D, lse, B, Hq, Hkv, D,
                                        0, 1.0, cap, ws, nb, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    is_mean(out, lse, v.double().cpu().numpy(), n, dt, Hq, D)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_prefill(cap, dt):
    B, S, Hq, Hkv, D = 1, 100, 4, 2, 128
    inp = W.prefill_inputs(B, S, S, Hq, Hkv, D, dtype=dt, device="cuda")
    q = half_zero(S, Hq, D, dt)
    out, lse, st = torch.empty_like(q), torch.empty(S, Hq, device="cuda"), status_tensor()
    binding.lat_attn_prefill_softcap(DT[dt], q, Hq * D, inp.k, inp.k.stride(0), inp.v, inp.v.stride(0), out, Hq * D, lse,
                                     B, S, S, Hq, Hkv, D, 0, 0, 1.0, cap, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    is_mean(out, lse, np.broadcast_to(inp.v[:, :Hkv * D].double().cpu().numpy().reshape(1, S, Hkv, D),
                                      (S, S, Hkv, D)), S, dt, Hq, D)
