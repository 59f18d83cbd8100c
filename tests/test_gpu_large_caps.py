"""Score caps far above every score, up to the largest float: as no cap, for the decodes over
reduced caches.  Tolerances: those decodes' own."""
import pytest
import torch

import workloads as W
from gpu_helpers import ensure_library
from test_gpu_blocks import check_decode as check_blocks
from test_gpu_blocks import decode as decode_blocks
from test_gpu_blocks import i32
from test_gpu_q4 import check_decode, decode, filled

pytestmark = pytest.mark.gpu

CAPS = [1e6, 1e30, 1e37, 2.4e38, 3.4028234663852886e38]


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_4_bit_cache(cap, dt):
    B, Hq, Hkv, D, lens = 2, 8, 2, 80, [150, 31]
    c, kh, vh = filled(B, 150, Hkv, D, lens, dt, 3)
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q")
    out, lse, st = decode(c, q, i32(lens), dt, Hq, softcap=cap)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, kh, vh, lens, dt, Hq, D, 0, 0.0, "cap %g" % cap)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_chosen_blocks(cap, dt):
    B, Hq, Hkv, D, n, block = 2, 8, 2, 128, 160, 32
    k, v = (W.normal((B, n, Hkv, D), dtype=dt, device="cuda", seed=4, role=r) for r in "kv")
    q = W.normal((B, Hq * D), dtype=dt, device="cuda", seed=2, role="q")
    lists = i32([[[0, 2, 4]] * Hkv] * B)
    out, lse, st = decode_blocks(q, k, v, [n, n], block, lists, Hq, D, dt, softcap=cap)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_blocks(out, lse, q, k, v, [n, n], block, lists, Hq, D, dt)
