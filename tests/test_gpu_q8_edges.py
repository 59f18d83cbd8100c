"""The 8-bit cache's calls at the ends of their arguments' ranges."""
import pytest
import torch

import workloads as W
from gpu_helpers import DT, ensure_library, status_tensor
from gqa_attention_lat_gb300 import binding
from oracle import q8
from test_gpu_q8 import Cache, assert_same, check_decode, decode, f64, held, i32, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 80])
def test_the_last_rows_that_an_int_can_say(dt, block, D):
    """Into and out of the last block of a cache of 2^31 - 1 rows, all of it and then two rows again.  (The
    blocks before are not looked at, so records 16 bytes apart will do: the last one's are its own.)"""
    Hkv, cap = 2, 2 ** 31 - 1
    first, n = cap // block * block, block - 1  # rows of the block
    rb = binding.lat_kv_q8_block_bytes(D, block)
    at = first // block * 16
    t = torch.full((at + Hkv * rb + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    strides, st = (16, rb, t.numel() // 16 * 16), status_tensor()
    want = [q8.Rows(block, Hkv, D, block) for _ in range(2)]
    for pos, m in ((0, n), (n - 2, 2)):
        new = [rows(1, m, Hkv, D, dt, 5 + m, r) * (1 if m == n else 64) for r in ("k", "v")]
        binding.lat_kv_append_q8(DT[dt], t, *strides, block, cap, *new, Hkv * D, i32([first + pos]), m, 1, Hkv, D, st)
        for w, x in zip(want, new):
            w.append(f64(x[0]), pos)
        got = [torch.empty(n, Hkv * D, dtype=W.torch_dtype(dt), device="cuda") for _ in range(2)]
        binding.lat_kv_expand_q8(DT[dt], t, *strides, block, cap, *got, Hkv * D, i32([first]), n, 1, Hkv, D, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        for x, w, what in zip(got, want, "KV"):
            assert_same(x.view(n, Hkv, D), w.value[:n], what)
    # nothing before the first record or behind the last, nor in their rows that there are not, nor between
    used = torch.zeros(Hkv, rb, dtype=torch.bool, device="cuda")
    used[:, :n * 2 * D] = used[:, block * 2 * D:block * 2 * D + 8] = True
    assert (t[:at] == 255).all() and (t[at + Hkv * rb:] == 255).all()
    assert (t[at:at + Hkv * rb].view(Hkv, rb)[~used] == 255).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.1, 0.1])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_a_key_of_zeros_among_huge_ones(dt, scale, softcap):
    """A block whose scale times the query's leaves fp32: its key of zeros has the score 0 all the
    same, and all the weight where the others' scores lie far below."""
    B, Hq, Hkv, D, cap, block, at = 2, 4, 1, 128, 70, 32, 40
    k = rows(B, cap, Hkv, D, "f32", 1, "k").abs() + 0.5
    k = k * (2.0 ** 123 if scale < 0 else -2.0 ** 123)
    k[:, at] = 0.0
    v = rows(B, cap, Hkv, D, "f32", 1, "v")
    q = (W.normal((B, Hq * D), dtype="f32", device="cuda", seed=2, role="q").abs() + 0.5) * 2.0 ** 40
    k, v, q = (x.to(W.torch_dtype(dt)) for x in (k, v, q))
    c = Cache(B, cap, Hkv, D, block)
    c.append(k, v, [0] * B, cap, dt=dt)
    lens = [cap, at + 1]
    out, lse, st = decode(c, q, i32(lens), dt, Hq, softcap=softcap, scale=scale)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode(out, lse, q, held(k, block), held(v, block), lens, dt, Hq, D, 0, softcap, "zeros", scale=scale)
