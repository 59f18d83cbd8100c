"""Refusals of the chosen-block calls, on the host and before any launch (no GPU)."""
import pytest
import torch

from gqa_attention_lat_gb300 import binding
from gqa_attention_lat_gb300.build import build_library

# These addresses are never device memory: run only where no launch could reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer host checks run only without a GPU")
FAKE = 0x10000
INVALID, UNSUPPORTED, WORKSPACE = (binding.LAT_ERR_INVALID_ARG, binding.LAT_ERR_UNSUPPORTED,
                                   binding.LAT_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    binding.library(build_library())


def refused(fn, args, kw, code):
    with pytest.raises(binding.LatError) as e:
        fn(**dict(args, **kw))
    assert e.value.status == code


BOUNDS = dict(dt=binding.LAT_BF16, k_cache=FAKE, cache_rs=1024, cache_head_stride=128, cache_seq_stride=1 << 20,
              capacity=1024, bounds=FAKE, bounds_rs=2048, bounds_head_stride=256, bounds_seq_stride=1 << 16,
              block_size=64, pos=FAKE, n_new=4, batch=2, n_kv_heads=8, head_dim=128)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), INVALID), (dict(batch=-1), INVALID), (dict(n_new=-1), INVALID), (dict(capacity=-1), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(block_size=0), INVALID), (dict(block_size=24), INVALID),
    (dict(block_size=1040), INVALID), (dict(block_size=-16), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(k_cache=None), INVALID), (dict(bounds=None), INVALID), (dict(pos=None), INVALID),
    (dict(k_cache=FAKE + 8), INVALID), (dict(bounds=FAKE + 2), INVALID), (dict(cache_rs=1028), INVALID),
    (dict(cache_head_stride=0), INVALID), (dict(bounds_rs=2044), INVALID), (dict(bounds_seq_stride=-8), INVALID),
    (dict(n_new=1 << 30, batch=65535, block_size=16), UNSUPPORTED),
])
def test_bounds_refuse(kw, code):
    refused(binding.lat_kv_block_bounds, BOUNDS, kw, code)


def test_bounds_of_nothing_are_a_no_op():
    binding.lat_kv_block_bounds(**dict(BOUNDS, batch=0, k_cache=None))
    binding.lat_kv_block_bounds(**dict(BOUNDS, n_new=0, k_cache=None))


SELECT = dict(dt=binding.LAT_BF16, q=FAKE, q_rs=4096, bounds=FAKE, bounds_rs=2048, bounds_head_stride=256,
              bounds_seq_stride=1 << 16, block_size=64, kv_lens=FAKE, max_kv_len=4096, blocks=FAKE, n_sel=8,
              n_first=1, n_last=2, batch=2, n_heads=32, n_kv_heads=8, head_dim=128, workspace=FAKE,
              workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), INVALID), (dict(batch=-1), INVALID), (dict(max_kv_len=-1), INVALID), (dict(n_heads=30), INVALID),
    (dict(block_size=8), INVALID), (dict(n_sel=0), INVALID), (dict(n_first=-1), INVALID), (dict(n_last=-1), INVALID),
    (dict(n_first=5, n_last=4), INVALID), (dict(n_first=2 ** 31 - 1, n_last=2 ** 31 - 1), INVALID),
    (dict(head_dim=72), UNSUPPORTED), (dict(q=None), INVALID), (dict(bounds=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(blocks=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(q_rs=4095), INVALID), (dict(q_rs=2048), INVALID), (dict(bounds_rs=0), INVALID),
    (dict(bounds_head_stride=260), INVALID), (dict(max_kv_len=(1 << 20) + 1, block_size=16), UNSUPPORTED),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=FAKE + 16), WORKSPACE),
])
def test_select_refuses(kw, code):
    refused(binding.lat_attn_select_blocks, SELECT, kw, code)


def test_select_workspace_size():
    size = binding.lat_attn_select_blocks_workspace_size
    assert size(2, 8, 64, 4096) == 2 * 8 * 64 * 16
    for bad in [(-1, 8, 64, 4096), (2, 0, 64, 4096), (2, 8, 40, 4096), (2, 8, 64, -1), (2, 8, 16, (1 << 20) + 1)]:
        assert size(*bad) == 0


DECODE = dict(dt=binding.LAT_BF16, q=FAKE, q_rs=4096, k_cache=FAKE, v_cache=FAKE, cache_rs=1024,
              cache_head_stride=128, cache_seq_stride=1 << 22, kv_lens=FAKE, max_kv_len=4096, block_size=64,
              blocks=FAKE, n_sel=8, out=FAKE, out_rs=4096, lse=None, batch=2, n_heads=32, n_kv_heads=8,
              head_dim=128, scale=0.088, softcap=0.0, workspace=FAKE, workspace_bytes=1 << 40)


@pytest.mark.parametrize("dt", [binding.LAT_BF16, binding.LAT_F32])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(max_kv_len=-1), INVALID), (dict(n_heads=30), INVALID),
    (dict(block_size=0), INVALID), (dict(block_size=2048), INVALID), (dict(n_sel=0), INVALID),
    (dict(n_sel=65537), UNSUPPORTED), (dict(head_dim=72), UNSUPPORTED), (dict(blocks=None), INVALID),
    (dict(q=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(out=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(softcap=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 4), INVALID), (dict(v_cache=FAKE + 8), INVALID),
    (dict(q_rs=4000), INVALID), (dict(out_rs=4098), INVALID), (dict(cache_rs=1026), INVALID),
    (dict(cache_seq_stride=0), INVALID), (dict(batch=65536), UNSUPPORTED),
])
def test_decode_refuses(dt, kw, code):
    refused(binding.lat_attn_decode_blocks, DECODE, dict(kw, dt=dt), code)


def test_decode_of_nothing_is_a_no_op():
    for dt in (binding.LAT_BF16, binding.LAT_F32):
        binding.lat_attn_decode_blocks(**dict(DECODE, dt=dt, batch=0, q=None, blocks=None))
    refused(binding.lat_attn_decode_blocks, DECODE, dict(dt=5), INVALID)


def test_an_fp32_decode_of_too_many_heads_is_refused():
    refused(binding.lat_attn_decode_blocks, DECODE,
            dict(dt=binding.LAT_F32, batch=65535, n_heads=32768, q_rs=1 << 24, out_rs=1 << 24, head_dim=512), UNSUPPORTED)
