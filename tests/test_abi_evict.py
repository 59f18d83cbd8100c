"""Refusals of the key weights' and eviction's calls, on the host and before any launch (no GPU)."""
import pytest
import torch

from gqa_attention_lat_gb300 import binding
from gqa_attention_lat_gb300.build import build_library

# These addresses are never device memory: run only where no launch could reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer host checks run only without a GPU")
FAKE = 0x10000
INVALID, UNSUPPORTED = binding.LAT_ERR_INVALID_ARG, binding.LAT_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    binding.library(build_library())


def refused(fn, args, kw, code):
    args = dict(args, **kw)
    with pytest.raises(binding.LatError) as e:
        fn(**args)
    assert e.value.status == code


WEIGH = dict(dt=binding.LAT_BF16, q=FAKE, q_rs=4096, n_q=4, k_cache=FAKE, cache_rs=1024, cache_head_stride=128,
             cache_seq_stride=4096 * 1024, kv_lens=FAKE, max_kv_len=4096, lse=FAKE, weights=FAKE,
             weights_head_stride=4096, weights_seq_stride=8 * 4096, batch=32, n_heads=32, n_kv_heads=8, head_dim=128,
             causal=1, window=0, scale=0.088, softcap=0.0)
F32 = binding.LAT_F32


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), INVALID), (dict(n_heads=30), INVALID), (dict(n_kv_heads=0), INVALID), (dict(batch=-1), INVALID),
    (dict(n_q=-1), INVALID), (dict(max_kv_len=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("inf")), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k_cache=None), INVALID), (dict(kv_lens=None), INVALID), (dict(lse=None), INVALID),
    (dict(weights=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(k_cache=FAKE + 8), INVALID),
    (dict(q_rs=4095), INVALID), (dict(q_rs=4100), INVALID), (dict(cache_rs=1028), INVALID),
    (dict(cache_head_stride=0), INVALID), (dict(cache_seq_stride=-8), INVALID),
    (dict(weights_head_stride=4095), INVALID), (dict(weights_seq_stride=4095), INVALID),
    (dict(batch=65536), UNSUPPORTED), (dict(n_q=1 << 27), UNSUPPORTED),
    (dict(n_heads=1 << 25, n_kv_heads=8, q_rs=1 << 32), UNSUPPORTED),
    (dict(dt=F32, batch=16384), UNSUPPORTED), (dict(dt=F32, q_rs=4095), INVALID),
    (dict(batch=60000, max_kv_len=1 << 24, weights_head_stride=1 << 24, weights_seq_stride=1 << 30, n_q=1), UNSUPPORTED),
])
def test_key_weights_refuse(kw, code):
    refused(binding.lat_attn_key_weights, WEIGH, kw, code)


def test_key_weights_of_nothing_are_no_ops():
    binding.lat_attn_key_weights(**dict(WEIGH, batch=0, q=None))
    binding.lat_attn_key_weights(**dict(WEIGH, n_q=0, lse=None))


CHOOSE = dict(weights=FAKE, weights_head_stride=4096, weights_seq_stride=8 * 4096, kv_lens=FAKE, max_kv_len=4096,
              kept=FAKE, n_keep=512, n_first=4, n_last=64, weights_out=FAKE, out_head_stride=4096,
              out_seq_stride=8 * 4096, new_lens=FAKE + 4096, batch=4, n_kv_heads=8)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(max_kv_len=-1), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_keep=0), INVALID),
    (dict(n_first=-1), INVALID), (dict(n_last=-1), INVALID), (dict(n_first=449), INVALID),
    (dict(n_first=(1 << 31) - 1, n_last=(1 << 31) - 1), INVALID), (dict(weights=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(kept=None), INVALID), (dict(new_lens=None), INVALID),
    (dict(new_lens=FAKE), INVALID), (dict(weights_head_stride=4095), INVALID), (dict(weights_seq_stride=4095), INVALID),
    (dict(out_head_stride=4095), INVALID), (dict(out_head_stride=5000, out_seq_stride=40000), INVALID),
    (dict(weights_out=FAKE + 64, out_seq_stride=4095), INVALID),
    (dict(max_kv_len=425985, weights_head_stride=1 << 20, weights_seq_stride=1 << 23, weights_out=None), UNSUPPORTED),
    (dict(batch=1 << 20, n_kv_heads=1 << 10), UNSUPPORTED),
])
def test_choose_refuses(kw, code):
    refused(binding.lat_kv_evict_choose, CHOOSE, kw, code)


ROWS = dict(dt=binding.LAT_BF16, k_cache=FAKE, v_cache=FAKE + (1 << 20), cache_rs=1024, cache_head_stride=128,
            cache_seq_stride=4096 * 1024, capacity=4096, kept=FAKE, n_keep=512, batch=4, n_kv_heads=8, head_dim=128)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), INVALID), (dict(batch=-1), INVALID), (dict(capacity=-1), INVALID), (dict(n_keep=0), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(k_cache=None), INVALID),
    (dict(v_cache=None), INVALID), (dict(kept=None), INVALID), (dict(k_cache=FAKE + 8), INVALID),
    (dict(v_cache=FAKE + 8), INVALID), (dict(cache_rs=1028), INVALID), (dict(cache_head_stride=0), INVALID),
    (dict(cache_seq_stride=-1024), INVALID), (dict(cache_rs=1 << 62), INVALID), (dict(dt=F32, cache_rs=1026), INVALID),
    (dict(batch=1 << 20, n_kv_heads=1 << 10), UNSUPPORTED),
])
def test_rows_refuse(kw, code):
    refused(binding.lat_kv_evict_rows, ROWS, kw, code)


def test_eviction_from_nothing_is_a_no_op():
    binding.lat_kv_evict_choose(**dict(CHOOSE, batch=0, weights=None))
    binding.lat_kv_evict_rows(**dict(ROWS, batch=0, k_cache=None))
