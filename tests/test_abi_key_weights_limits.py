"""The longest sequences that the key weights take, refused on the host beyond (no GPU)."""
import pytest
import torch

from gqa_attention_lat_gb300 import binding
from gqa_attention_lat_gb300.build import build_library
from test_abi_evict import WEIGH, refused

# These addresses are never device memory: run only where no launch could reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer host checks run only without a GPU")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    binding.library(build_library())


LONG = dict(batch=1, n_heads=2, n_kv_heads=1, head_dim=64, n_q=1, weights_head_stride=1 << 31, weights_seq_stride=1 << 31,
            cache_seq_stride=1 << 41)


@pytest.mark.parametrize("dt", [binding.LAT_BF16, binding.LAT_F32])
@pytest.mark.parametrize("n", [2 ** 31 - 127, 2 ** 31 - 1])
def test_keys_whose_tile_has_no_end_are_refused(dt, n):
    """A key tile that ends at 2^31 or behind it has keys without an int."""
    refused(binding.lat_attn_key_weights, WEIGH, dict(LONG, dt=dt, max_kv_len=n), binding.LAT_ERR_UNSUPPORTED)


@pytest.mark.parametrize("dt", [binding.LAT_BF16, binding.LAT_F32])
def test_the_last_ones_before_are_not(dt):
    """(There is no device to run them on: another error, behind all refusals.)"""
    refused(binding.lat_attn_key_weights, WEIGH, dict(LONG, dt=dt, max_kv_len=2 ** 31 - 128), binding.LAT_ERR_CUDA)
