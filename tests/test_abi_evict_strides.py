"""Eviction's rows: strides whose bytes no 64-bit number can say (no GPU)."""
import pytest
import torch

from gqa_attention_lat_gb300 import binding
from gqa_attention_lat_gb300.build import build_library
from test_abi_evict import F32, ROWS, refused

# These addresses are never device memory: run only where no launch could reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer host checks run only without a GPU")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    binding.library(build_library())


@pytest.mark.parametrize("which", ["cache_rs", "cache_head_stride", "cache_seq_stride"])
@pytest.mark.parametrize("dt,stride", [(F32, 8 - (1 << 62)), (F32, 8 - (1 << 63)), (binding.LAT_BF16, 16 - (1 << 63)),
                                       (F32, (1 << 62) + 8), (binding.LAT_BF16, 0)])
def test_strides_beyond_64_bits_of_bytes_are_refused(which, dt, stride):
    """Among them negative ones whose bytes would come out positive."""
    refused(binding.lat_kv_evict_rows, ROWS, {which: stride, "dt": dt}, binding.LAT_ERR_INVALID_ARG)
