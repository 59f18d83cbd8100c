"""Query rows of 2^31 elements and more are refused by the decodes over reduced caches (no GPU)."""
import pytest
import torch

from gqa_attention_lat_gb300 import binding
from gqa_attention_lat_gb300.build import build_library
from test_abi_blocks import DECODE, SELECT
from test_abi_q4 import DECODE as Q4

# These addresses are never device memory: run only where no launch could reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer host checks run only without a GPU")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    binding.library(build_library())


@pytest.mark.parametrize("head_dim,n_heads", [(512, 1 << 22), (64, 1 << 25), (128, 5 << 22)])
@pytest.mark.parametrize("call", ["q4", "select", "blocks", "blocks_f32"])
def test_a_query_row_past_32_bits(call, head_dim, n_heads):
    fn, args = {"q4": (binding.lat_attn_decode_q4, Q4), "select": (binding.lat_attn_select_blocks, SELECT),
                "blocks": (binding.lat_attn_decode_blocks, DECODE),
                "blocks_f32": (binding.lat_attn_decode_blocks, dict(DECODE, dt=binding.LAT_F32))}[call]
    wide = dict(args, batch=1, n_heads=n_heads, n_kv_heads=1, head_dim=head_dim, q_rs=1 << 33,
                **({} if call == "select" else {"out_rs": 1 << 33}))
    with pytest.raises(binding.LatError) as e:
        fn(**wide)
    assert e.value.status == binding.LAT_ERR_UNSUPPORTED
    if call == "q4":
        assert binding.lat_attn_decode_q4_workspace_size(args["dt"], 1, n_heads, 1, head_dim, 64) == 0
    if call.startswith("blocks"):
        assert binding.lat_attn_decode_blocks_workspace_size(wide["dt"], 1, n_heads, 1, head_dim, 64, 8) == 0
