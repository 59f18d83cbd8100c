"""Refusals of the 4-bit cache's calls, on the host and before any launch (no GPU)."""
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
    args = dict(args, **kw)
    with pytest.raises(binding.LatError) as e:
        fn(**args)
    assert e.value.status == code


def test_row_bytes():
    assert [binding.lat_kv_q4_row_bytes(d) for d in (64, 80, 128, 256, 512, 96, 0, -64)] == [
        80, 128, 160, 320, 640, 0, 0, 0]


STORE = dict(dt=binding.LAT_BF16, cache=FAKE, cache_rs=8 * 160, cache_head_stride=160,
             cache_seq_stride=64 * 8 * 160, capacity=64, pos=FAKE, batch=2, n_kv_heads=8, head_dim=128)
STORE_BAD = [
    (dict(dt=7), INVALID), (dict(batch=-1), INVALID), (dict(n=-1), INVALID), (dict(capacity=-1), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(cache=None), INVALID),
    (dict(x=None), INVALID), (dict(pos=None), INVALID), (dict(cache=FAKE + 8), INVALID),
    (dict(cache_rs=8 * 160 + 8), INVALID), (dict(cache_head_stride=0), INVALID), (dict(cache_seq_stride=-16), INVALID),
    (dict(rs=8 * 128 - 1), INVALID), (dict(batch=1 << 20, n=1 << 8, n_kv_heads=8), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", STORE_BAD)
@pytest.mark.parametrize("expand", [False, True])
def test_rows_in_and_out_refuse(kw, code, expand):
    kw = dict(dict(n=4, x=FAKE, rs=8 * 128), **kw)
    names = dict(n="n_rows", x="v_out", rs="out_rs") if expand else dict(n="n_new", x="v_new", rs="new_rs")
    kw = {names.get(k, k): v for k, v in kw.items()}
    base = dict(STORE, **({"k_out": FAKE} if expand else {"k_new": FAKE}))
    refused(binding.lat_kv_expand_q4 if expand else binding.lat_kv_append_q4, base, kw, code)


def test_rows_in_and_out_of_nothing_are_no_ops():
    for kw in (dict(batch=0, n_new=3), dict(n_new=0)):
        binding.lat_kv_append_q4(**dict(STORE, k_new=None, v_new=None, new_rs=0, **kw))
    binding.lat_kv_expand_q4(**dict(STORE, k_out=None, v_out=None, out_rs=0, n_rows=0))


DECODE = dict(dt=binding.LAT_BF16, q=FAKE, q_rs=4096, cache=FAKE, cache_rs=8 * 160, cache_head_stride=160,
              cache_seq_stride=4096 * 8 * 160, kv_lens=FAKE, max_kv_len=4096, out=FAKE, out_rs=4096, lse=None,
              batch=32, n_heads=32, n_kv_heads=8, head_dim=128, window=0, scale=0.088, softcap=0.0,
              workspace=FAKE, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), INVALID), (dict(n_heads=30), INVALID), (dict(n_kv_heads=0), INVALID), (dict(batch=-1), INVALID),
    (dict(max_kv_len=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(softcap=-1.0), INVALID),
    (dict(softcap=float("nan")), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(cache=None), INVALID), (dict(kv_lens=None), INVALID), (dict(out=None), INVALID),
    (dict(q=FAKE + 2), INVALID), (dict(out=FAKE + 8), INVALID), (dict(cache=FAKE + 4), INVALID),
    (dict(q_rs=4000), INVALID), (dict(out_rs=4100), INVALID), (dict(cache_rs=8 * 160 + 8), INVALID),
    (dict(cache_head_stride=-160), INVALID), (dict(dt=binding.LAT_F32, q_rs=4098), INVALID),
    (dict(batch=65536), UNSUPPORTED),
])
def test_decode_refuses(kw, code):
    refused(binding.lat_attn_decode_q4, DECODE, kw, code)


def test_decode_of_nothing_is_a_no_op():
    binding.lat_attn_decode_q4(**dict(DECODE, batch=0, q=None))


@pytest.mark.parametrize("args", [(2, 8, 16, 8, 64, 100), (1, 8, 15, 8, 64, 100), (1, 8, 16, 8, 96, 100),
                                  (1, -1, 16, 8, 64, 100), (1, 65536, 16, 8, 64, 100), (0, 8, 16, 8, 64, -1)])
def test_workspace_size_is_zero_for_what_is_refused(args):
    assert binding.lat_attn_decode_q4_workspace_size(*args) == 0
