"""The choice of blocks at the ends of its arguments' ranges."""
import pytest
import torch

import workloads as W
from gpu_helpers import ensure_library
from test_gpu_blocks import select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


def test_a_list_as_long_as_an_int_can_say():
    """Every block there is, and -1 to the end of 2^31 - 1 entries."""
    D, nb, n_sel = 64, 5, 2 ** 31 - 1
    bd = W.normal((1, nb, 1, 2 * D), dtype="f32", device="cuda", seed=2, role="k")
    q = W.normal((1, D), dtype="f32", device="cuda", seed=2, role="q")
    got, st = select(q, bd, [nb * 16], 16, 1, 1, D, "f32", n_sel, 3, 4)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert got[0, 0, :nb].tolist() == list(range(nb))
    for part in got[0, 0, nb:].split(1 << 28):
        assert int((part != -1).sum()) == 0
