"""Eviction's calls at the ends of their arguments' ranges."""
import pytest
import torch

from gpu_helpers import ensure_library
from test_gpu_evict import choose, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


@pytest.mark.parametrize("n,cap", [(50, 50), (0, 50), (100_000, 425_984)])
def test_a_choice_as_long_as_an_int_can_say(n, cap):
    """Every key there is, and -1 to the end of 2^31 - 1 entries; by one CTA and by eight."""
    n_keep = 2 ** 31 - 1
    w = weights(1, 1, cap, 3)
    kept, o, new, st = choose(w, [n], n_keep, 3, 7)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and new.tolist() == [n]
    assert torch.equal(kept[0, 0, :n], torch.arange(n, dtype=torch.int32, device="cuda"))
    for part in kept[0, 0, n:].split(1 << 28):
        assert int((part != -1).sum()) == 0
    assert torch.equal(o[0, 0, :n], w[0, 0, :n]) and (o[0, 0, n:] == -7).all()
