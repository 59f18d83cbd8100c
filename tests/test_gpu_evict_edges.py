"""Eviction's calls at the ends of their arguments' ranges."""
import pytest
import torch

from gpu_helpers import ensure_library
from gqa_attention_lat_gb300 import binding
from test_gpu_evict import caches, choose, move, weights

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


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f32", 512)])
def test_rows_by_a_list_as_long_as_an_int_can_say(dt, D):
    """Some rows, and -1 to the end of 2^31 - 1 entries: in a fraction of the time that a wait has.  An entry
    behind the cache's capacity is reported."""
    cap, n = 5000, 4321
    k, v = caches(1, cap, 1, D, dt, 6)
    was = [k.clone(), v.clone()]
    at = torch.randperm(cap, generator=torch.Generator().manual_seed(1))[:n].sort().values.cuda()
    kept = torch.full((1, 1, 2 ** 31 - 1), -1, dtype=torch.int32, device="cuda")
    kept[0, 0, :n] = at.int()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    st = move(k, v, kept, dt, D)
    end.record()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, y in zip((k, v), was):
        assert torch.equal(x[:, :n], y[:, at]) and torch.equal(x[:, n:], y[:, n:])
    assert begin.elapsed_time(end) < 1000
    kept[0, 0, :n] = torch.arange(n, dtype=torch.int32, device="cuda")
    for i in (cap, 2 ** 31 - 2):
        kept[0, 0, i] = cap - 1
        st = move(x, y, kept, dt, D)
        torch.cuda.synchronize()
        assert int(st.item()) == binding.LAT_ERR_BOUNDS
        kept[0, 0, i] = -1


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 80), ("f32", 512)])
@pytest.mark.parametrize("B", [1, 60])
def test_lists_that_end_where_a_stretch_does(dt, D, B):
    """Lists of every power of two and of its neighbours, in far longer room; by a cluster and by one CTA."""
    cap, n_keep, H = 2500, 20000, 2
    k, v = caches(B, cap, H, D, dt, 7)
    sizes = [0, 1, 2] + [(1 << e) + d for e in range(4, 12) for d in (-1, 0, 1)]
    for first in range(0, len(sizes), B * H):
        x, y = k.clone(), v.clone()
        kept = torch.full((B, H, n_keep), -1, dtype=torch.int32)
        g = torch.Generator().manual_seed(first)
        for u, n in enumerate(sizes[first:first + B * H]):
            kept[u // H, u % H, :n] = torch.randperm(cap, generator=g)[:n].sort().values.int()
        st = move(x, y, kept.cuda(), dt, D)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        for u, n in enumerate(sizes[first:first + B * H]):
            b, h = divmod(u, H)
            at = kept[b, h, :n].long().cuda()
            for new, old in ((x, k), (y, v)):
                assert torch.equal(new[b, :n, h], old[b, at, h]) and torch.equal(new[b, n:, h], old[b, n:, h])
