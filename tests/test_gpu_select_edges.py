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


def by_definition(q, bd, D):
    """The definition's scores [n] of one KV head in fp64, a NaN in either product kept; NaN as +inf
    and a half, so that it goes first."""
    q, r = q.double().cpu().view(-1, 1, D), bd.double().cpu()
    terms = torch.maximum(q * r[:, :D], q * r[:, D:])  # [heads, n, D]
    s = terms.sum(-1)
    s = torch.where(torch.isnan(s), torch.full_like(s, float("inf")), s.clamp(max=1e300)).amax(0)
    return s.tolist()


def kept(scores, n_sel):
    order = sorted(range(len(scores)), key=lambda i: (-scores[i], i))
    return sorted(order[:n_sel])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4, 11])
@pytest.mark.parametrize("nb", [60, 1500])
def test_an_infinite_bound_of_a_channel_that_the_query_lacks(dt, G, nb):
    """0 times an infinity is no number, on whichever side the infinity is: such blocks go first;
    an infinity on the side that a nonzero channel does not take changes nothing."""
    D, block, n_sel = 128, 16, 9
    mid = W.normal((nb, D), dtype="f32", device="cuda", seed=3, role="k")
    half = W.normal((nb, D), dtype="f32", device="cuda", seed=4, role="k").abs()
    bd = torch.cat([mid + half, mid - half], 1)
    q = W.normal((1, G, D), dtype="f32", device="cuda", seed=5, role="q")
    q[:, :, 7] = 0.0
    q[:, :, 8] = -0.0
    q[:, :, 9] = q[:, :, 9].abs() + 0.5
    q[:, :, 10] = -q[:, :, 10].abs() - 0.5
    inf = float("inf")
    bd[41, 7] = inf             # hi, zero channel: NaN
    bd[33, D + 7] = -inf        # lo, zero channel: NaN
    bd[52, D + 8] = -inf        # lo, minus zero: NaN
    bd[17, D + 9] = -inf        # lo where q > 0: hi counts
    bd[18, 10] = inf            # hi where q < 0: lo counts
    bd[19, 9] = inf             # inf
    bd[20, D + 10] = -inf       # q < 0 times -inf: inf
    bd[21, 9] = bd[21, D + 9] = -inf  # -inf
    bd = bd.to(W.torch_dtype(dt)).view(1, nb, 1, 2 * D)
    q = q.to(W.torch_dtype(dt)).view(1, G * D)
    s = by_definition(q[0], bd[0, :, 0], D)
    assert [s[i] == inf for i in (41, 33, 52, 17, 18, 21)] == [True] * 3 + [False] * 3
    for n in (2, 3, 4, 5, n_sel):
        got, st = select(q, bd, [nb * block], block, G, 1, D, dt, n, 0, 0)
        assert int(st.item()) == 0
        assert got[0, 0].tolist() == kept(s, n), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nb", [300, 1500])
@pytest.mark.parametrize("q_exp,k_exp", [(-70, -70), (-72, -75), (-66, -64), (-60, -60)])
def test_scores_down_to_the_least_floats(dt, nb, q_exp, k_exp):
    """Products and sums among fp32's subnormal numbers, where a sum is off by parts of itself:
    the choice is that of the exact scores (products of fp32 numbers are exact in fp64, and sums
    of 64 of them are compared far above its rounding)."""
    D, block, G, n_sel = 64, 16, 3, 40
    mid = W.normal((nb, D), dtype="f32", device="cuda", seed=13, role="k")
    half = W.normal((nb, D), dtype="f32", device="cuda", seed=14, role="k").abs()
    bd = (torch.cat([mid + half, mid - half], 1) * 2.0 ** k_exp).to(W.torch_dtype(dt)).view(1, nb, 1, 2 * D)
    q = (W.normal((1, G * D), dtype="f32", device="cuda", seed=15, role="q") * 2.0 ** q_exp).to(W.torch_dtype(dt))
    s = by_definition(q[0], bd[0, :, 0], D)
    gaps = sorted(s)
    assert min(b - a for a, b in zip(gaps, gaps[1:])) > 2.0 ** (q_exp + k_exp - 40)
    got, st = select(q, bd, [nb * block], block, G, 1, D, dt, n_sel, 0, 0)
    assert int(st.item()) == 0
    assert got[0, 0].tolist() == kept(s, n_sel)
