"""The 4-bit cache's oracle against hand-worked groups and its own bounds (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import q4


def group(*head):
    x = np.zeros(32, dtype=np.float32)
    x[:len(head)] = head
    return x


@pytest.mark.parametrize("x,want", [
    (group(), group()),                                       # nothing there
    (group(15.0, 7.4, 7.5, 8.5), group(15.0, 7.0, 8.0, 8.0)),  # s = 1, z = 0; ties to even
    (group(-15.0, -0.5, -1.5), group(-15.0, 0.0, -2.0)),       # s = 1, z = 15
    (group(10.0, -5.0, 3.4, -0.6), group(10.0, -5.0, 3.0, -1.0)),  # s = 1, z = 5
    (group(30.0, 1.0, 3.0), group(30.0, 0.0, 4.0)),            # s = 2: 0.5 -> 0, 1.5 -> 2
])
def test_hand_worked_groups(x, want):
    assert np.array_equal(q4.readback(x), want)


def test_bf16_is_torchs():
    x = torch.randn(4096, generator=torch.Generator().manual_seed(0)) * 3
    assert np.array_equal(q4.bf16(x.numpy()), x.bfloat16().float().numpy())


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_group_without_a_grid_reads_nan_and_no_other(bad):
    x = np.full(64, 15.0, dtype=np.float32)  # a step of 1: 15 reads back as it is
    x[40] = bad
    got = q4.readback(x)
    assert np.isnan(got[32:]).all() and (got[:32] == 15.0).all()


def test_error_is_within_the_step():
    """Half a step inside the grid.  s is off by 2^-9 and z by half a step, so an end of the
    range may lie up to 15 * 2^-9 + 1/2 < 0.53 steps beyond the grid's last place, whose own
    nearest neighbour is at most half a step further: below 1.03 steps in all."""
    x = (np.random.default_rng(1).standard_normal((500, 80)) * 2).astype(np.float32)
    got = q4.readback(x)
    for lo in range(0, 80, 32):
        g = x[:, lo:lo + 32]
        step = (np.maximum(g.max(-1), 0) - np.minimum(g.min(-1), 0)) / 15 * (1 + 2.0 ** -9)
        assert (np.abs(got[:, lo:lo + 32] - g) <= 1.03 * step[:, None]).all()
        assert np.median(np.abs(got[:, lo:lo + 32] - g) / step[:, None]) < 0.3
