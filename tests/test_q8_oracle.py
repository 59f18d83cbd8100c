"""The 8-bit cache's oracle against hand-worked blocks and its own bounds (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import q8


@pytest.mark.parametrize("x,want", [
    (0.0, 0.0), (448.0, 448.0), (447.0, 448.0), (17.0, 16.0), (18.0, 18.0), (19.0, 20.0),  # ties to even
    (2.0 ** -9, 2.0 ** -9), (2.0 ** -10, 0.0), (3 * 2.0 ** -10, 2.0 ** -8), (-1.0625, -1.0), (-1.1, -1.125),
    (500.0, 448.0), (np.inf, np.nan), (np.nan, np.nan),
])
def test_hand_worked_codes(x, want):
    assert np.array_equal(q8.e4m3(x), want, equal_nan=True)


def test_codes_are_torchs():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0)) * 2.0 ** torch.linspace(-12, 6, 20000)
    x = x.clamp(-448, 448)
    assert np.array_equal(q8.e4m3(x.numpy()), x.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("amax,e", [(0.0, -100), (448.0, 0), (448.1, 1), (1.0, -8), (1.75, -8), (1.7500001, -7),
                                    (3e38, 119), (1e-38, -100), (224.0, -1)])
def test_exponents(amax, e):
    assert q8.exponent(amax) == e


def test_a_block_grows():
    """1 and 2^-12 under e = -8 (steps of 2^-17 below 2^-14), then 448 under e = 0 (2^-9)."""
    r = q8.Rows(3, 1, 2, 16)
    r.append(np.array([[[1.0, 2.0 ** -12]]]), 0)
    assert r.exp[0, 0] == -8 and np.array_equal(r.value[0, 0], [1.0, 2.0 ** -12])
    r.append(np.array([[[448.0, 0.0]], [[np.inf, 3.0]]]), 1)
    assert r.exp[0, 0] == 0
    assert np.array_equal(r.value[:, 0], [[1.0, 0.0], [448.0, 0.0], [np.nan, 3.0]], equal_nan=True)


def test_error_is_within_half_a_step():
    """Half of 2^-3 of a value's own power of two, or half of 2^-9 * 2^e among the subnormals;
    amax / 448 > 2^(e - 1), so 2^(e - 10) < amax / 448 * 2^-9."""
    x = np.random.default_rng(1).standard_normal((64, 3, 80)) * np.exp2(np.arange(80) / 8.0)
    err = np.abs(q8.readback(x, 32) - x)
    amax = np.abs(x).reshape(2, 32, 3, 80).max((1, 3)).repeat(32, 0)[:, :, None]
    assert (err <= np.maximum(2.0 ** -4 * np.abs(x), amax / 448 * 2.0 ** -9)).all()
