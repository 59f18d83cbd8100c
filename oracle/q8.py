"""fp64 oracle of the 8-bit KV cache: what appended rows read back as.

By the definition: a block of `block` rows of one KV head has one exponent e for K and one for V,
the least in -100 .. 119 with which the largest finite magnitude of the rows appended to it is at
most 448 * 2^e; a value reads back as the e4m3 number nearest to x / 2^e (ties to even, held in
+-448; NaN for what is not finite) times 2^e.  Rows that go on in a block may raise its e; the values
before them are then rounded to the new one.
"""
from __future__ import annotations

import numpy as np

MIN_EXP, MAX_EXP = -100, 119


def exponent(amax):
    """The least e in range with amax <= 448 * 2^e (amax >= 0, finite)."""
    e = MIN_EXP
    while e < MAX_EXP and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def e4m3(x):
    """The e4m3 number nearest to x, ties to even, held in +-448; NaN for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    y = np.where(ok, x, 0.0)
    _, k = np.frexp(y)  # |y| in [2^(k-1), 2^k)
    step = np.exp2(np.maximum(k - 1, -6) - 3.0)
    return np.where(ok, np.clip(np.rint(y / step) * step, -448.0, 448.0), np.nan)


class Rows:
    """One sequence's cache rows of one tensor: values [cap, heads, D] as they read back."""

    def __init__(self, cap, heads, D, block):
        self.block = block
        self.value = np.full((cap, heads, D), np.nan)
        self.exp = np.zeros((-(-cap // block), heads), dtype=int)

    def append(self, x, pos):
        x = np.asarray(x, dtype=np.float64)
        for n in range(pos // self.block, -(-(pos + len(x)) // self.block)):
            first = n * self.block
            lo, hi = max(pos, first), min(pos + len(x), first + self.block)
            new = x[lo - pos:hi - pos]
            for h in range(x.shape[1]):
                mag = np.abs(new[:, h])
                e = exponent(mag[np.isfinite(mag)].max(initial=0.0))
                if lo > first:
                    e = max(e, self.exp[n, h])
                    old = self.value[first:lo, h]
                    self.value[first:lo, h] = e4m3(old / 2.0 ** e) * 2.0 ** e
                self.value[lo:hi, h] = e4m3(new[:, h] / 2.0 ** e) * 2.0 ** e
                self.exp[n, h] = e


def readback(x, block):
    """x [rows, heads, D] appended in one call from row 0 on."""
    r = Rows(len(x), x.shape[1], x.shape[2], block)
    r.append(x, 0)
    return r.value
