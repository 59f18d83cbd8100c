"""Oracle of the chosen-block decode: block bounds, exact block scores, the choice.

By the definitions: a block's bounds are the channels' largest and smallest keys in it; a
block's score for a KV head is the largest over its query heads of sum_d max(q_d hi_d, q_d lo_d),
here as the correctly rounded sum (math.fsum) of products that fp64 holds exactly (bf16 or fp32
factors); the choice is the first n_first, the last n_last and the best scored others, ties to
the lowest, ascending, -1 behind.
"""
from __future__ import annotations

import math

import numpy as np


def bounds(k, block):
    """k [n, D] -> (hi, lo) [ceil(n / block), D]; a NaN makes both NaN."""
    k = np.asarray(k)
    parts = [k[lo:lo + block] for lo in range(0, k.shape[0], block)]
    return np.stack([p.max(0) for p in parts]), np.stack([p.min(0) for p in parts])


def scores(q, hi, lo):
    """q [G, D], hi and lo [n, D] -> [n]."""
    q, hi, lo = (np.asarray(x, dtype=np.float64) for x in (q, hi, lo))
    out = []
    for h, l in zip(hi, lo):
        terms = np.maximum(q * h, q * l)
        out.append(max(math.fsum(t) for t in terms))
    return np.array(out)


def choose(score, n_sel, n_first, n_last):
    """score [n] of the blocks there are -> [n_sel]."""
    n = len(score)
    if n <= n_sel:
        kept = list(range(n))
    else:
        forced = list(range(n_first)) + list(range(n - n_last, n))
        free = sorted(range(n_first, n - n_last), key=lambda i: (-score[i], i))
        kept = sorted(forced + free[:n_sel - n_first - n_last])
    return np.array(kept + [-1] * (n_sel - len(kept)), dtype=np.int64)


def rows_of(blocks, block, length):
    """The cache rows that a list of blocks holds below `length`."""
    return [j for n in blocks if n >= 0 for j in range(n * block, min(length, (n + 1) * block))]
