"""Bounds on the paged attention's results that follow each form's own roundings."""
from __future__ import annotations

import numpy as np

from oracle import paged_oracle as P

U = 2.0 ** -24  # half an fp32 step


def bound(out, mag, lin, n_keys, weight_steps, out_step, lost=0.0, terms=1):
    """Element by element, for results whose operands are exact: a score is off by (terms d + 4) half
    steps of `lin` (a dot product of that many exact products in fp32, its scale, and the difference from the
    row's reference) and its weight by 2^-22 more (exp2), above and below the fraction line; weights are
    rounded to `weight_steps` (relative half steps) for the products, sums have n_keys terms, and the result
    is rounded to `out_step`.  lost: the largest |v| times what a weight may lose absolutely."""
    x = (terms * out.shape[-1] + 4) * U * lin + 2.0 ** -22
    moved = (np.exp(2 * x) - 1)[..., None] + (np.prod([1 + s for s in weight_steps]) - 1) + (n_keys + 16) * U
    return moved * mag * 1.01 + out_step * np.abs(out) + n_keys * lost + 1e-30


def piece_case(d, seed=12):
    """40 rows of 4 heads over one kv head's last of 60 tokens, 12 of them in the window and 2 in front: few keys,
    large queries, key scales of full mantissas, so that a score's error shows.  Codes and scales by token (the
    second of each pair the values'), float64 keys and values, queries in bf16."""
    rng = np.random.default_rng(seed)
    n, rows = 60, 40
    codes = rng.integers(-7, 8, (2, n, 1, d))
    sc = np.ldexp(1 + rng.integers(0, 128, (2, n, 1, d // 32)) / 128, rng.integers(-4, -1, (2, n, 1, d // 32)))
    val = codes.astype(np.float64) * np.repeat(sc, 32, -1)
    q = P.bf16(24 * rng.normal(size=(rows, 4, d)).astype(np.float32)).astype(np.float64)
    return n, rows, codes, sc, val[0], val[1], q


def piece_bound(want, mag, lin, v):
    """Weights in fp16 (2^-30 of the row's largest may be lost whole), keys exact in two parts, values exact."""
    return bound(want, mag, lin, 14, [2.0 ** -11], 2.0 ** -8, lost=2.0 ** -30 * np.abs(v).max(), terms=2)


def few_case(d, rows, seed=15):
    """Few rows of 4 heads over one kv head, values whose weighted sums cancel: what weights lose shows.  bf16."""
    rng = np.random.default_rng(seed)
    n = 60
    q, k, v = (P.bf16(rng.normal(size=(m, w, d)).astype(np.float32)).astype(np.float64) for m, w in ((rows, 4), (n, 1), (n, 1)))
    return n, q, k, v


def few_bound(want, mag, lin, n):
    """Weights in two bf16 parts: each rounding leaves 2^-8 at most, the second one of the first's rest."""
    return bound(want, mag, lin, n, [2.0 ** -16], 2.0 ** -8)
