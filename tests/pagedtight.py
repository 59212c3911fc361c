"""Bounds on the paged attention's results that follow each form's own roundings."""
from __future__ import annotations

import numpy as np

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
