"""The bounds of the tight paged-attention tests tell a kernel that loses bits from one that does not: mistakes are
planted in the float64 values.  No GPU is needed."""
import numpy as np
import pytest

from oracle import paged_oracle as P
from pagedtight import few_bound, few_case, piece_bound, piece_case


def worst(got, want, lim):
    return (np.abs(got - want) / lim).max()


@pytest.mark.parametrize("d", [64, 128])
def test_bound_of_pieces_shows_what_keys_lose(d):
    n, rows, _, _, k, v, q = piece_case(d)
    want, mag, lin = P.attention(q, k, v, n, 12, 2)
    lim = piece_bound(want, mag, lin, v)

    def out(keys):
        return P.attention(q, keys, v, n, 12, 2)[0]

    high = P.bf16(k.astype(np.float32)).astype(np.float64)
    rest = k - high
    assert (P.bf16(rest.astype(np.float32)) == rest).all()  # the second part is exact
    assert worst(P.bf16(want.astype(np.float32)), want, lim) < 1
    for wrong in (high,                                               # without the second part
                  high + np.roll(rest, 8, -1),                        # in the next chunk of 16 bytes
                  high + np.roll(rest, 1, 0),                         # of the token before
                  high + np.where(np.arange(d) < d // 2, rest, 0)):   # half of the products left out
        assert worst(out(wrong), want, lim) > 2


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 4])
def test_bound_of_few_rows_shows_what_weights_lose(d, rows):
    n, q, k, v = few_case(d, rows)
    want, mag, lin = P.attention(q, k, v, n, 0, 0)
    lim = few_bound(want, mag, lin, n)

    def out(parts):
        got = np.zeros_like(want)
        for i in range(rows):
            for h in range(4):
                s = k[:n - rows + i + 1, 0] @ q[i, h] / np.sqrt(d)
                w = np.exp(s - s.max()).astype(np.float32)
                high = P.bf16(w)
                got[i, h] = (high.astype(np.float64) + (P.bf16(w - high) if parts == 2 else 0)) @ v[:len(s), 0] / w.astype(np.float64).sum()
        return got

    assert worst(out(2), want, lim) < 1 and worst(out(1), want, lim) > 2
