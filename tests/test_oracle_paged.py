"""Pins of the paged-cache oracle: layout of the 4-bit rows byte by byte, rounding cases, the
window's closed forms, and the library's pure-host refusals.  No GPU is needed."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from rag_kv_cache_rope_gb300 import binding as b
from rag_kv_cache_rope_gb300 import build as B


def test_packed_rows_byte_by_byte():
    d = 128
    codes = np.arange(d) % 15 - 7
    k, v = P.pack(codes[None], False)[0], P.pack(codes[None], True)[0]
    u = codes + 8
    # word (c, g) of a K row: dims 32g + 8c + (0 2 4 6 1 3 5 7) from the lowest nibble up
    for g in range(4):
        for c in range(4):
            w = int.from_bytes(k[c * 16 + 4 * g:c * 16 + 4 * g + 4].tobytes(), "little")
            assert [(w >> (4 * i)) & 15 for i in range(8)] == [u[32 * g + 8 * c + e] for e in (0, 2, 4, 6, 1, 3, 5, 7)]
        for r in range(8):
            w = int.from_bytes(v[r * 8 + 2 * g:r * 8 + 2 * g + 2].tobytes(), "little")
            assert [(w >> (4 * i)) & 15 for i in range(4)] == [u[32 * g + 4 * r + e] for e in range(4)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value_row", [False, True])
def test_every_dim_has_its_own_place(d, value_row):
    assert len({P.dim_place(d, i, value_row) for i in range(d)}) == d
    rng = np.random.default_rng(d)
    codes = rng.integers(-8, 8, (3, d))
    ones = np.ones((3, d // 32))
    assert (P.unpack(P.pack(codes, value_row), ones, value_row) == codes).all()


def test_quantise_hand_cases():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :4] = [7.0, -7.0, 0.5, 1.5]     # scale 1: halves go to the even code
    x[0, 40] = np.inf
    n, s = P.quantise(x)
    assert s[0, 0] == 1.0 and n[0, :4].tolist() == [7, -7, 0, 2] and n[0, 4:32].any() == 0
    assert np.isnan(s[0, 1]) and not n[0, 32:].any()
    n, s = P.quantise(np.zeros((2, 32), dtype=np.float32))
    assert not n.any() and not s.any()
    # a scale that rounds down leaves max / scale above 7: still code 7
    y = np.full((1, 32), 7 * (1 + 2.0 ** -9), dtype=np.float32)
    n, s = P.quantise(y)
    assert s[0, 0] == 1.0 and (n == 7).all()
    # the scale is the fp32 product with fp32's 1/7: just below a tie of bf16 it is the tie, where a
    # division would stay below it
    y = np.full((1, 32), np.nextafter(np.float32(7 * (1 + 3 * 2.0 ** -8)), np.float32(0)), dtype=np.float32)
    assert P.quantise(y)[1][0, 0] == 1 + 2.0 ** -6


def test_rotation_forms_agree():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 128))
    for pos in (-70000, -1, 0, 1, 131071):
        a, f = P.rotate(x, pos, 1e6), P.rotate_f32(x, pos, 1e6)
        # |x| < 5: inputs, cos/sin, two products and a sum, each off by at most 2^-24 relative
        assert np.abs(a - f).max() <= 5 * 2 * 4 * 2.0 ** -24
    assert np.allclose(P.rotate(P.rotate(x, 5, 1e4), 7, 1e4), P.rotate(x, 12, 1e4), atol=1e-12)


def test_window_and_sinks():
    assert P.visible(5, 0, 0) == [0, 1, 2, 3, 4, 5]
    assert P.visible(5, 2, 0) == [4, 5] and P.visible(5, 2, 1) == [0, 4, 5]
    assert P.visible(5, 1, 9) == [0, 1, 2, 3, 4, 5] and P.visible(0, 1, 0) == [0] and P.visible(-1, 4, 2) == []
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(2, 2, 32)), rng.normal(size=(6, 1, 32)), rng.normal(size=(6, 1, 32))
    full, _, _ = P.attention(q, k, v, 6, 0, 0)
    assert np.allclose(P.attention(q, k, v, 6, 6, 0)[0], full)           # a window of every token
    one, _, _ = P.attention(q, k, v, 6, 1, 0)
    assert np.allclose(one[1], v[5]) and np.allclose(one[0], v[4])       # a window of one: the row's own value
    empty, _, _ = P.attention(q, k[:1], v[:1], 1, 0, 0)
    assert not empty[0].any() and np.allclose(empty[1], v[0])            # a row before the first token


def test_pages_are_checked_without_a_gpu():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    ok = b.PagesRef(k, k.clone(), t)
    assert (ok.c.format, ok.c.page_tokens, ok.c.n_pages, ok.c.n_seq, ok.c.max_pages) == (b.PAGES_MODEL, 16, 4, 1, 4)
    k4, s4 = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), torch.zeros(4, 2, 16, 2, dtype=torch.bfloat16)
    ok = b.PagesRef(k4, k4.clone(), t, s4, s4.clone())
    assert ok.c.format == b.PAGES_INT4 and ok.head_dim == 64
    for bad in (lambda: b.PagesRef(k, k[:3], t), lambda: b.PagesRef(k, k.float(), t),
                lambda: b.PagesRef(k, k, t.long()), lambda: b.PagesRef(k, k, t[0]),
                lambda: b.PagesRef(k.transpose(0, 1), k.transpose(0, 1), t), lambda: b.PagesRef(k, k, t, s4, s4),
                lambda: b.PagesRef(k4, k4, t), lambda: b.PagesRef(k4, k4, t, s4, s4.float()),
                lambda: b.PagesRef(k4, k4, t, s4[:2], s4), lambda: b.PagesRef(k[0], k[0], t)):
        with pytest.raises(ValueError):
            bad()


def test_calls_without_a_handle_are_refused():
    B.build()
    lib, vp = b.lib(), C.c_void_p(1 << 20)
    pg = b.Pages(b.PAGES_MODEL, 16, 4, 1, 4, 1 << 20, 1 << 20, 1 << 20, None, None)
    assert lib.paged_append(None, C.byref(pg), vp, 128, vp, 128, None, 0, None, vp, vp, None, vp, 1, None) == b.EINVAL
    assert lib.paged_gather(None, C.byref(pg), vp, vp, None, vp, 1, vp, vp, None) == b.EINVAL
    assert lib.paged_attention(None, C.byref(pg), vp, 256, vp, vp, 1, 1, 0, 0, vp, None) == b.EINVAL
    assert b"handle" in lib.blend_last_error(None)


PROBE = r"""
#include <stddef.h>
#include <stdio.h>
#include "blend.h"
#define P(f) printf(#f " %zu\n", offsetof(blend_pages, f));
int main(void) {
  printf("size %zu\n", sizeof(blend_pages));
  P(format) P(page_tokens) P(n_pages) P(n_seq) P(max_pages) P(table) P(k) P(v) P(k_scale) P(v_scale)
  return 0;
}
"""


def test_pages_struct_layout_matches_c(tmp_path):
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(PROBE)
    subprocess.run(["gcc", "-I", os.path.join(B.ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True).stdout
    got = {k: int(v) for k, v in (line.split() for line in out.splitlines())}
    assert got.pop("size") == C.sizeof(b.Pages)
    assert set(got) == {f for f, _ in b.Pages._fields_}
    for f, off in got.items():
        assert getattr(b.Pages, f).offset == off, f
