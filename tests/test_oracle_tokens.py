"""Pins of the oracle of the token operators (4-bit weights, log probabilities, rotary positions), and the
parts of their binding that need no GPU."""
import ctypes as C
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import token_oracle as O
from rag_kv_cache_rope_gb300 import binding as b
from rag_kv_cache_rope_gb300 import build as B


def test_w4_codes_scales_and_ties():
    w = np.zeros((1, 64), dtype=np.float32)
    w[0, :8] = [7, -7, 3.5, 2.5, -0.5, 1.5, 0.49, -6.6]  # scale 1: ties go to the even integer
    codes, scales = O.w4_quantise(w, 32)
    assert scales.tolist() == [[1.0, 0.0]]
    assert codes[0, :8].tolist() == [15, 1, 12, 10, 8, 10, 8, 1] and (codes[0, 8:] == 8).all()
    w[0, 40] = np.inf
    codes, scales = O.w4_quantise(w, 32)
    assert math.isnan(scales[0, 1]) and (codes[0, 32:] == 8).all() and scales[0, 0] == 1.0


def test_w4_layout_of_the_binding_is_the_documented_one():
    rng = np.random.default_rng(0)
    for k in (8, 128, 136, 688):
        codes = rng.integers(0, 16, (3, k))
        assert np.array_equal(b.w4_layout(torch.from_numpy(codes)).numpy(), O.w4_rows(codes)), k
    places = {O.w4_place(i) for i in range(256)}
    assert len(places) == 256 and max(p[0] for p in places) == 127
    # word 4t + w of a chunk, input e at bit 4 (e / 2) + 16 (e % 2)
    assert O.w4_place(0) == (0, 0) and O.w4_place(1) == (2, 0) and O.w4_place(2) == (0, 4) and O.w4_place(7) == (3, 4)
    assert O.w4_place(8) == (16, 0) and O.w4_place(32) == (4, 0) and O.w4_place(128) == (64, 0)


def test_logprobs_rules():
    inf = np.inf
    x = np.array([[0.0, -0.0, -inf, 1.0], [-inf] * 4, [np.nan, 2.0, inf, 2.0], [5.0, 5.0, 5.0, 5.0]])
    logp, ent, top_id, top_logp = O.logprobs(x, 1.0, np.array([[3, -1], [0, -1], [1, -1], [2, 0]]), 4)
    z = 2 + math.e
    assert logp[0, 0] == pytest.approx(1 - math.log(z)) and logp[0, 1] == 0
    assert top_id[0].tolist() == [3, 0, 1, 2] and top_logp[0, 3] == -inf
    assert (logp[1, 0], ent[1]) == (-inf, 0) and top_id[1].tolist() == [0, 1, 2, 3]
    assert math.isnan(logp[2, 0]) and math.isnan(ent[2]) and top_id[2].tolist() == [2, 1, 3, 0]
    assert ent[3] == pytest.approx(math.log(4)) and top_id[3].tolist() == [0, 1, 2, 3]


def test_rope_frequencies():
    e = O.rope_freqs(1e4, 64)
    assert e[0] == 1 and e[16] == pytest.approx(1e-2)
    assert np.allclose(O.rope_freqs(1e4, 64, "linear", 4.0), e / 4)
    base = O.rope_freqs(1e4, 64, "base", 4.0)
    assert base[0] == 1 and base[31] == pytest.approx(e[31] / 4)  # the slowest pair ends at 1 / factor
    bands = O.rope_freqs(1e4, 64, "bands", 8.0, 1.0, 4.0, 8192)
    turns = 8192 * e / (2 * math.pi)
    assert np.array_equal(bands[turns > 4], e[turns > 4]) and np.allclose(bands[turns < 1], e[turns < 1] / 8)
    yarn = O.rope_freqs(1e4, 64, "yarn", 8.0, 1.0, 32.0, 8192)
    assert yarn[0] == 1 and yarn[31] == pytest.approx(e[31] / 8) and (np.diff(yarn) < 0).all()


def test_rope_turns_compose_and_leave_the_rest():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 2, 64))
    f = O.rope_freqs(1e4, 32)
    for layout in ("half", "pairs"):
        one = O.rope(O.rope(x, np.full(5, 9), f, layout), np.full(5, -4), f, layout)
        assert np.allclose(one, O.rope(x, np.full(5, 5), f, layout)) and np.array_equal(one[..., 32:], x[..., 32:])
    # the layouts are permutations of one another
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2), np.arange(32, 64)])
    assert np.allclose(O.rope(x, np.arange(5), f, "pairs")[..., perm], O.rope(x[..., perm], np.arange(5), f, "half"))


PROBE = r"""
#include <stddef.h>
#include <stdio.h>
#include "blend.h"
#define P(T, f) printf(#T "." #f " %zu\n", offsetof(T, f));
int main(void) {
  printf("blend_w4 %zu\nblend_rope %zu\nblend_rope_rows %zu\n", sizeof(blend_w4), sizeof(blend_rope), sizeof(blend_rope_rows));
  P(blend_w4, group) P(blend_w4, codes) P(blend_w4, scale)
  P(blend_rope, trained_len) P(blend_rope, theta) P(blend_rope, high) P(blend_rope, magnitude)
  P(blend_rope_rows, dst) P(blend_rope_rows, src_layer) P(blend_rope_rows, dst_row) P(blend_rope_rows, n_layers)
  printf("max %d %d %d %d\n", BLEND_MAX_TOP, BLEND_W4_SWIGLU, BLEND_ROPE_PAIRS, BLEND_ROPE_YARN);
  return 0;
}
"""


def test_structs_match_c(tmp_path):
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(PROBE)
    subprocess.run(["gcc", "-I", os.path.join(B.ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines()
    mirror = {"blend_w4": b.W4, "blend_rope": b.Rope, "blend_rope_rows": b.RopeRows}
    for line in out[:-1]:
        name, v = line.rsplit(" ", 1)
        s, _, f = name.partition(".")
        assert (getattr(mirror[s], f).offset if f else C.sizeof(mirror[s])) == int(v), name
    assert out[-1] == f"max {b.MAX_TOP} {b.W4_SWIGLU} {b.ROPE_PAIRS} {b.ROPE_YARN}"


def test_calls_without_a_handle_and_bad_descriptions():
    B.build()
    lib, vp = b.lib(), C.c_void_p(1 << 20)
    assert lib.w4_pack(None, None, vp, 8, None) == b.EINVAL
    assert lib.w4_unpack(None, None, vp, 8, None) == b.EINVAL
    assert lib.w4_linear(None, None, vp, 8, 1, vp, 8, b.F32, b.W4_STORE, None) == b.EINVAL
    assert lib.token_logprobs(None, vp, 8, b.F32, 1, 8, 1.0, vp, 1, vp, vp, 0, None, None, None) == b.EINVAL
    assert lib.rope_rows(None, None, None, 1, vp, vp, 1, None) == b.EINVAL
    codes, scale = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.bfloat16)
    ref = b.W4Ref(codes, scale, 136, 64)
    assert (ref.n, ref.k, ref.c.group) == (4, 136, 64)
    for bad in (lambda: b.W4Ref(codes, scale, 136, 48), lambda: b.W4Ref(codes, scale, 128, 64),
                lambda: b.W4Ref(codes, scale, 136, 32), lambda: b.W4Ref(codes.int(), scale, 136, 64),
                lambda: b.W4Ref(codes, scale.float(), 136, 64), lambda: b.W4Ref(codes.t(), scale, 136, 64),
                lambda: b.W4Ref(torch.zeros(4, 256, dtype=torch.uint8)[:, ::2], scale, 136, 64)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError, match="not on a GPU"):
        b.w4_linear(None, ref, torch.zeros(1, 136), torch.zeros(1, 4))
    with pytest.raises(ValueError, match="not on a GPU"):
        b.token_logprobs(None, torch.zeros(1, 136))
