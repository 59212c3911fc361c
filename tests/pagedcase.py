"""Cases of the paged-cache tests: a handle of a given head shape, pages filled with known rows
in random page order, and the float64 values they stand for."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

from oracle import paged_oracle as P
from rag_kv_cache_rope_gb300 import binding as b

THETA, MAX_POS = 1e4, 4096
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
# half a rounding step relative to the value
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def handle(dtype, hq, hkv, d, max_pos=MAX_POS, stream=None):
    dt = TORCH[dtype]

    def zeros(*shape):
        return torch.zeros(*shape, dtype=dt, device="cuda")

    w = {"embed": zeros(16, 16), "attn_norm": zeros(1, 16), "w_qkv": zeros(1, (hq + 2 * hkv) * d, 16),
         "w_o": zeros(1, 16, hq * d), "mlp_norm": zeros(1, 16), "w_gu": zeros(1, 32, 16), "w_down": zeros(1, 16, 16),
         "final_norm": zeros(16)}
    cfg = b.ModelCfg(1, 16, hq, hkv, d, 16, 16, b.F32 if dtype == "f32" else b.BF16, THETA, 1e-6, max_pos)
    return b.blend_init(cfg, w, b.Limits(1, 1, 1, 1), stream=stream)


@dataclasses.dataclass
class Cache:
    """A paged cache and its float64 contents per sequence ([len][hkv][d])."""
    pages: b.PagesRef
    k: list
    v: list
    tensors: dict

    @property
    def table(self):
        return self.tensors["table"]


def table_of(lens, page, spare, rng, cols=None):
    need = [(n + page - 1) // page for n in lens]
    cols = cols or max(max(need), 1)
    order = rng.permutation(sum(need) + spare)
    t = np.full((len(lens), cols), -1, dtype=np.int32)  # never read past a sequence's pages
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = order[at:at + n]
        at += n
    return t


def filled(dtype, fmt, hkv, d, page, lens, seed, poison=True, cols=None):
    """Pages holding random rows of every sequence.  poison: everything no sequence holds (slots past
    a length, spare pages) is NaN, in the scales for 4-bit pages."""
    rng = np.random.default_rng(seed)
    t = table_of(lens, page, 2, rng, cols)
    n_pages = sum((n + page - 1) // page for n in lens) + 2
    shape = (n_pages, hkv, page, d)
    ks, vs = [], []
    if fmt == "model":
        pools = [np.full(shape, np.nan if poison else 0.0, dtype=np.float32) for _ in range(2)]
    else:
        pools = [rng.integers(0, 256, (*shape[:3], d // 2)).astype(np.uint8) for _ in range(2)]
        scales = [np.full((*shape[:3], d // 32), np.nan if poison else 1.0, dtype=np.float32) for _ in range(2)]
    for s, n in enumerate(lens):
        pos = np.arange(n)
        pg, row = t[s][pos // page], pos % page
        for i, into in enumerate((ks, vs)):
            x = rng.normal(size=(n, hkv, d)).astype(np.float32)
            if fmt == "model":
                if dtype == "bf16":
                    x = P.bf16(x)
                pools[i][pg, :, row] = x
                into.append(x.astype(np.float64))
            else:
                codes, sc = P.quantise(x)
                pools[i][pg, :, row] = P.pack(codes, i == 1)
                scales[i][pg, :, row] = sc
                into.append(P.unpack(P.pack(codes, i == 1), sc, i == 1))
    dt = TORCH[dtype] if fmt == "model" else torch.uint8
    ten = {"k": torch.from_numpy(pools[0]).to("cuda", dt), "v": torch.from_numpy(pools[1]).to("cuda", dt),
           "table": torch.from_numpy(t).cuda(), "k_scale": None, "v_scale": None}
    if fmt == "int4":
        ten["k_scale"], ten["v_scale"] = (torch.from_numpy(x).to("cuda", torch.bfloat16) for x in scales)
    return Cache(b.PagesRef(ten["k"], ten["v"], ten["table"], ten["k_scale"], ten["v_scale"]), ks, vs, ten)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def attention_bound(dtype, fmt, out, mag, lin, n_keys, many_rows):
    """How far a result may be from the float64 one, element by element.

    bf16, matrix instructions: the weights are rounded to bf16 (4-bit pages: once more with the
    values' scale), which moves a result by at most one half step of `mag` each, and the result is
    rounded.  Tiles of 4-bit pages for many rows turn keys and values into bf16 first: values move
    `mag` by another half step, keys a score by a half step of `lin`, hence a weight's share by
    exp(2 x).  fp32: a score is off by (d + 4) fp32 half steps of `lin` and 2^-22 from exp2, sums of
    n_keys terms by as many half steps (the fp32 part is in the bf16 bound too)."""
    d = out.shape[-1]
    u = 2.0 ** -24
    x = (d + 4) * u * lin + 2.0 ** -22
    if dtype == "bf16":
        r = STEP["bf16"]
        n_round = 1
        if fmt == "int4":
            n_round = 2
            if many_rows:
                x = x + r * lin
        base = (1 + r) ** n_round - 1
    else:
        base = 0.0
    moved = (np.exp(2 * x) - 1)[..., None] + base + (n_keys + 16) * u
    return moved * mag * 1.01 + STEP[dtype] * np.abs(out) + 1e-30
