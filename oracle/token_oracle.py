"""Plain float64 restatement of what follows a finished cache per token: products with 4-bit
weights, log probabilities, rotary positions of other layouts.  Test infrastructure; shares no
code with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.paged_oracle import bf16


# ---------------------------------------------------------------- 4-bit weights
def w4_quantise(w: np.ndarray, group: int):
    """(codes 0..15 [n][k], scales [n][ceil(k / group)]) of float32 w [n][k]."""
    n, k = w.shape
    codes = np.full((n, k), 8, dtype=np.int64)
    scales = np.zeros((n, -(-k // group)))
    for g in range(scales.shape[1]):
        x = w[:, g * group:(g + 1) * group].astype(np.float64)
        top = np.abs(x).max(axis=1)
        bad = ~np.isfinite(top)
        s = bf16((np.where(bad, 0.0, top) / 7).astype(np.float32)).astype(np.float64)
        q = np.divide(x, s[:, None], out=np.zeros_like(x), where=(s > 0)[:, None] & np.isfinite(x))
        codes[:, g * group:(g + 1) * group] = np.where(bad[:, None], 8, 8 + np.clip(np.rint(q), -7, 7))
        scales[:, g] = np.where(bad, np.nan, s)
    return codes, scales


def w4_place(i: int):
    """(byte, shift) of input i's code in a packed row."""
    chunk, r = divmod(i, 128)
    word, r = divmod(r, 32)
    t, e = divmod(r, 8)
    bit = 4 * (e // 2) + 16 * (e % 2)
    return 64 * chunk + 4 * (4 * t + word) + bit // 8, bit % 8


def w4_rows(codes: np.ndarray) -> np.ndarray:
    """Packed rows, uint8 [n][ceil(k / 128) * 64]; padding holds codes of 8."""
    n, k = codes.shape
    chunks = -(-k // 128)
    rows = np.zeros((n, chunks * 64), dtype=np.uint8)
    for i in range(chunks * 128):
        byte, shift = w4_place(i)
        rows[:, byte] |= ((codes[:, i] if i < k else np.full(n, 8)) << shift).astype(np.uint8)
    return rows


def w4_values(codes: np.ndarray, scales: np.ndarray, group: int) -> np.ndarray:
    return (codes - 8.0) * np.repeat(scales, group, axis=1)[:, :codes.shape[1]]


def silu(x):
    return x / (1 + np.exp(-x))


def w4_linear(values: np.ndarray, x: np.ndarray, swiglu: bool = False) -> np.ndarray:
    y = x.astype(np.float64) @ values.T
    if swiglu:
        y = y.reshape(y.shape[0], -1, 2, 16)
        y = (silu(y[:, :, 0]) * y[:, :, 1]).reshape(y.shape[0], -1)
    return y


# ---------------------------------------------------------------- log probabilities
def logprobs(logits: np.ndarray, scale: float, ids: np.ndarray, top: int):
    """logp of ids, entropy, top ids and their logp."""
    z = logits.astype(np.float64) * scale
    rows, vocab = z.shape
    logp, entropy = np.zeros(ids.shape), np.zeros(rows)
    top_id, top_logp = np.zeros((rows, top), dtype=np.int64), np.zeros((rows, top))
    for r in range(rows):
        if np.isnan(z[r]).any() or (z[r] == np.inf).any():
            lp, entropy[r] = np.full(vocab, np.nan), np.nan
        elif (z[r] == -np.inf).all():
            lp = np.full(vocab, -np.inf)
        else:
            m = z[r].max()
            lp = (z[r] - m) - math.log(np.exp(z[r] - m).sum())
            p = np.exp(lp)
            entropy[r] = -(p[p > 0] * lp[p > 0]).sum()
        for i, t in enumerate(ids[r]):
            logp[r, i] = 0.0 if t < 0 else lp[t]
        x = logits[r].astype(np.float64)
        order = sorted(range(vocab), key=lambda j: (math.isnan(x[j]), 0.0 if math.isnan(x[j]) else -x[j], j))[:top]
        top_id[r], top_logp[r] = order, lp[order]
    return logp, entropy, top_id, top_logp


# ---------------------------------------------------------------- rotary positions
def rope_freqs(theta, rot_dim, scaling="none", factor=1.0, low=0.0, high=0.0, trained_len=0):
    if scaling == "base":
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    f = []
    for i in range(rot_dim // 2):
        e = theta ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            e /= factor
        elif scaling == "bands":
            m = min(1.0, max(0.0, (trained_len * e / (2 * math.pi) - low) / (high - low)))
            e *= m + (1 - m) / factor
        elif scaling == "yarn":
            a, b = (rot_dim * math.log(trained_len / (2 * math.pi * t)) / (2 * math.log(theta)) for t in (high, low))
            a, b = max(0, math.floor(a)), min(rot_dim - 1, math.ceil(b))
            m = 1 - min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            e *= m + (1 - m) / factor
        f.append(e)
    return np.array(f)


def rope(x: np.ndarray, rot: np.ndarray, freqs: np.ndarray, layout: str, magnitude: float = 1.0) -> np.ndarray:
    """x [..][rows][heads][d] turned by rot [rows] positions."""
    n = 2 * len(freqs)
    a, b = (slice(0, n // 2), slice(n // 2, n)) if layout == "half" else (slice(0, n, 2), slice(1, n, 2))
    angle = rot.astype(np.float64)[:, None, None] * freqs
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    y = x.astype(np.float64).copy()
    x1, x2 = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    return y
