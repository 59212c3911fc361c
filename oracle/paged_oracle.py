"""Plain float64 restatement of the paged-cache calls (include/blend.h, "paged cache"): page
lookup, the 4-bit form, rotation, and attention with a sliding window and sinks, written as
loops over rows, tokens and heads.  Test infrastructure only; the 4-bit codes alone follow the
format's fp32 steps, since their bits are part of the format."""
from __future__ import annotations

import numpy as np

F32 = np.float32


def bf16(x):
    """Round to the nearest bf16 (ties to even); NaN and infinities stay."""
    x = np.asarray(x, dtype=F32)
    u = x.view(np.uint32)
    r = ((u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)).view(F32)
    return np.where(np.isfinite(x), r, x)


def slot(table, page_tokens, seq, pos):
    """(page, row in page) of token pos of a sequence."""
    return int(table[seq][pos // page_tokens]), pos % page_tokens


def rotate(x, pos, theta):
    """x [heads][d] (float64) rotated by pos positions: pairs (i, i + d/2), angle pos theta^(-2i/d)."""
    half = x.shape[-1] // 2
    a = pos * np.power(float(theta), -2.0 * np.arange(half) / (2 * half))
    c, s = np.cos(a), np.sin(a)
    x1, x2 = x[..., :half], x[..., half:]
    return np.concatenate([x1 * c - x2 * s, x2 * c + x1 * s], -1)


def rotate_f32(x, pos, theta):
    """The same with cos and sin rounded to fp32 and every product and sum rounded to fp32."""
    half = x.shape[-1] // 2
    if pos == 0:
        return np.asarray(x, dtype=F32)
    a = abs(pos) * np.power(float(theta), -2.0 * np.arange(half) / (2 * half))
    c, s = np.cos(a).astype(F32), np.sin(a).astype(F32)
    if pos < 0:
        s = -s
    x = np.asarray(x, dtype=F32)
    x1, x2 = x[..., :half], x[..., half:]
    return np.concatenate([x1 * c - x2 * s, x2 * c + x1 * s], -1)


def quantise(x):
    """(codes -7..7, scales) of x [..][d] fp32: 32 dims share bf16(max|x| * (1/7 in fp32));
    a group that is not finite gets a NaN scale and codes 0."""
    y = np.asarray(x, dtype=F32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(all="ignore"):
        fin = np.isfinite(y).all(-1)
        s = np.where(fin, bf16(np.abs(np.where(np.isfinite(y), y, 0)).max(-1) * (F32(1) / F32(7))), F32(np.nan))
        n = np.where((s > 0)[..., None], np.clip(np.rint(y / s[..., None]), -7, 7), 0)
    return n.reshape(x.shape).astype(np.int64), s


def dim_place(d, dim, value_row):
    """(byte, shift) of a dim's code in a packed row of d / 2 bytes."""
    g, r = divmod(dim, 32)
    if value_row:
        r, e = divmod(r, 4)
        bit = 8 * (r * (d // 16) + 2 * g) + 4 * e
    else:
        c, e = divmod(r, 8)
        bit = 8 * (c * (d // 8) + 4 * g) + 4 * (e // 2) + 16 * (e % 2)
    return bit // 8, bit % 8


def pack(codes, value_row):
    """Codes [..][d] to bytes [..][d / 2]."""
    d = codes.shape[-1]
    out = np.zeros((*codes.shape[:-1], d // 2), dtype=np.uint8)
    for dim in range(d):
        b, sh = dim_place(d, dim, value_row)
        out[..., b] |= ((codes[..., dim] + 8) << sh).astype(np.uint8)
    return out


def unpack(packed, scales, value_row):
    """Values (float64) of packed rows [..][d / 2] with scales [..][d / 32]."""
    d = packed.shape[-1] * 2
    out = np.zeros((*packed.shape[:-1], d))
    for dim in range(d):
        b, sh = dim_place(d, dim, value_row)
        out[..., dim] = (((packed[..., b].astype(np.int64) >> sh) & 15) - 8) * scales[..., dim // 32].astype(np.float64)
    return out


def visible(p, window, n_sink):
    """Tokens a row at position p sees, ascending."""
    return [j for j in range(p + 1) if window == 0 or j > p - window or j < n_sink]


def attention(q, k, v, kv_len, window, n_sink):
    """One sequence: q [n_q][hq][d], its last tokens; k, v [kv_len][hkv][d], float64.  Returns
    (out, mag, lin): out [n_q][hq][d]; mag the same with |v| (what a relative change of the weights
    moves); lin [n_q][hq] the largest sum |q_e k_e| / sqrt(d) over the keys seen."""
    n_q, hq, d = q.shape
    group = hq // k.shape[1]
    out, mag, lin = np.zeros((n_q, hq, d)), np.zeros((n_q, hq, d)), np.zeros((n_q, hq))
    for i in range(n_q):
        see = visible(kv_len - n_q + i, window, n_sink)
        if not see:
            continue
        for h in range(hq):
            kk, vv = k[see, h // group], v[see, h // group]
            s = kk @ q[i, h] / np.sqrt(d)
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
            lin[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() / np.sqrt(d)
    return out, mag, lin
