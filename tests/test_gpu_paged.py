"""Paged-cache calls against the float64 oracle: append and gather (bit for bit where a value is only
moved or held in 4 bits), attention with windows and sinks over both page forms, refusals,
device-side checks, streams, captured graphs, and the calls together behind a blended prefill."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from rag_kv_cache_rope_gb300 import binding as b
from pagedcase import MAX_POS, STEP, TORCH, attention_bound, f64, filled, handle, i32

pytestmark = pytest.mark.gpu
THETA = 1e4


# ---------------------------------------------------------------- append
HEADS = [("bf16", 8, 2, 128), ("bf16", 9, 3, 64), ("f32", 4, 2, 64), ("f32", 5, 1, 128)]


def append_case(dtype, fmt, hq, hkv, d, page, seed, rot, n=37, pad=5, with_q=True):
    """Rows of a fused projection into poisoned pages; returns everything before and after."""
    rng = np.random.default_rng(seed)
    lens = [3, 50, 1, 20]
    c = filled(dtype, fmt, hkv, d, page, lens, seed, cols=(64 + page - 1) // page)
    # give every sequence all its columns
    t = np.arange(4 * c.table.shape[1], dtype=np.int32).reshape(4, -1)
    n_pages = t.size + 1
    ten = c.tensors
    for k in ("k", "v", "k_scale", "v_scale"):
        if ten[k] is not None:
            ten[k] = torch.cat([ten[k]] * (n_pages // ten[k].shape[0] + 1))[:n_pages].contiguous()
    ten["table"] = torch.from_numpy(rng.permutation(n_pages)[:t.size].reshape(t.shape).astype(np.int32)).cuda()
    pages = b.PagesRef(ten["k"], ten["v"], ten["table"], ten["k_scale"], ten["v_scale"])
    where = rng.permutation(4 * 64)[:n + pad]
    seq, pos = where // 64, where % 64
    seq[rng.permutation(n)[:3]] = -1
    x = rng.normal(size=(n + pad, hq + 2 * hkv, d)).astype(np.float32)
    qkv = torch.from_numpy(x).to("cuda", TORCH[dtype])
    r = None if rot is None else rng.integers(-rot, rot + 1, n + pad)
    return ten, pages, seq, pos, r, qkv


@pytest.mark.parametrize("dtype,hq,hkv,d", HEADS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("rot", [None, 0, MAX_POS - 1])
def test_append_model_pages(dtype, hq, hkv, d, page, rot):
    h = handle(dtype, hq, hkv, d)
    n = 37
    ten, pages, seq, pos, r, qkv = append_case(dtype, "model", hq, hkv, d, page, 11, rot, n)
    before = {k: ten[k].clone() for k in ("k", "v")}
    q_out = torch.full((n + 5, hq, d), 7.0, dtype=TORCH[dtype], device="cuda")
    b.paged_append(h, pages, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], i32(seq), i32(pos), i32([n]), n + 5,
                   q=qkv[:, :hq], q_out=q_out, rot=None if r is None else i32(r))
    b.blend_device_status(h)
    want_k, want_v = f64(before["k"]), f64(before["v"])
    touched = np.zeros(want_k.shape[:1] + want_k.shape[2:3], dtype=bool)
    x = f64(qkv)
    table = ten["table"].cpu().numpy()
    got_k, got_v, got_q = f64(ten["k"]), f64(ten["v"]), f64(q_out)
    for i in range(n):
        if seq[i] < 0:
            assert (got_q[i] == 7.0).all()
            continue
        by = pos[i] if r is None else r[i]
        pg, row = P.slot(table, page, seq[i], pos[i])
        touched[pg, row] = True
        want_v[pg, :, row] = x[i, hq + hkv:]
        # the fp32 rotation: cos, sin, two products and a sum, each half a step of |x1| + |x2|
        lim = 4 * 2.0 ** -24 * np.abs(x[i]).reshape(-1, 2, d // 2).sum(1).repeat(2, 0).reshape(-1, d)
        turned = P.rotate(x[i], by, THETA)
        for got, want, li in ((got_k[pg, :, row], turned[hq:hq + hkv], lim[hq:hq + hkv]),
                              (got_q[i], turned[:hq], lim[:hq])):
            assert (np.abs(got - want) <= li + STEP[dtype] * (np.abs(want) + li)).all()
            if by == 0:
                assert (got == want).all()
    assert (got_q[n:] == 7.0).all()
    assert np.array_equal(got_v, want_v, equal_nan=True)
    keep = ~touched
    assert np.array_equal(np.moveaxis(got_k, 1, 2)[keep], np.moveaxis(want_k, 1, 2)[keep], equal_nan=True)


@pytest.mark.parametrize("dtype,hq,hkv,d", HEADS)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("rot", [None, 700])
def test_append_int4_pages_bit_for_bit(dtype, hq, hkv, d, page, rot):
    h = handle(dtype, hq, hkv, d)
    n = 37
    ten, pages, seq, pos, r, qkv = append_case(dtype, "int4", hq, hkv, d, page, 12, rot, n)
    # groups of zeros, with an infinity, with a NaN, with tiny and with huge values
    live = np.flatnonzero(seq[:n] >= 0)
    qkv[live[0], hq:, :32] = 0
    qkv[live[1], hq, 3] = float("inf")
    qkv[live[2], hq + hkv, 5] = float("nan")
    qkv[live[3], hq:] *= 1e-30
    qkv[live[4], hq:] *= 1e30
    want = {k: ten[k].cpu().clone() for k in ("k", "v", "k_scale", "v_scale")}
    k_new, v_new = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    b.paged_append(h, pages, k_new, v_new, i32(seq), i32(pos), i32([n]), n + 5, rot=None if r is None else i32(r))
    b.blend_device_status(h)
    table = ten["table"].cpu().numpy()
    for i in range(n):
        if seq[i] < 0:
            continue
        pg, row = P.slot(table, page, seq[i], pos[i])
        with np.errstate(all="ignore"):
            kk = P.rotate_f32(k_new[i].float().cpu().numpy(), int(pos[i] if r is None else r[i]), THETA)
        for name, x in (("k", kk), ("v", v_new[i].float().cpu().numpy())):
            codes, sc = P.quantise(x)
            want[name][pg, :, row] = torch.from_numpy(P.pack(codes, name == "v"))
            want[name + "_scale"][pg, :, row] = torch.from_numpy(sc).to(torch.bfloat16)
    for k in want:
        got = ten[k].cpu()
        same = got.view(torch.int16 if got.dtype == torch.bfloat16 else torch.uint8) == \
            want[k].view(torch.int16 if got.dtype == torch.bfloat16 else torch.uint8)
        if got.dtype == torch.bfloat16:
            same |= torch.isnan(got) & torch.isnan(want[k])
        assert same.all(), k


def test_int4_scale_is_the_product_with_a_seventh():
    """Maxima just below ties of bf16, where a product with fp32's 1/7 and a division by 7 part."""
    tie = 7 * (1 + (1 + 2 * np.arange(64)) * 2.0 ** -8)
    m = np.nextafter(tie.astype(np.float32), np.float32(0)) * np.float32(2.0) ** np.arange(-32, 32).astype(np.float32)
    assert (P.bf16(m * (np.float32(1) / np.float32(7))) != P.bf16(m / np.float32(7))).any()
    rng = np.random.default_rng(3)
    x = (rng.uniform(-1, 1, (64, 4, 32)) * m[:, None, None]).astype(np.float32)
    x[:, :, 5] = m[:, None]
    x = x.reshape(64, 2, 64)
    h, c = handle("f32", 4, 2, 64), filled("f32", "int4", 2, 64, 64, [64], 3)
    kv = torch.from_numpy(x).cuda()
    b.paged_append(h, c.pages, kv, kv, i32([0] * 64), i32(list(range(64))), i32([64]), 64, rot=i32([0] * 64))
    b.blend_device_status(h)
    codes, s = P.quantise(x)
    at = int(c.table[0, 0])
    for i, (name, scale) in enumerate((("k", "k_scale"), ("v", "v_scale"))):
        assert np.array_equal(c.tensors[name][at].cpu().numpy(), P.pack(codes, i == 1).transpose(1, 0, 2))
        assert np.array_equal(f64(c.tensors[scale][at]), s.transpose(1, 0, 2))


def test_append_in_place_q_one_row_and_no_rows():
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [5], 3)
    q = torch.randn(1, 8, 128, device="cuda").bfloat16()
    kv = torch.randn(2, 1, 2, 128, device="cuda").bfloat16()
    want = P.rotate(f64(q)[0], 4, THETA)
    b.paged_append(h, c.pages, kv[0], kv[1], i32([0]), i32([4]), i32([1]), 1, q=q, q_out=q)
    assert (np.abs(f64(q)[0] - want) <= STEP["bf16"] * np.abs(want) + 1e-5).all()
    before = c.tensors["k"].clone()
    b.paged_append(h, c.pages, kv[0], kv[1], i32([0]), i32([2]), i32([0]), 1)
    b.paged_append(h, c.pages, kv[0][:0], kv[1][:0], i32([]), i32([]), i32([0]), 0)
    b.blend_device_status(h)
    assert torch.equal(torch.nan_to_num(before), torch.nan_to_num(c.tensors["k"]))


# ---------------------------------------------------------------- gather
@pytest.mark.parametrize("dtype,hq,hkv,d", HEADS)
@pytest.mark.parametrize("fmt", ["model", "int4"])
@pytest.mark.parametrize("rot", [None, MAX_POS - 1])
def test_gather_rows_and_values(dtype, hq, hkv, d, fmt, rot):
    h = handle(dtype, hq, hkv, d)
    lens = [33, 1, 80]
    c = filled(dtype, fmt, hkv, d, 32, lens, 21)
    rng = np.random.default_rng(5)
    n, pad = 61, 4
    seq = rng.integers(0, 3, n + pad)
    pos = np.array([rng.integers(0, lens[s]) for s in seq])
    seq[7] = -1
    seq[11], pos[11] = seq[10], pos[10]  # the same row twice
    r = None if rot is None else rng.integers(-rot, rot + 1, n + pad)
    k_out = torch.full((n + pad, hkv, d), 9.0, dtype=TORCH[dtype], device="cuda")
    v_out = torch.full_like(k_out, 9.0)
    b.paged_gather(h, c.pages, i32(seq), i32(pos), i32([n]), n + pad, k_out, v_out, rot=None if r is None else i32(r))
    b.blend_device_status(h)
    gk, gv = f64(k_out), f64(v_out)
    assert (gk[n:] == 9).all() and (gv[n:] == 9).all() and (gk[7] == 9).all() and (gv[7] == 9).all()
    for i in range(n):
        if i == 7:
            continue
        k, v = c.k[seq[i]][pos[i]], c.v[seq[i]][pos[i]]
        assert np.array_equal(gv[i], f64(torch.from_numpy(v).to(TORCH[dtype])))
        if r is None or r[i] == 0:
            assert np.array_equal(gk[i], f64(torch.from_numpy(k).to(TORCH[dtype])))
        else:
            want = P.rotate(k, r[i], THETA)
            lim = 4 * 2.0 ** -24 * np.abs(k).reshape(-1, 2, d // 2).sum(1).repeat(2, 0).reshape(-1, d)
            assert (np.abs(gk[i] - want) <= lim + STEP[dtype] * (np.abs(want) + lim)).all()


# ---------------------------------------------------------------- attention
# sequences as (query rows, length)
DECODE = [(1, 1), (1, 700), (1, 16), (1, 17), (0, 40), (1, 255)]
FEW = [(3, 3), (5, 200), (2, 90), (0, 0), (8, 65), (1, 33)]
EMPTY = [(4, 2), (1, 0), (3, 130), (0, 10)]
PIECE = [(70, 70), (130, 400), (1, 300), (33, 34), (64, 257)]
WINDOWS = [(0, 0), (1, 0), (100, 4), (40, 70), (5000, 3), (0, 9)]


def attend(h, c, q, q_start, lens, max_q, window=0, sink=0, **kw):
    out = torch.full((q.shape[0], q.shape[1] * q.shape[2]), 3.0, dtype=q.dtype, device="cuda")
    b.paged_attention(h, c.pages, q, q_start, i32(lens), max_q, out, window=window, n_sink=sink, **kw)
    return out


def check_attention(dtype, fmt, hq, hkv, d, page, seqs, window, sink, seed, scale=1.0, tc=True, spare_rows=3):
    h = handle(dtype, hq, hkv, d)
    if not tc:
        b.blend_set_tensor_cores(h, False)
    n_q, lens = [s[0] for s in seqs], [s[1] for s in seqs]
    c = filled(dtype, fmt, hkv, d, page, lens, seed)
    start = np.concatenate([[0], np.cumsum(n_q)])
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(start[-1] + spare_rows, hq + 1, d, generator=g) * scale).to("cuda", TORCH[dtype])
    q = wide[:, :hq]  # rows with a gap between them
    out = attend(h, c, q, i32(start), lens, max(n_q), window, sink)
    again = attend(h, c, q, i32(start), lens, max(n_q), window, sink)
    b.blend_device_status(h)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))  # bit for bit
    got = f64(out)
    assert (got[start[-1]:] == 3.0).all()  # rows behind the last sequence
    for s, (nq, ln) in enumerate(seqs):
        if nq == 0:
            continue
        qs = f64(q[start[s]:start[s + 1]])
        want, mag, lin = P.attention(qs, c.k[s], c.v[s], ln, window, sink)
        lim = attention_bound(dtype, fmt, want, mag, lin, ln, tc and nq * (hq // hkv) > 32)
        err = np.abs(got[start[s]:start[s + 1]].reshape(nq, hq, d) - want)
        assert np.isfinite(err).all(), (s, nq, ln)
        assert (err <= lim).all(), (s, nq, ln, (err / lim).max(), np.unravel_index((err / lim).argmax(), err.shape))


@pytest.mark.parametrize("fmt", ["model", "int4"])
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 9, 3, 64), ("f32", 4, 2, 64), ("f32", 5, 1, 128)])
@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("seqs", [DECODE, FEW, EMPTY], ids=["decode", "few", "empty"])
def test_attention(dtype, fmt, hq, hkv, d, window, sink, seqs):
    check_attention(dtype, fmt, hq, hkv, d, 16, seqs, window, sink, 31)


@pytest.mark.parametrize("fmt", ["model", "int4"])
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 10, 2, 128), ("bf16", 9, 3, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("window,sink", WINDOWS)
def test_attention_pieces(dtype, fmt, hq, hkv, d, window, sink):
    check_attention(dtype, fmt, hq, hkv, d, 32, PIECE, window, sink, 37)


@pytest.mark.parametrize("fmt", ["model", "int4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,d", [(32, 1, 128), (3, 3, 64), (12, 1, 128), (14, 2, 64)])
def test_attention_groups_and_pages(fmt, page, hq, hkv, d):
    check_attention("bf16", fmt, hq, hkv, d, page, [(1, 300), (2, 140), (0, 5), (1, 1)], 0, 0, 41)
    check_attention("bf16", fmt, hq, hkv, d, page, [(40, 300), (2, 140), (0, 5), (129, 129)], 90, 20, 43)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_attention_peaked_weights(dtype, fmt):
    """Rows whose weight sits on a few keys: a wrong key or a lost rescale shows in full."""
    check_attention(dtype, fmt, 8, 2, 128, 16, [(1, 900), (2, 333), (1, 64)], 0, 0, 47, scale=6.0)
    check_attention(dtype, fmt, 8, 2, 128, 64, [(50, 900), (140, 333)], 200, 5, 53, scale=6.0)


@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_attention_without_tensor_cores(fmt):
    check_attention("bf16", fmt, 8, 2, 128, 16, [(1, 300), (40, 90), (0, 3)], 60, 3, 59, tc=False)


def test_attention_long_ragged():
    """One long sequence beside short ones, lengths far below what the table allows."""
    h = handle("bf16", 8, 2, 128)
    lens = [20000, 3, 700, 1]
    c = filled("bf16", "model", 2, 128, 16, lens, 61, cols=2500)
    q = torch.randn(4, 8, 128, device="cuda").bfloat16()
    got = f64(attend(h, c, q, i32([0, 1, 2, 3, 4]), lens, 1)).reshape(4, 8, 128)
    b.blend_device_status(h)
    for s in range(4):
        want, mag, lin = P.attention(f64(q[s:s + 1]), c.k[s], c.v[s], lens[s], 0, 0)
        assert (np.abs(got[s] - want[0]) <= attention_bound("bf16", "model", want, mag, lin, lens[s], False)[0]).all()


@pytest.mark.parametrize("dtype,fmt", [("bf16", "model"), ("bf16", "int4"), ("f32", "model")])
@pytest.mark.parametrize("n_seq", [129, 300, 1024])
def test_attention_many_sequences(dtype, fmt, n_seq):
    """As many sequences as a table may have, some empty, and among few-row ones a few long pieces."""
    rng = np.random.default_rng(n_seq)
    seqs = [(int(rng.integers(0, 3)), int(rng.integers(0, 60))) for _ in range(n_seq)]
    seqs[n_seq // 2], seqs[-1] = (0, 0), (1, 7)
    check_attention(dtype, fmt, 4, 2, 64, 16, seqs, 0, 0, 73)
    if dtype == "bf16":
        for i in rng.integers(0, n_seq, 5):
            seqs[i] = (40, 40 + int(rng.integers(0, 90)))
        check_attention(dtype, fmt, 4, 2, 64, 16, seqs, 33, 5, 79)


@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_attention_parts_of_every_tile_size(fmt):
    """Long contexts of few heads, cut into many parts: 1 to 32 pairs, and two-tile items."""
    for hq, seqs in ((5, [(1, 5000)]), (4, [(3, 3000), (1, 20)]), (4, [(8, 3000), (5, 900)]), (16, [(1, 2500)]),
                     (4, [(40, 5000)]), (2, [(120, 2000), (300, 1500), (17, 900)]), (32, [(9, 2000)])):
        check_attention("bf16", fmt, hq, 1, 128, 64, seqs, 0, 0, 83)
    check_attention("bf16", fmt, 6, 2, 64, 32, [(150, 2600), (400, 400), (1, 1500)], 1000, 40, 89)


@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_short_sequences_in_a_call_sized_for_pieces(fmt):
    """Row counts that announce a full batch of pieces, and a device that holds shorter ones, or none."""
    h = handle("bf16", 8, 2, 128)
    lens = [300, 70, 0, 5, 1000]
    c = filled("bf16", fmt, 2, 128, 16, lens, 109)
    q = torch.randn(5 * 40, 8, 128, device="cuda").bfloat16()
    for n_q in ([40, 40, 0, 5, 1], [1, 1, 0, 1, 1], [0, 0, 0, 0, 40], [0, 0, 0, 0, 0], [40, 8, 1, 9, 40]):
        start = np.concatenate([[0], np.cumsum(n_q)])
        out = attend(h, c, q, i32(start), lens, 40)
        b.blend_device_status(h)
        assert (f64(out)[start[-1]:] == 3.0).all()
        for s in range(5):
            if n_q[s]:
                want, mag, lin = P.attention(f64(q[start[s]:start[s + 1]]), c.k[s], c.v[s], lens[s], 0, 0)
                lim = attention_bound("bf16", fmt, want, mag, lin, lens[s], True)
                got = f64(out[start[s]:start[s + 1]]).reshape(n_q[s], 8, 128)
                assert (np.abs(got - want) <= lim).all(), (n_q, s)


@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_queries_and_keys_of_extreme_size(fmt):
    """Scores of ordinary size from huge queries and tiny keys, and the other way round."""
    for up in (2.0 ** 60, 2.0 ** -60):
        for rows in (1, 40):
            h = handle("bf16", 8, 2, 128)
            c = filled("bf16", fmt, 2, 128, 16, [300], 97, poison=False)
            if fmt == "model":
                c.tensors["k"].div_(up)
            else:
                c.tensors["k_scale"].div_(up)
            q = (torch.randn(rows, 8, 128, device="cuda") * up).bfloat16()
            got = f64(attend(h, c, q, i32([0, rows]), [300], rows)).reshape(rows, 8, 128)
            want, mag, lin = P.attention(f64(q), c.k[0] / up, c.v[0], 300, 0, 0)
            assert (np.abs(got - want) <= attention_bound("bf16", fmt, want, mag, lin, 300, rows > 8)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_int4_values_of_pieces_are_exact(d):
    """Rows of few keys, keys that are bf16 values: what is left are the weights' fp16 rounding (half a
    step 2^-11, and 2^-30 of the largest weight where that is lost) and the result's."""
    rows, n = 70, 300
    h, c = handle("bf16", 8, 2, d), filled("bf16", "int4", 2, d, 32, [n], 131)
    ks = c.tensors["k_scale"]
    ks.copy_(torch.where(torch.isnan(ks), ks, torch.full_like(ks, 0.125)))
    k, v = torch.empty(2, n, 2, d, dtype=torch.bfloat16, device="cuda")
    b.paged_gather(h, c.pages, i32([0] * n), i32(list(range(n))), i32([n]), n, k, v)  # n / 8 is a bf16 value
    q = torch.randn(rows, 8, d, device="cuda").bfloat16()
    for window, sink in ((4, 0), (1, 2), (3, 1)):
        got = f64(attend(h, c, q, i32([0, rows]), [n], rows, window, sink)).reshape(rows, 8, d)
        want, mag, lin = P.attention(f64(q), f64(k), c.v[0], n, window, sink)
        x = (d + 4) * 2.0 ** -24 * lin + 2.0 ** -22
        moved = (np.exp(2 * x) - 1)[..., None] + 2.0 ** -11 + 20 * 2.0 ** -24
        lim = 1.01 * moved * mag + 4 * 2.0 ** -30 * np.abs(c.v[0]).max() + STEP["bf16"] * np.abs(want)
        assert (np.abs(got - want) <= lim).all(), (np.abs(got - want) / lim).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32])
def test_int4_value_scales_of_any_size(d, page):
    """Scales far from 1 and zero, over whole sequences, in turn by pages, and in single groups of 32 dims."""
    lens, n_q = [300, 500, 260, 400], [40, 64, 33, 128]
    h, c = handle("bf16", 8, 2, d), filled("bf16", "int4", 2, d, page, lens, 137)
    vs, table, rng = c.tensors["v_scale"], c.table.cpu().numpy(), np.random.default_rng(5)
    for s, n in enumerate(lens):
        for p in range((n + page - 1) // page):
            up = np.ones(d // 32)
            if s == 0:
                up[:] = 2.0 ** -40
            elif s == 1:
                up[:] = 2.0 ** (10 * (p // 2 % 3))  # 1, 2^10 and 2^20 by turns
            elif s == 2:
                up[rng.integers(d // 32)] = [2.0 ** 30, 2.0 ** -30, 0.0][p % 3]
            else:
                up[:] = 2.0 ** rng.integers(-8, 8)
            vs[int(table[s, p])] *= torch.from_numpy(up).to(vs)
            at = slice(p * page, min((p + 1) * page, n))
            c.v[s][at] *= up.repeat(32)
    start = np.concatenate([[0], np.cumsum(n_q)])
    q = torch.randn(start[-1], 8, d, device="cuda").bfloat16()
    for window, sink in ((0, 0), (70, 3)):
        out = f64(attend(h, c, q, i32(start.tolist()), lens, 128, window, sink))
        for s, n in enumerate(lens):
            got = out[start[s]:start[s + 1]].reshape(-1, 8, d)
            want, mag, lin = P.attention(f64(q[start[s]:start[s + 1]]), c.k[s], c.v[s], n, window, sink)
            lim = attention_bound("bf16", "int4", want, mag, lin, n, True)
            assert (np.abs(got - want) <= lim).all(), (s, (np.abs(got - want) / lim).max())
    b.blend_device_status(h)


@pytest.mark.parametrize("dtype,fmt", [("bf16", "model"), ("bf16", "int4"), ("f32", "model")])
@pytest.mark.parametrize("page", [16, 128])
def test_pages_left_behind_by_the_window_may_be_gone(dtype, fmt, page):
    """Table entries of pages that no row sees (a serving loop frees them) are not read or reported."""
    h = handle(dtype, 8, 2, 128)
    lens, window, sink = [1000, 700], 150, 3
    c = filled(dtype, fmt, 2, 128, page, lens, 101)
    for rows in (1, 40):
        t = c.table.clone()
        for s, n in enumerate(lens):
            lo = n - rows - window + 1
            for p in range(t.shape[1]):
                if p * page >= sink and (p + 1) * page <= lo:
                    t[s, p] = -5
        pages = b.PagesRef(c.tensors["k"], c.tensors["v"], t, c.tensors["k_scale"], c.tensors["v_scale"])
        q = torch.randn(2 * rows, 8, 128, device="cuda").to(TORCH[dtype])
        out = torch.empty(2 * rows, 1024, dtype=q.dtype, device="cuda")
        b.paged_attention(h, pages, q, i32([0, rows, 2 * rows]), i32(lens), rows, out, window=window, n_sink=sink)
        b.blend_device_status(h)
        for s, n in enumerate(lens):
            want, mag, lin = P.attention(f64(q[s * rows:(s + 1) * rows]), c.k[s], c.v[s], n, window, sink)
            lim = attention_bound(dtype, fmt, want, mag, lin, window + rows + 3, rows > 8)
            assert (np.abs(f64(out[s * rows:(s + 1) * rows]).reshape(rows, 8, 128) - want) <= lim).all()


@pytest.mark.parametrize("rows", [1, 40])
def test_two_handles_on_two_streams(rows):
    """Handles have workspaces of their own: calls in flight together give what they give alone."""
    case = []
    for seed in (103, 107):
        h, st = handle("bf16", 8, 2, 128), torch.cuda.Stream()
        lens = [5000, 300, 2100]
        c = filled("bf16", "model", 2, 128, 16, lens, seed)
        q = torch.randn(3 * rows, 8, 128, device="cuda").bfloat16()
        start = i32([0, rows, 2 * rows, 3 * rows])
        alone = attend(h, c, q, start, lens, rows)
        case.append((h, st, c, q, start, i32(lens), alone, torch.empty_like(alone)))
    torch.cuda.synchronize()
    for _ in range(20):
        for h, st, c, q, start, lens, _, out in case:
            b.paged_attention(h, c.pages, q, start, lens, rows, out, stream=st)
    torch.cuda.synchronize()
    for h, *_, alone, out in case:
        assert torch.equal(alone, out)
        b.blend_device_status(h)


def test_nan_in_a_query_reaches_its_row_alone():
    for fmt, rows in (("model", 1), ("int4", 1), ("model", 60), ("int4", 60)):
        h = handle("bf16", 8, 2, 128)
        c = filled("bf16", fmt, 2, 128, 16, [200, 200], 67)
        q = torch.randn(2 * rows, 8, 128, device="cuda").bfloat16()
        q[0, 3, 5] = float("nan")
        out = attend(h, c, q, i32([0, rows, 2 * rows]), [200, 200], rows).reshape(2 * rows, 8, 128)
        bad = torch.isnan(out).any(-1)
        assert bad[0, 3] and torch.isnan(out[0, 3]).all() and bad.sum() == 1
    h = handle("f32", 8, 2, 128)
    c = filled("f32", "model", 2, 128, 16, [200], 67)
    q = torch.randn(1, 8, 128, device="cuda")
    q[0, 3, 5] = float("nan")
    out = attend(h, c, q, i32([0, 1]), [200], 1).reshape(8, 128)
    assert torch.isnan(out[3]).all() and torch.isnan(out).any(-1).sum() == 1


@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_masked_tokens_may_hold_anything(fmt):
    """Tokens between the sinks and the window hold NaN: single-token rows do not notice."""
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", fmt, 2, 128, 16, [400], 71)
    t, page = c.table.cpu().numpy(), 16
    for j in range(7, 400 - 50):
        pg, row = P.slot(t, page, 0, j)
        if fmt == "model":
            c.tensors["k"][pg, :, row] = float("nan")
            c.tensors["v"][pg, :, row] = float("inf")
        else:
            c.tensors["k_scale"][pg, :, row] = float("nan")
            c.tensors["v_scale"][pg, :, row] = float("nan")
    q = torch.randn(1, 8, 128, device="cuda").bfloat16()
    got = f64(attend(h, c, q, i32([0, 1]), [400], 1, 50, 7)).reshape(1, 8, 128)
    want, mag, lin = P.attention(f64(q), c.k[0], c.v[0], 400, 50, 7)
    assert (np.abs(got - want) <= attention_bound("bf16", fmt, want, mag, lin, 57, False)).all()


# ---------------------------------------------------------------- offsets past 32 bits
@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_pool_past_32_bit_offsets(fmt):
    hq, hkv, d, page = 8, 8, 128, 128
    n_pages = (1 << 31) // (hkv * page * d) * (1 if fmt == "model" else 2) + 40  # the last pages start past 2^31
    h = handle("bf16", hq, hkv, d)
    if fmt == "model":
        k = torch.zeros(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
        ks = vs = None
    else:
        k = torch.zeros(n_pages, hkv, page, d // 2, dtype=torch.uint8, device="cuda")
        ks = torch.zeros(n_pages, hkv, page, d // 32, dtype=torch.bfloat16, device="cuda")
        vs = torch.zeros_like(ks)
    v = torch.zeros_like(k)
    n = 300
    table = i32([[n_pages - 1, 0, n_pages - 3]])
    pages = b.PagesRef(k, v, table, ks, vs)
    x = torch.randn(2, n, hkv, d, device="cuda").bfloat16()
    seq, pos = i32([0] * n), i32(list(range(n)))
    b.paged_append(h, pages, x[0], x[1], seq, pos, i32([n]), n, rot=i32([0] * n))
    ko, vo = torch.empty_like(x[0]), torch.empty_like(x[1])
    b.paged_gather(h, pages, seq, pos, i32([n]), n, ko, vo)
    b.blend_device_status(h)
    if fmt == "model":
        assert torch.equal(ko, x[0]) and torch.equal(vo, x[1])
    kk, vv = [], []
    for i, into in ((0, kk), (1, vv)):
        if fmt == "model":
            into.append(f64(x[i]))
        else:
            codes, sc = P.quantise(x[i].float().cpu().numpy())
            into.append(P.unpack(P.pack(codes, i == 1), sc, i == 1))
            assert np.array_equal(f64((ko, vo)[i]), f64(torch.from_numpy(into[0]).bfloat16()))
    for rows in (1, 40):
        q = torch.randn(rows, hq, d, device="cuda").bfloat16()
        out = torch.empty(rows, hq * d, dtype=torch.bfloat16, device="cuda")
        b.paged_attention(h, pages, q, i32([0, rows]), i32([n]), rows, out)
        want, mag, lin = P.attention(f64(q), kk[0], vv[0], n, 0, 0)
        lim = attention_bound("bf16", fmt, want, mag, lin, n, rows > 32)
        assert (np.abs(f64(out).reshape(rows, hq, d) - want) <= lim).all()


def test_append_rows_that_take_two_launches():
    """More rows than the threads of one launch, queries in place: rows on both sides of the border are
    rotated once.  All rows but a few are padding."""
    hq, hkv, d = 32, 2, 64
    most = (1 << 31) // ((hq + hkv) * (d // 16))
    n = most + 700
    need = n * d * (hq + 2 * hkv) * 2 + 3 * n * 4
    if torch.cuda.mem_get_info()[0] < need + (20 << 30):
        pytest.skip("needs some 95 GB of free memory")
    h = handle("bf16", hq, hkv, d)
    c = filled("bf16", "model", hkv, d, 16, [64], 109)
    q = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(2, n, hkv, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, most - 512, most - 1, most, most + 1, n - 1] + [most // 512 * 512 + i for i in range(-1, 40)])
    q[rows.cuda()] = torch.randn(len(rows), hq, d, device="cuda").bfloat16()
    kv[:, rows.cuda()] = torch.randn(2, len(rows), hkv, d, device="cuda").bfloat16()
    seq, pos = torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    where = torch.arange(len(rows), dtype=torch.int32, device="cuda")
    seq[rows.cuda()], pos[rows.cuda()] = 0, where
    before = f64(q[rows.cuda()])
    b.paged_append(h, c.pages, kv[0], kv[1], seq, pos, i32([n]), n, q=q, q_out=q)
    b.blend_device_status(h)
    got = f64(q[rows.cuda()])
    for i, r in enumerate(rows):
        want = P.rotate(before[i], i, THETA)
        assert (np.abs(got[i] - want) <= STEP["bf16"] * np.abs(want) + 1e-5).all(), r
    ko, vo = torch.empty(2, len(rows), hkv, d, dtype=torch.bfloat16, device="cuda")
    b.paged_gather(h, c.pages, i32([0] * len(rows)), where, i32([len(rows)]), len(rows), ko, vo)
    assert torch.equal(vo, kv[1][rows.cuda()])
    del q, kv
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- refusals and device-side checks
def test_refused_calls_launch_nothing():
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [40], 3)
    lib = b.lib()
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    out = torch.empty(2, 1024, dtype=torch.bfloat16, device="cuda")
    st, ln, n = i32([0, 1]), i32([40]), i32([1])
    P_, L_ = q.data_ptr(), b.blend_launch_count

    def pg(**kw):
        x = b.Pages(*[getattr(c.pages.c, f) for f, _ in b.Pages._fields_])
        for k, v in kw.items():
            setattr(x, k, v)
        return C.byref(x)

    def att(p=None, qp=P_, ld=1024, s=st.data_ptr(), l=ln.data_ptr(), rows=1, mq=1, win=0, sink=0, o=out.data_ptr()):
        return lib.paged_attention(h.ptr, p or pg(), qp, ld, s, l, rows, mq, win, sink, o, None)

    def app(p=None, k=P_, ldk=256, v=P_, ldv=256, qq=None, ldq=0, qo=None, s=st.data_ptr(), ps=ln.data_ptr(),
            m=n.data_ptr(), mx=1):
        return lib.paged_append(h.ptr, p or pg(), k, ldk, v, ldv, qq, ldq, qo, s, ps, None, m, mx, None)

    before = L_()
    for kw in (dict(format=2), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=256), dict(n_pages=0),
               dict(n_seq=0), dict(n_seq=1025), dict(max_pages=0), dict(max_pages=(1 << 20) + 1), dict(table=None),
               dict(k=None), dict(v=None), dict(k=P_ + 2), dict(v=P_ + 8), dict(table=P_ + 2),
               dict(format=b.PAGES_INT4), dict(format=b.PAGES_INT4, k_scale=P_, v_scale=P_ + 2)):
        assert att(pg(**kw)) == b.EINVAL and app(pg(**kw)) == b.EINVAL, kw
        assert lib.paged_gather(h.ptr, pg(**kw), st.data_ptr(), ln.data_ptr(), None, n.data_ptr(), 1, P_, P_,
                                None) == b.EINVAL
    for kw in (dict(qp=None), dict(qp=P_ + 2), dict(ld=1020), dict(ld=1000), dict(ld=1028), dict(s=None), dict(l=None),
               dict(rows=-1), dict(mq=0), dict(mq=-1), dict(win=-1), dict(sink=-1), dict(o=None), dict(o=P_),
               dict(o=out.data_ptr() + 4), dict(rows=(1 << 24) + 1)):
        assert att(**kw) == b.EINVAL, kw
    for kw in (dict(k=None), dict(v=None), dict(k=P_ + 2), dict(ldk=248), dict(ldv=260), dict(qq=P_), dict(qo=P_),
               dict(qq=P_, qo=P_, ldq=1032), dict(qq=P_, qo=P_ + 16, ldq=1016), dict(s=None), dict(ps=None),
               dict(m=None), dict(mx=-1), dict(mx=(1 << 24) + 1)):
        assert app(**kw) == b.EINVAL, kw
    for a in ((None, P_, P_), (st.data_ptr(), None, P_), (st.data_ptr(), P_, None), (st.data_ptr(), P_ + 2, P_)):
        assert lib.paged_gather(h.ptr, pg(), a[0], ln.data_ptr(), None, n.data_ptr(), 1, a[1], a[2], None) == b.EINVAL
    big = pg(n_seq=1024, max_pages=1 << 20)
    assert att(big) == b.EINVAL and b"2^31" in lib.blend_last_error(h.ptr)
    assert att(rows=0, mq=0) == b.OK and app(mx=0) == b.OK
    assert L_() == before
    for bad in (lambda: b.paged_attention(h, c.pages, q.float(), st, ln, 1, out),
                lambda: b.paged_attention(h, c.pages, q, st.long(), ln, 1, out),
                lambda: b.paged_attention(h, c.pages, q, st[:1], ln, 1, out),
                lambda: b.paged_attention(h, c.pages, q, st, ln, 1, out[:1]),
                lambda: b.paged_attention(h, c.pages, q[..., :64], st, ln, 1, out),
                lambda: b.paged_attention(h, c.pages, q.cpu(), st, ln, 1, out),
                lambda: b.paged_attention(handle("f32", 8, 2, 128), c.pages, q, st, ln, 1, out),
                lambda: b.paged_attention(handle("bf16", 8, 4, 128), c.pages, q, st, ln, 1, out)):
        with pytest.raises(ValueError):
            bad()
    assert L_() <= before + 4  # the two handles' own


def test_outputs_over_inputs_are_refused():
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [40], 3)
    buf = torch.zeros(32768, dtype=torch.bfloat16, device="cuda")
    rows, at = 5, buf.data_ptr()
    start, ln, n = i32([0, rows]), i32([40]), i32([rows])
    seq, pos = i32([0] * rows), i32(list(range(rows)))
    lib, before = b.lib(), b.blend_launch_count()

    def att(q, ld, o):
        return lib.paged_attention(h.ptr, c.pages.ref, at + 2 * q, ld, start.data_ptr(), ln.data_ptr(), rows, rows, 0, 0,
                                   at + 2 * o, None)

    def app(k, v, ldk, q, ldq, qo):
        return lib.paged_append(h.ptr, c.pages.ref, at + 2 * k, ldk, at + 2 * v, ldk, at + 2 * q, ldq, at + 2 * qo,
                                seq.data_ptr(), pos.data_ptr(), None, n.data_ptr(), rows, None)

    for a in ((0, 1024, 1024), (0, 1024, 5112), (5112, 1024, 0), (0, 2048, 9208), (1024, 1024, 1024)):
        assert att(*a) == b.EINVAL, a
    for a in ((0, 16384, 256, 8192, 1024, 1272), (16384, 0, 256, 8192, 1024, 1272), (20000, 24000, 256, 0, 1024, 5112),
              (1024, 1280, 1536, 0, 1536, 7672)):
        assert app(*a) == b.EINVAL, a
    assert b.blend_launch_count() == before
    assert att(0, 1024, 5120) == b.OK and att(0, 2048, 9216) == b.OK
    assert app(20000, 24000, 256, 0, 1024, 8192) == b.OK and app(20000, 24000, 256, 0, 1024, 0) == b.OK
    assert app(1024, 1280, 1536, 0, 1536, 7680) == b.OK
    b.blend_device_status(h)


def status(h):
    try:
        b.blend_device_status(h)
        return b.OK
    except b.BlendError as e:
        return e.code


@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_bad_rows_are_skipped_and_reported(fmt):
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", fmt, 2, 128, 16, [40, 40], 3, poison=False)
    kv = torch.randn(2, 9, 2, 128, device="cuda").bfloat16()
    t = c.table.clone()
    t[1, 2] = c.tensors["k"].shape[0]  # one past the pool
    pages = b.PagesRef(c.tensors["k"], c.tensors["v"], t, c.tensors["k_scale"], c.tensors["v_scale"])
    seq, pos = [2, 0, 0, 1, 0, 0, 0, -1, 0], [0, -1, 48, 39, 5, 6, 7, 900, 8]
    rot = [0, 0, 0, 0, MAX_POS, -MAX_POS, 0, 0, 0]
    before = {k: v.clone() for k, v in c.tensors.items() if v is not None}
    b.paged_append(h, pages, kv[0], kv[1], i32(seq), i32(pos), i32([9]), 9, rot=i32(rot))
    assert status(h) == b.EDEVICE and status(h) == b.OK
    rows = {P.slot(t.cpu().numpy(), 16, 0, p) for p in (7, 8)}
    for name in ("k", "v"):
        diff = (before[name].view(torch.uint8) != c.tensors[name].view(torch.uint8)).flatten(3).any(3).any(1)
        assert {tuple(x) for x in diff.nonzero().tolist()} == rows
    ko, vo = torch.full_like(kv[0], 4.0), torch.full_like(kv[1], 4.0)
    b.paged_gather(h, pages, i32(seq), i32(pos), i32([9]), 9, ko, vo, rot=i32(rot))
    assert status(h) == b.EDEVICE
    for i in range(9):
        assert bool((ko[i] == 4).all()) == (i not in (6, 8)) and bool((vo[i] == 4).all()) == (i not in (6, 8))
    # counts outside 0..max_n
    for n, want in ((12, 2), (-3, 0)):
        ko.fill_(4.0)
        b.paged_gather(h, pages, i32([0, 0]), i32([1, 2]), i32([n]), 2, ko, vo)
        assert status(h) == b.EDEVICE and int((ko != 4).flatten(1).any(1).sum()) == want


@pytest.mark.parametrize("fmt", ["model", "int4"])
@pytest.mark.parametrize("rows", [1, 40])
def test_bad_sequences_are_skipped_and_reported(fmt, rows):
    h = handle("bf16", 8, 2, 128)
    lens = [60, 60, 60]
    c = filled("bf16", fmt, 2, 128, 16, lens, 3, poison=False)
    q = torch.randn(3 * rows, 8, 128, device="cuda").bfloat16()
    good = attend(h, c, q, i32([0, rows, 2 * rows, 3 * rows]), lens, rows)
    assert status(h) == b.OK
    parts = [P.attention(f64(q[s * rows:(s + 1) * rows]), c.k[s], c.v[s], 60, 0, 0) for s in range(3)]

    def right(s, part):
        # (a skipped sequence shifts where the others' keys are split, so not bit for bit)
        lim = attention_bound("bf16", fmt, *parts[s], 60, rows * 4 > 32)
        return (np.abs(f64(part).reshape(rows, 8, 128) - parts[s][0]) <= lim).all()

    assert all(right(s, good[s * rows:(s + 1) * rows]) for s in range(3))
    for start, ln, skipped in (([0, rows, 2 * rows, 3 * rows], [60, 65, 60], 1), ([0, rows, 2 * rows, 3 * rows], [60, -1, 60], 1),
                               ([0, rows, 2 * rows, 3 * rows + 1], lens, 2), ([-1, rows, 2 * rows, 3 * rows], lens, 0)):
        out = attend(h, c, q, i32(start), ln, rows + 1)
        assert status(h) == b.EDEVICE
        for s in range(3):
            part = out[s * rows:(s + 1) * rows]
            assert bool((part == 3.0).all()) == (s == skipped)
            if s != skipped:
                assert right(s, part)
    # more rows than max_q says
    out = attend(h, c, q, i32([0, rows, 3 * rows, 3 * rows]), lens, rows)
    assert status(h) == b.EDEVICE and bool((out[rows:] == 3.0).all()) and right(0, out[:rows])
    # a page index outside the pool inside a length
    t = c.table.clone()
    t[1, 1] = -7
    bad = b.PagesRef(c.tensors["k"], c.tensors["v"], t, c.tensors["k_scale"], c.tensors["v_scale"])
    out = torch.zeros_like(good)
    b.paged_attention(h, bad, q, i32([0, rows, 2 * rows, 3 * rows]), i32(lens), rows, out)
    assert status(h) == b.EDEVICE
    assert torch.equal(out[:rows], good[:rows]) and torch.equal(out[2 * rows:], good[2 * rows:])


def test_attention_after_an_expired_wait():
    """blend_device_status after a timeout leaves the handle as it was: parts are joined as before."""
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [3000, 700], 139)
    q, start = torch.randn(41, 8, 128, device="cuda").bfloat16(), i32([0, 1, 41])
    want = attend(h, c, q, start, [3000, 700], 40)
    b.blend_wait_flag(h, i32([0]), 10)
    assert status(h) == b.ETIMEOUT and status(h) == b.OK
    assert torch.equal(attend(h, c, q, start, [3000, 700], 40), want)
    b.blend_device_status(h)


# ---------------------------------------------------------------- streams, graphs
@pytest.mark.parametrize("dtype,fmt", [("bf16", "model"), ("bf16", "int4"), ("f32", "model")])
def test_captured_decode_steps_replay_with_new_lengths(dtype, fmt):
    """One captured append + attention replayed as the sequences grow, against separate calls."""
    hq, hkv, d, page, steps = 8, 2, 128, 16, 5
    lens0 = [300, 15, 60]
    h, side = handle(dtype, hq, hkv, d), torch.cuda.Stream()
    c = filled(dtype, fmt, hkv, d, page, [n + steps for n in lens0], 5, poison=False)
    ref = filled(dtype, fmt, hkv, d, page, [n + steps for n in lens0], 5, poison=False)
    x = torch.randn(steps, 3, hq + 2 * hkv, d, device="cuda").to(TORCH[dtype])
    cur, pos, lens = x[0].clone(), i32(lens0), i32([n + 1 for n in lens0])
    seq, n, start = i32([0, 1, 2]), i32([3]), i32([0, 1, 2, 3])
    q, out = torch.empty(3, hq, d, dtype=TORCH[dtype], device="cuda"), torch.empty(3, hq * d, dtype=TORCH[dtype], device="cuda")

    def step(pages, stream=None):
        b.paged_append(h, pages, cur[:, hq:hq + hkv], cur[:, hq + hkv:], seq, pos, n, 3, q=cur[:, :hq], q_out=q,
                       stream=stream)
        b.paged_attention(h, pages, q, start, lens, 1, out, window=100, n_sink=4, stream=stream)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(c.pages)
    for i in range(steps):
        cur.copy_(x[i])
        pos.copy_(i32([m + i for m in lens0]))
        lens.copy_(i32([m + i + 1 for m in lens0]))
        g.replay()
        got = out.clone()
        side.wait_stream(torch.cuda.current_stream())
        step(ref.pages, side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, out)
    b.blend_device_status(h)
    assert torch.equal(c.tensors["k"].view(torch.uint8), ref.tensors["k"].view(torch.uint8))


@pytest.mark.parametrize("fmt", ["model", "int4"])
@pytest.mark.parametrize("most", [48, 60])
def test_captured_pieces_replay_with_new_lengths(fmt, most):
    """Pieces in a captured call (one launch where every sequence could have max_q rows, else two),
    replayed between eager calls with other row counts and lengths."""
    h, other, side = handle("bf16", 8, 2, 128), handle("bf16", 8, 2, 128), torch.cuda.Stream()
    c = filled("bf16", fmt, 2, 128, 16, [900, 500, 70], 127, poison=False)
    q = torch.randn(144, 8, 128, device="cuda").bfloat16()
    start, lens = i32([0, 48, 96, 144]), i32([900, 500, 70])
    out = torch.empty(144, 1024, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        b.paged_attention(h, c.pages, q, start, lens, most, out, window=300, n_sink=4, stream=side)
    for rows, ln in (([48, 48, 48], [900, 500, 70]), ([1, 48, 0], [17, 48, 0]), ([40, 7, 33], [41, 300, 33])):
        start.copy_(i32(np.concatenate([[0], np.cumsum(rows)]).tolist()))
        lens.copy_(i32(ln))
        out.fill_(3.0)
        g.replay()
        got = out.clone()
        out.fill_(3.0)
        b.paged_attention(other, c.pages, q, start, lens, most, out, window=300, n_sink=4)
        assert torch.equal(got, out)
        b.paged_attention(h, c.pages, q, start, lens, most, out, window=300, n_sink=4)
        assert torch.equal(got, out)
    b.blend_device_status(h)


# ---------------------------------------------------------------- together, behind a prefill
@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_prefill_then_pages_then_decode(fmt):
    """A full prefill's finished cache goes into pages (keys as they are), the query rows attend over
    them, tokens are appended and attended, and the pages come back as a contiguous cache."""
    from rag_kv_cache_rope_gb300 import synth
    hq, hkv, d, L = 8, 2, 128, 2
    sh = synth.ModelShape("paged-bf16", L, 256, hq, hkv, d, 512, 300, THETA)
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(1)
    Pn, lens, Q = 8, [64, 48], 16
    w = synth.model_weights(sh, 0)
    rows = [Pn + n for n in lens]
    tok = torch.cat([synth.token_ids(r, sh.vocab, g) for r in rows]).to(dev)
    zeros = torch.zeros(L, sum(rows), hkv, d, dtype=torch.bfloat16, device=dev)
    pool = b.PoolRef(zeros, zeros.clone(), tok, Pn, lens, [0, rows[0]])
    N = Pn + sum(lens) + Q
    h = b.blend_init(b.model_cfg(sh, 1024), b.pack_weights({k: v.to(dev) for k, v in w.items()}),
                     b.Limits(N, N, sum(lens), 1))
    out = b.OutputsRef(k=torch.zeros(L, N, hkv, d, dtype=torch.bfloat16, device=dev),
                       v=torch.zeros(L, N, hkv, d, dtype=torch.bfloat16, device=dev),
                       hidden=torch.zeros(Q, 256, dtype=torch.bfloat16, device=dev),
                       q_last=torch.zeros(Q, hq, d, dtype=torch.bfloat16, device=dev))
    req = b.RequestRef([0, 1], synth.token_ids(Q, sh.vocab, g).to(dev), mode="full")
    b.blend_prefill(h, [req], pool, out)
    K, V = out["k"][L - 1], out["v"][L - 1]
    page, steps = 32, 3
    cols = (N + steps + page - 1) // page
    shape = (cols + 1, hkv, page, d if fmt == "model" else d // 2)
    dt = torch.bfloat16 if fmt == "model" else torch.uint8
    ten = [torch.zeros(shape, dtype=dt, device=dev) for _ in range(2)]
    sc = [torch.zeros(*shape[:3], d // 32, dtype=torch.bfloat16, device=dev) if fmt == "int4" else None for _ in range(2)]
    table = torch.arange(cols, 0, -1, dtype=torch.int32, device=dev)[None].contiguous()
    pages = b.PagesRef(ten[0], ten[1], table, *sc)
    ids = torch.arange(N, dtype=torch.int32, device=dev)
    zero = torch.zeros_like(ids)
    b.paged_append(h, pages, K, V, zero, ids, i32([N]), N, rot=zero)
    ko, vo = torch.empty_like(K), torch.empty_like(V)
    b.paged_gather(h, pages, zero, ids, i32([N]), N, ko, vo)
    if fmt == "model":
        assert torch.equal(ko, K) and torch.equal(vo, V)
        kk, vv = f64(K), f64(V)
    else:
        kk, vv = (P.unpack(P.pack(*(lambda q: (q[0], v_))(P.quantise(f64(t).astype(np.float32)))),
                           P.quantise(f64(t).astype(np.float32))[1], v_) for t, v_ in ((K, False), (V, True)))
        assert np.array_equal(f64(ko), f64(torch.from_numpy(kk).bfloat16()))
    got = torch.empty(Q, hq * d, dtype=torch.bfloat16, device=dev)
    b.paged_attention(h, pages, out["q_last"], i32([0, Q]), i32([N]), Q, got)
    want, mag, lin = P.attention(f64(out["q_last"]), kk, vv, N, 0, 0)
    assert (np.abs(f64(got).reshape(Q, hq, d) - want) <= attention_bound("bf16", fmt, want, mag, lin, N, True)).all()
    for i in range(steps):
        x = torch.randn(1, hq + 2 * hkv, d, device=dev).bfloat16()
        q, o = torch.empty(1, hq, d, dtype=torch.bfloat16, device=dev), torch.empty(1, hq * d, dtype=torch.bfloat16, device=dev)
        b.paged_append(h, pages, x[:, hq:hq + hkv], x[:, hq + hkv:], i32([0]), i32([N + i]), i32([1]), 1, q=x[:, :hq], q_out=q)
        b.paged_attention(h, pages, q, i32([0, 1]), i32([N + i + 1]), 1, o, window=64, n_sink=Pn)
        b.blend_device_status(h)
        k1 = P.rotate_f32(f64(x)[0, hq:hq + hkv], N + i, THETA)
        v1 = f64(x)[0, hq + hkv:].astype(np.float32)
        if fmt == "model":
            k1, v1 = P.bf16(k1), P.bf16(v1)
        else:
            k1, v1 = (P.unpack(P.pack(P.quantise(t)[0], v_), P.quantise(t)[1], v_) for t, v_ in ((k1, False), (v1, True)))
        kk, vv = np.concatenate([kk, k1[None]]), np.concatenate([vv, v1[None]])
        want, mag, lin = P.attention(f64(q), kk, vv, N + i + 1, 64, Pn)
        lim = attention_bound("bf16", fmt, want, mag, lin, 80, False)
        assert (np.abs(f64(o).reshape(1, hq, d) - want) <= lim).all()
