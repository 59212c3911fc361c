"""Paged-cache calls at their edges: the reset after an error, totals and sizes at their limits, values and
queries of extreme size, and what masked tokens may hold."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from rag_kv_cache_rope_gb300 import binding as b
from pagedcase import attention_bound, f64, filled, handle, i32
from pagedtight import bound, few_bound, few_case, piece_bound, piece_case

pytestmark = pytest.mark.gpu


def status(h, stream=None):
    try:
        b.blend_device_status(h, stream)
        return b.OK
    except b.BlendError as e:
        return e.code


def attend(h, pages, q, q_start, lens, max_q, window=0, sink=0, stream=None):
    out = torch.full((q.shape[0], q.shape[1] * q.shape[2]), 3.0, dtype=q.dtype, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    b.paged_attention(h, pages, q, i32(q_start), i32(lens), max_q, out, window=window, n_sink=sink, stream=stream)
    return out


# ---------------------------------------------------------------- the reset after an error
def arrival_counters(h):
    """The handle's arrival counters, a part of its workspace: 640 of them, before the prefix sums of 152
    CTAs at its end."""
    ws = h._keep[1]
    need = b.blend_workspace_size(h.cfg, h.lim)
    at = need - -(-152 * (b.MAX_SEQS + 1) * 4 // 256) * 256 - 640 * 4
    return ws[at:at + 640 * 4].view(torch.int32)


def test_status_clears_what_an_interrupted_attention_left():
    """Arrivals that were counted by a call that gave up would let later parts be joined too early."""
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [3000, 700], 139)
    q = torch.randn(41, 8, 128, device="cuda").bfloat16()
    want = attend(h, c.pages, q, [0, 1, 41], [3000, 700], 40)
    assert status(h) == b.OK
    left = arrival_counters(h)
    assert not left.any()
    left.fill_(1)
    b.blend_wait_flag(h, i32([0]), 10)
    assert status(h) == b.ETIMEOUT and status(h) == b.OK
    assert not left.any()
    assert torch.equal(attend(h, c.pages, q, [0, 1, 41], [3000, 700], 40), want)
    assert status(h) == b.OK and not left.any()


def test_status_is_ordered_on_its_own_stream():
    """The reset goes through the call's stream: it neither waits for the default stream's work nor can it
    come behind it, into the next call on a stream that does not wait for the default one."""
    side = torch.cuda.Stream()
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [3000, 700], 139)
    q = torch.randn(41, 8, 128, device="cuda").bfloat16()
    want = attend(h, c.pages, q, [0, 1, 41], [3000, 700], 40)
    out, start, lens, zero = torch.zeros_like(want), i32([0, 1, 41]), i32([3000, 700]), i32([0])
    left = arrival_counters(h)

    def error_then_attention():
        with torch.cuda.stream(side):
            left.fill_(1)
        b.blend_wait_flag(h, zero, 10, stream=side)
        assert status(h, side) == b.ETIMEOUT and status(h, side) == b.OK
        b.paged_attention(h, c.pages, q, start, lens, 40, out, stream=side)
        assert status(h, side) == b.OK

    error_then_attention()  # once before: every kernel is loaded
    torch.cuda.synchronize()
    out.zero_()
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    torch.cuda._sleep(1 << 30)  # about half a second on the default stream
    busy.record()
    error_then_attention()
    assert not busy.query()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not left.any()


# ---------------------------------------------------------------- totals
def test_rows_claimed_again_and_again_are_reported():
    """Bounds that go down and up again: 512 sequences claim the same 8192 rows, more work units than 32 bits
    count.  Nothing of it is done, and the call says so."""
    hq, hkv, d, page, n_seq, rows, tokens = 256, 8, 64, 128, 1024, 8192, 1 << 17
    h = handle("bf16", hq, hkv, d)
    k = torch.zeros(1, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    pages = b.PagesRef(k, k.clone(), torch.zeros(n_seq, tokens // page, dtype=torch.int32, device="cuda"))
    q = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    out = attend(h, pages, q, [0, rows] * (n_seq // 2) + [0], [tokens] * n_seq, rows)
    assert status(h) == b.EDEVICE and bool((out == 3.0).all())


@pytest.mark.parametrize("dtype,fmt", [("bf16", "model"), ("bf16", "int4"), ("f32", "model")])
def test_rows_claimed_twice(dtype, fmt):
    """Rows that two sequences claim hold either's result; the first sequence's own rows are right."""
    h = handle(dtype, 8, 2, 128)
    c = filled(dtype, fmt, 2, 128, 16, [60, 60, 60], 3, poison=False)
    q = torch.randn(80, 8, 128, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    out = attend(h, c.pages, q, [0, 40, 20, 60], [60, 60, 60], 40)
    assert status(h) == b.EDEVICE and torch.isfinite(out).all()
    want, mag, lin = P.attention(f64(q[:40]), c.k[0], c.v[0], 60, 0, 0)
    lim = attention_bound(dtype, fmt, want, mag, lin, 60, True)
    assert (np.abs(f64(out[:20]).reshape(20, 8, 128) - want[:20]) <= lim[:20]).all()
    assert bool((out[60:] == 3.0).all())


# ---------------------------------------------------------------- 4-bit scales of any size
def scaled_pages(hkv, d, page, n, seed, k_exp, v_exp):
    """n tokens of one sequence with codes -8..7 of every dim and scales of full bf16 mantissas and exponents
    drawn from the given ranges, and their values n s in float64."""
    rng = np.random.default_rng(seed)
    n_pages = (n + page - 1) // page
    ten, val = [], []
    for lo, hi in (k_exp, v_exp):
        codes = rng.integers(-8, 8, (n_pages, hkv, page, d))
        sc = np.ldexp(1 + rng.integers(0, 128, (n_pages, hkv, page, d // 32)) / 128, rng.integers(lo, hi, (n_pages, hkv, page, d // 32)))
        packed = P.pack(codes, len(ten) == 1)
        x = P.unpack(packed, sc, len(ten) == 1)
        val.append(np.moveaxis(x, 1, 2).reshape(-1, hkv, d)[:n])
        ten.append((torch.from_numpy(packed).cuda(), torch.from_numpy(sc).to("cuda", torch.bfloat16)))
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None].contiguous()
    return b.PagesRef(ten[0][0], ten[1][0], table, ten[0][1], ten[1][1]), val[0], val[1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_gather_of_scales_of_any_size(dtype, d):
    """Every value is n s, from denormal scales to the largest whose values are finite, bit for bit."""
    h, n, dt = handle(dtype, 4, 2, d), 600, torch.bfloat16 if dtype == "bf16" else torch.float32
    pages, k, v = scaled_pages(2, d, 16, n, 7, (-126, 125), (118, 125))
    ko, vo = (torch.empty(n, 2, d, dtype=dt, device="cuda") for _ in range(2))
    b.paged_gather(h, pages, i32([0] * n), i32(list(range(n))), i32([n]), n, ko, vo)
    assert status(h) == b.OK
    assert torch.equal(ko.cpu(), torch.from_numpy(k).float().to(dt)) and torch.equal(vo.cpu(), torch.from_numpy(v).float().to(dt))
    assert torch.isfinite(vo).all()  # 8 (2 - 2^-7) 2^124 at most
    # turned: what a rotation adds is within its own rounding
    pages, k, v = scaled_pages(2, d, 16, n, 8, (118, 123), (118, 125))
    rot = np.arange(n) - n // 2
    b.paged_gather(h, pages, i32([0] * n), i32(list(range(n))), i32([n]), n, ko, vo, rot=i32(rot))
    lim = 4 * 2.0 ** -24 * np.abs(k).reshape(n, -1, 2, d // 2).sum(2).repeat(2, 1).reshape(n, -1, d)
    want = np.stack([P.rotate(k[i], rot[i], 1e4) for i in range(n)])
    assert (np.abs(f64(ko) - want) <= lim + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * (np.abs(want) + lim)).all()


SCALES = [((110, 115), (-100, 50)), ((122, 125), (-3, 2)), ((-110, -105), (40, 57))]


@pytest.mark.parametrize("rows", [1, 3, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k_exp,v_exp", SCALES)
def test_few_rows_over_scales_of_any_size(rows, d, k_exp, v_exp):
    n, h = 150, handle("bf16", 4, 1, d)
    pages, k, v = scaled_pages(1, d, 16, n, 10, k_exp, v_exp)
    g = torch.Generator().manual_seed(4)
    q = (torch.randn(rows, 4, d, generator=g).double() * 2.0 ** (-2 - k_exp[1])).to("cuda", torch.bfloat16)
    out = attend(h, pages, q, [0, rows], [n], rows, window=90, sink=5)
    assert status(h) == b.OK
    want, mag, lin = P.attention(f64(q), k, v, n, 90, 5)
    # P times the values' scale is rounded once, to bf16; queries below 2^-126 have fewer bits than fp32 products
    # keep of them: 2^-150 a product, times the largest scale
    lim = bound(want, mag, lin + d * 2.0 ** -126 * 2.0 ** k_exp[1], n, [2.0 ** -8], 2.0 ** -8)
    assert (np.abs(f64(out).reshape(rows, 4, d) - want) <= lim).all()


@pytest.mark.parametrize("rows", [1, 3, 8, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["model", "int4"])
def test_scores_of_queries_with_a_wide_range(rows, d, fmt):
    """Every eighth element of a query is 2^16 to 2^20 times the others, where the keys are 0: the scores are the
    small ones', and as near as sums of those alone."""
    n, h = 40, handle("bf16", 4, 1, d)
    rng = np.random.default_rng(11)
    big = np.arange(d) % 8 == 3
    codes = rng.integers(-7, 8, (3, 1, 16, d))
    codes[..., big] = 0
    sc = np.ldexp(1 + rng.integers(0, 128, (3, 1, 16, d // 32)) / 128, rng.integers(10, 13, (3, 1, 16, d // 32)))
    ones = np.full((3, 1, 16, d // 32), 0.125)
    vc = rng.integers(-7, 8, (3, 1, 16, d))
    table = i32([[2, 0, 1]])
    k, v = P.unpack(P.pack(codes, False), sc, False), P.unpack(P.pack(vc, True), ones, True)
    if fmt == "int4":
        pages = b.PagesRef(torch.from_numpy(P.pack(codes, False)).cuda(), torch.from_numpy(P.pack(vc, True)).cuda(), table,
                           torch.from_numpy(sc).to("cuda", torch.bfloat16), torch.from_numpy(ones).to("cuda", torch.bfloat16))
    else:
        k, v = P.bf16(k).astype(np.float64), P.bf16(v).astype(np.float64)
        pages = b.PagesRef(torch.from_numpy(k).to("cuda", torch.bfloat16), torch.from_numpy(v).to("cuda", torch.bfloat16), table)
    k, v = (np.moveaxis(x[[2, 0, 1]], 1, 2).reshape(-1, 1, d)[:n] for x in (k, v))
    q = rng.normal(size=(rows, 4, d)) * 2.0 ** -14
    q[..., big] *= 2.0 ** rng.integers(16, 21, (rows, 4, int(big.sum())))
    q = torch.from_numpy(q).to("cuda", torch.bfloat16)
    out = attend(h, pages, q, [0, rows], [n], rows)
    assert status(h) == b.OK
    want, mag, lin = P.attention(f64(q), k, v, n, 0, 0)
    # weights in bf16, those of pieces over 4-bit pages in fp16
    half = 2.0 ** -11 if fmt == "int4" and rows == 40 else 2.0 ** -8
    lim = bound(want, mag, lin, n, [half], 2.0 ** -8, lost=2.0 ** -30 if half < 2.0 ** -8 else 0.0, terms=2 if rows == 40 else 1)
    assert (np.abs(f64(out).reshape(rows, 4, d) - want) <= lim).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k_exp,v_exp", SCALES)
def test_pieces_over_scales_of_any_size(dtype, d, k_exp, v_exp):
    """Keys of every scale against queries that bring the scores to ordinary size, values up to 2^60."""
    n, rows = 150, 40
    h = handle(dtype, 4, 2, d)
    pages, k, v = scaled_pages(2, d, 16, n, 9, k_exp, v_exp)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(rows, 4, d, generator=g).double() * 2.0 ** (-2 - k_exp[1])
    q = q.to("cuda", torch.bfloat16 if dtype == "bf16" else torch.float32)
    out = attend(h, pages, q, [0, rows], [n], rows, window=90, sink=5)
    assert status(h) == b.OK
    want, mag, lin = P.attention(f64(q), k, v, n, 90, 5)
    got = f64(out).reshape(rows, 4, d)
    if dtype == "bf16":  # P and n s in bf16, keys in two parts
        lim = bound(want, mag, lin, n, [2.0 ** -8, 2.0 ** -8], 2.0 ** -8, lost=2.0 ** -30 * np.abs(v).max(), terms=2)
    else:
        lim = bound(want, mag, lin, n, [], 2.0 ** -24)
    assert (np.abs(got - want) <= lim).all(), (np.abs(got - want) / lim).max()


# ---------------------------------------------------------------- pieces over 4-bit pages, tight
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("seed", [12, 13, 14])
def test_int4_keys_of_pieces_are_exact(d, page, seed):
    """Scores within fp32 of those of n s, for scales of full mantissas."""
    n, rows, codes, sc, k, v, q = piece_case(d, seed)
    h = handle("bf16", 4, 1, d)
    n_pages = -(-n // page)
    table = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    ten = []
    for i in range(2):
        packed = np.zeros((n_pages, 1, page, d // 2), dtype=np.uint8)
        scale = np.full((n_pages, 1, page, d // 32), np.nan)
        for t in range(n):
            packed[table[t // page], :, t % page] = P.pack(codes[i, t], i == 1)
            scale[table[t // page], :, t % page] = sc[i, t]
        ten.append((torch.from_numpy(packed).cuda(), torch.from_numpy(scale).to("cuda", torch.bfloat16)))
    pages = b.PagesRef(ten[0][0], ten[1][0], i32(table)[None].contiguous(), ten[0][1], ten[1][1])
    out = attend(h, pages, torch.from_numpy(q).to("cuda", torch.bfloat16), [0, rows], [n], rows, window=12, sink=2)
    assert status(h) == b.OK
    want, mag, lin = P.attention(q, k, v, n, 12, 2)
    err = np.abs(f64(out).reshape(rows, 4, d) - want) / piece_bound(want, mag, lin, v)
    assert err.max() <= 1, err.max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 2, 4])
@pytest.mark.parametrize("seed", [15, 16])
def test_weights_of_few_rows_keep_their_bits(d, rows, seed):
    """Up to 16 (row, head) pairs a tile over bf16 pages: weights in two parts."""
    n, q, k, v = few_case(d, rows, seed)
    h = handle("bf16", 4, 1, d)
    ten = []
    for x in (k, v):
        pool = torch.full((4, 1, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        for t in range(n):
            pool[3 - t // 16, :, t % 16] = torch.from_numpy(x[t]).to("cuda", torch.bfloat16)
        ten.append(pool)
    out = attend(h, b.PagesRef(*ten, i32([[3, 2, 1, 0]])), torch.from_numpy(q).to("cuda", torch.bfloat16), [0, rows], [n], rows)
    assert status(h) == b.OK
    want, mag, lin = P.attention(q, k, v, n, 0, 0)
    err = np.abs(f64(out).reshape(rows, 4, d) - want) / few_bound(want, mag, lin, n)
    assert err.max() <= 1, err.max()


# ---------------------------------------------------------------- between the sinks and the window
@pytest.mark.parametrize("dtype,fmt", [("bf16", "model"), ("bf16", "int4"), ("f32", "model"), ("f32", "int4")])
@pytest.mark.parametrize("rows", [3, 48, 200])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_tokens_between_sinks_and_window_may_hold_anything(dtype, fmt, rows, page):
    """NaN and infinities in every token that no row sees, a part of a block, a page and a tile at both ends."""
    n, window, sink = 700, 60, 21
    h = handle(dtype, 8, 2, 128)
    c = filled(dtype, fmt, 2, 128, page, [n, n], 17, poison=False)
    q = torch.randn(2 * rows, 8, 128, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    start = [0, rows, 2 * rows]
    want = attend(h, c.pages, q, start, [n, n], rows, window, sink)
    assert status(h) == b.OK and torch.isfinite(want).all()
    tok = torch.arange(sink, n - rows - window + 1, device="cuda")
    ten = c.tensors
    for s in range(2):
        pg, at = ten["table"][s].long()[tok // page], tok % page
        for i, name in enumerate(("k", "v")):
            into = ten[name] if fmt == "model" else ten[name + "_scale"]
            into[pg, :, at] = float("nan")
            into[pg[i::3], :, at[i::3]] = float("inf")
            if fmt == "int4":
                ten[name][pg, :, at] = 0x8F
    got = attend(h, c.pages, q, start, [n, n], rows, window, sink)
    assert status(h) == b.OK
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


# ---------------------------------------------------------------- refusals
def test_numbers_past_32_bits_are_refused():
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [40], 3)
    q, out = torch.zeros(5, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 1024, dtype=torch.bfloat16, device="cuda")
    start, lens = i32([0, 5]), i32([40])
    before = b.blend_launch_count()
    for kw in (dict(window=(1 << 32) + 1), dict(window=1 << 31), dict(n_sink=(1 << 32) + 2), dict(n_sink=1 << 63)):
        with pytest.raises(ValueError):
            b.paged_attention(h, c.pages, q, start, lens, 5, out, **kw)
    with pytest.raises(ValueError):
        b.paged_attention(h, c.pages, q, start, lens, (1 << 32) + 5, out)
    assert b.blend_launch_count() == before
    b.paged_attention(h, c.pages, q, start, lens, 5, out, window=(1 << 31) - 1, n_sink=(1 << 31) - 1)
    assert status(h) == b.OK


def test_gathered_rows_over_each_other_are_refused():
    h = handle("bf16", 8, 2, 128)
    c = filled("bf16", "model", 2, 128, 16, [40], 3)
    rows = torch.zeros(10, 2, 128, dtype=torch.bfloat16, device="cuda")
    seq, pos, n = i32([0] * 5), i32(list(range(5))), i32([5])
    before = b.blend_launch_count()
    for ko, vo in ((rows[:5], rows[:5]), (rows[:5], rows[4:9]), (rows[3:8], rows[:5])):
        with pytest.raises(b.BlendError) as e:
            b.paged_gather(h, c.pages, seq, pos, n, 5, ko, vo)
        assert e.value.code == b.EINVAL
    assert b.blend_launch_count() == before
    b.paged_gather(h, c.pages, seq, pos, n, 5, rows[:5], rows[5:])
    assert status(h) == b.OK and rows.any()
