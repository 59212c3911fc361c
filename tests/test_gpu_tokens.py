"""Token operators on the GPU against the float64 oracle: 4-bit weights (pack, read back, products),
log probabilities, rotary positions of every layout and scaling.

Bounds count roundings: half a step of the output's type relative to the value, and of fp32 sums one
step of 2^-23 (the matrix unit may cut where it adds) for each addition, relative to the sum of magnitudes."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as O
from rag_kv_cache_rope_gb300 import binding as b
from tests.pagedcase import STEP, TORCH, f64, handle, i32

pytestmark = pytest.mark.gpu

_handles = {}


def model(dtype, hq=4, hkv=2, d=128):
    key = (dtype, hq, hkv, d)
    if key not in _handles:
        _handles[key] = handle(dtype, hq, hkv, d)
    return _handles[key]


def inside(got, want, bound):
    """Equal infinities and NaN, and the rest within bound."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    special = ~np.isfinite(want)
    assert np.array_equal(got[special], want[special], equal_nan=True)
    err, bound = np.abs(got[~special] - want[~special]), np.broadcast_to(bound, want.shape)[~special]
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(err / np.maximum(bound, 1e-300))))


# ---------------------------------------------------------------- 4-bit weights
def weights(n, k, group, seed):
    """Codes of every value, scales of any size; in the packed form the scales' padding is poisoned."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (n, k))
    scales = rng.uniform(0.5, 2.0, (n, -(-k // group))) * 2.0 ** rng.integers(-8, 3, (n, 1))
    scales = torch.from_numpy(scales).to(torch.bfloat16)
    chunks = -(-k // 128)
    held = torch.full((n, chunks * (128 // group)), float("nan"), dtype=torch.bfloat16)
    held[:, :scales.shape[1]] = scales
    rows = torch.from_numpy(O.w4_rows(codes))
    w4 = b.W4Ref(rows.cuda(), held.cuda(), k, group)
    return w4, O.w4_values(codes, scales.double().numpy(), group)


def read_back(w4):
    """The float64 values of packed weights, from their bytes."""
    bytes_ = w4.codes.cpu().numpy()
    codes = np.empty((w4.n, w4.k), dtype=np.int64)
    for i in range(w4.k):
        byte, shift = O.w4_place(i)
        codes[:, i] = (bytes_[:, byte] >> shift) & 15
    return O.w4_values(codes, w4.scale.double().cpu().numpy(), w4.group)


def linear_bounds(values, x, out_dtype, swiglu):
    k = x.shape[1]
    mag = np.abs(x) @ np.abs(values).T
    y = x @ values.T
    err = (3 * k / 16 + k / 32 + 64) * 2.0 ** -23 * mag
    if swiglu:
        y, err = (v.reshape(x.shape[0], -1, 2, 16) for v in (y, err))
        (g, u), (eg, eu) = (y[:, :, 0], y[:, :, 1]), (err[:, :, 0], err[:, :, 1])
        s = O.silu(g)
        # |silu'| stays below 1.1; the exponential and the division are off by less than (2 + |g|) 2^-21 of it
        es = 1.1 * eg + (2 + np.abs(g)) * 2.0 ** -21 * np.abs(s)
        err = (np.abs(u) * es + np.abs(s) * eu + es * eu).reshape(x.shape[0], -1)
        y = (s * u).reshape(x.shape[0], -1)
    return y, err * 1.01 + STEP[out_dtype] * (np.abs(y) + err) + 1e-30


def rows_of(dtype, rows, k, seed, scale=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.full((rows, k + pad), float("nan"), dtype=TORCH[dtype])
    x[:, :k] = torch.randn(rows, k, generator=g) * scale
    return x.cuda()[:, :k]


LINEAR = [  # rows, n, k, group
    (1, 16, 8, 32), (1, 1, 128, 128), (2, 17, 136, 64), (3, 100, 256, 32), (1, 1537, 688, 32), (8, 48, 1536, 128),
    (9, 64, 688, 64), (16, 33, 1024, 128), (17, 96, 328, 64), (40, 200, 576, 32), (5, 4096, 5120, 128),
    (1, 256, 32768, 128), (2, 32, 14336, 64), (130, 320, 512, 128), (1, 6000, 4096, 32), (300, 256, 1000, 32),
    (64, 1000, 640, 64), (33, 2048, 2048, 32), (513, 130, 264, 128), (257, 384, 8, 32), (30, 128, 32768, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k,group", LINEAR)
def test_linear(rows, n, k, group, dtype):
    h = model(dtype)
    w4, values = weights(n, k, group, rows * n + k)
    x = rows_of(dtype, rows, k, 3, pad=8 if rows > 1 else 0)
    for out in ("bf16", "f32"):
        room = torch.full((rows + 1, n + 3), 7.0, dtype=TORCH[out], device="cuda")
        b.w4_linear(h, w4, x, room[:rows, 1:n + 1])
        want, bound = linear_bounds(values, f64(x), out, False)
        inside(f64(room[:rows, 1:n + 1]), want, bound)
        room[:rows, 1:n + 1] = 7.0
        assert bool((room == 7.0).all()), "written outside y"
    b.blend_device_status(h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k,group", [(1, 32, 128, 32), (3, 1376, 256, 128), (12, 64, 5120, 64), (20, 96, 688, 32),
                                            (1, 27648, 512, 32), (150, 128, 640, 128), (70, 2048, 1024, 64)])
def test_linear_swiglu_and_add(rows, n, k, group, dtype):
    h = model(dtype)
    w4, values = weights(n, k, group, 5)
    w4.scale.copy_((w4.scale.float() / 16).to(torch.bfloat16))  # (a power of two: exact)
    values = values / 16
    x = rows_of(dtype, rows, k, 4, 0.3)
    for out in ("bf16", "f32"):
        room = torch.full((rows + 1, n // 2 + 1), 7.0, dtype=TORCH[out], device="cuda")
        b.w4_linear(h, w4, x, room[:rows, :n // 2], epi="swiglu")
        want, bound = linear_bounds(values, f64(x), out, True)
        inside(f64(room[:rows, :n // 2]), want, bound)
        assert bool((room[rows:] == 7.0).all()) and bool((room[:, n // 2:] == 7.0).all())
    base = torch.randn(rows, n, device="cuda")
    y = base.clone()
    b.w4_linear(h, w4, x, y, epi="add")
    want, bound = linear_bounds(values, f64(x), "f32", False)
    want = want + f64(base)
    inside(f64(y), want, bound + STEP["f32"] * np.abs(want))
    b.blend_device_status(h)


def test_linear_outliers_with_weights_of_zero():
    """Sums hold up where one input is far larger than the others and its weights are 0: such products are
    exact zeros, so the others keep their bits."""
    h = model("bf16")
    for rows in (3, 40):
        w4, values = weights(64, 512, 64, 9)
        x = rows_of("bf16", rows, 512, 5)
        x[:, 100] = 2.0 ** 60
        x[1] *= 2.0 ** -100
        codes = np.rint(values / np.repeat(w4.scale.double().cpu().numpy(), 64, 1)).astype(np.int64) + 8
        codes[:, 100] = 8
        w4.codes.copy_(b.w4_layout(torch.from_numpy(codes)))
        values = read_back(w4)
        y = torch.empty(rows, 64, device="cuda")
        b.w4_linear(h, w4, x, y)
        xs = f64(x)
        xs[:, 100] = 0
        want, bound = linear_bounds(values, xs, "f32", False)
        inside(f64(y), want, bound)


def test_linear_nan_and_infinity_stay_in_their_row():
    h = model("bf16")
    for rows in (4, 30, 200):
        w4, values = weights(48, 256, 32, 11)
        x = rows_of("bf16", rows, 256, 6)
        clean = torch.empty(rows, 48, device="cuda")
        b.w4_linear(h, w4, x, clean)
        x[1, 7], x[2, 200] = float("nan"), float("inf")
        y = torch.empty(rows, 48, device="cuda")
        b.w4_linear(h, w4, x, y)
        keep = [r for r in range(rows) if r not in (1, 2)]
        assert torch.equal(y[keep], clean[keep]) and bool(y[1].isnan().all()) and not bool(y[2].isfinite().any())


def test_linear_is_deterministic_and_captures():
    h = model("bf16")
    for rows, n, k in ((1, 6144, 4096), (8, 512, 5120), (64, 1024, 1024), (200, 640, 2048)):
        w4, _ = weights(n, k, 128, 12)
        x = rows_of("bf16", rows, k, 7)
        y, z = (torch.empty(rows, n, device="cuda") for _ in range(2))
        b.w4_linear(h, w4, x, y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.w4_linear(h, w4, x, z)
        for _ in range(3):
            z.fill_(-1)
            graph.replay()
            assert torch.equal(y, z)
        # new inputs in the same place
        x.mul_(2)
        graph.replay()
        b.w4_linear(h, w4, x, y)
        assert torch.equal(y, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,group", [(1, 8, 32), (5, 128, 128), (33, 136, 64), (100, 688, 32), (17, 1000, 128), (300, 5120, 64)])
def test_pack_and_read_back(n, k, group, dtype):
    h = model(dtype)
    rng = np.random.default_rng(n + k)
    w = (rng.normal(size=(n, k)) * np.exp(rng.normal(size=(n, 1)) * 4)).astype(np.float32)
    w[0, :min(k, 40)] = 0
    if n > 4:
        w[1, 3], w[2, -1], w[3] = np.nan, -np.inf, 1e-40
        w[4, :8] = [7, -7, 3.5, 2.5, -0.5, 1.5, 0.5, 6.5]
        w[4, 8:] = 0.25
    room = torch.full((n, k + 8), float("nan"), dtype=TORCH[dtype], device="cuda")
    room[:, :k] = torch.from_numpy(w).cuda()
    w = room[:, :k].float().cpu().numpy()
    w4 = b.W4Ref.empty(n, k, group)
    w4.codes.fill_(255)
    w4.scale.fill_(7)
    b.w4_pack(h, room[:, :k], w4)
    codes, scales = O.w4_quantise(w, group)
    assert np.array_equal(w4.codes.cpu().numpy(), O.w4_rows(codes))
    held = w4.scale.double().cpu().numpy()
    assert np.array_equal(held[:, :scales.shape[1]], scales, equal_nan=True) and not held[:, scales.shape[1]:].any()
    out = torch.full((n + 1, k + 8), 3.0, dtype=TORCH[dtype], device="cuda")
    b.w4_unpack(h, w4, out[:n, :k])
    want = torch.from_numpy(O.w4_values(codes, scales, group)).to(TORCH[dtype])
    assert torch.equal(out[:n, :k].cpu().nan_to_num(9), want.nan_to_num(9))
    assert bool((out[n:] == 3).all()) and bool((out[:, k:] == 3).all())


def test_pack_fp32_quotients_at_borders():
    """Values next to a half-way quotient: the code is that of the exact quotient."""
    h = model("f32")
    rng = np.random.default_rng(3)
    w = np.zeros((64, 128), dtype=np.float32)
    top = rng.uniform(1, 2, 64).astype(np.float32)
    s = torch.from_numpy(top / np.float32(7)).to(torch.bfloat16).float().numpy()
    for r in range(64):
        half = (rng.integers(-7, 7, 127) + 0.5) * np.float64(s[r])
        w[r, 1:] = np.nextafter(half.astype(np.float32), rng.choice([-9, 9], 127).astype(np.float32))
        w[r, 0] = top[r]
        w[r] = np.clip(w[r], -top[r], top[r])
    w4 = b.W4Ref.empty(64, 128, 128)
    b.w4_pack(h, torch.from_numpy(w).cuda(), w4)
    codes, _ = O.w4_quantise(w, 128)
    assert np.array_equal(w4.codes.cpu().numpy(), O.w4_rows(codes))


def test_w4_refusals():
    h = model("bf16")
    w4, _ = weights(64, 256, 64, 1)
    x, y = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), torch.full((4, 64), 5.0, device="cuda")
    glu = torch.zeros(4, 32, device="cuda")
    lib, E, p = b.lib(), b.EINVAL, lambda t: t.data_ptr()

    def raw(w=w4.ref, x_=None, ld_x=256, rows=4, y_=None, ld_y=64, dt=b.F32, epi=b.W4_STORE):
        return lib.w4_linear(h.ptr, w, p(x) if x_ is None else x_, ld_x, rows, p(y) if y_ is None else y_, ld_y, dt, epi, None)

    bad_w = [b.W4(0, 256, 64, p(w4.codes), p(w4.scale)), b.W4(64, 252, 64, p(w4.codes), p(w4.scale)),
             b.W4(64, 32776, 64, p(w4.codes), p(w4.scale)), b.W4(64, 256, 48, p(w4.codes), p(w4.scale)),
             b.W4(64, 256, 64, None, p(w4.scale)), b.W4(64, 256, 64, p(w4.codes) + 8, p(w4.scale))]
    calls = [lambda w=w: raw(w=C.byref(w)) for w in bad_w]
    calls += [lambda: raw(w=None), lambda: raw(x_=p(x) + 2), lambda: raw(ld_x=248), lambda: raw(ld_x=260),
              lambda: raw(rows=-1), lambda: raw(rows=(1 << 18) + 1), lambda: raw(ld_y=63), lambda: raw(dt=2),
              lambda: raw(epi=3), lambda: raw(epi=b.W4_ADD, dt=b.BF16), lambda: raw(y_=p(y) + 2), lambda: raw(y_=p(x)),
              lambda: raw(y_=p(w4.codes)), lambda: lib.w4_pack(h.ptr, w4.ref, None, 256, None),
              lambda: lib.w4_pack(h.ptr, w4.ref, p(x), 128, None),
              lambda: lib.w4_unpack(h.ptr, w4.ref, p(w4.codes), 256, None)]
    before = b.blend_launch_count()
    for i, f in enumerate(calls):
        assert f() == E, i
    assert raw(rows=0) == b.OK
    w_odd = b.W4(48 + 8, 256, 64, p(w4.codes), p(w4.scale))
    assert raw(w=C.byref(w_odd), epi=b.W4_SWIGLU) == E and b"multiple of 32" in lib.blend_last_error(h.ptr)
    for f in (lambda: b.w4_linear(h, w4, x.float(), y), lambda: b.w4_linear(h, w4, x[:, :128], y),
              lambda: b.w4_linear(h, w4, x, y[:3]), lambda: b.w4_linear(h, w4, x, glu),
              lambda: b.w4_linear(h, w4, x.cpu(), y), lambda: b.w4_linear(h, w4, x, y.half()),
              lambda: b.w4_linear(model("f32"), w4, x, y), lambda: b.w4_linear(h, w4, x.t().contiguous().t(), y)):
        with pytest.raises(ValueError):
            f()
    assert bool((y == 5).all()) and b.blend_launch_count() == before


# ---------------------------------------------------------------- log probabilities
def logprobs(h, logits, ids, top, scale):
    rows = logits.shape[0]
    got = dict(logp=torch.full(ids.shape, 9.0, device="cuda"), entropy=torch.full((rows,), 9.0, device="cuda"),
               top_id=torch.full((rows, top), -9, dtype=torch.int32, device="cuda"),
               top_logp=torch.full((rows, top), 9.0, device="cuda"))
    b.token_logprobs(h, logits, ids=ids, scale=scale, **got)
    return got


def check_logprobs(logits, ids, top, scale):
    """Against the oracle.  Terms 2^t are off by |t| 2^-24 + 2^-22, sums by 2^-24 an addition (a thread adds every
    512th vector at most), and what is reported by a few steps of its parts."""
    h = model("bf16")
    got = logprobs(h, logits, ids, top, scale)
    vocab = logits.shape[1]
    logp, entropy, top_id, top_logp = O.logprobs(f64(logits), scale, ids.cpu().numpy(), top)
    assert np.array_equal(got["top_id"].cpu().numpy(), top_id)
    spread = math.log(vocab) + 8
    base, step = (vocab / 512 + 64) * 2.0 ** -24 * spread, 8 * 2.0 ** -24
    inside(f64(got["logp"]), logp, base + step * np.abs(np.nan_to_num(logp, posinf=0, neginf=0)))
    inside(f64(got["top_logp"]), top_logp, base + step * np.abs(np.nan_to_num(top_logp, posinf=0, neginf=0)))
    inside(f64(got["entropy"]), entropy, 4 * base + step * spread)
    b.blend_device_status(h)
    return got


def random_logits(rows, vocab, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    room = torch.full((rows, vocab + pad), float("nan"), dtype=TORCH[dtype])
    x = 3 * torch.randn(rows, vocab, generator=g)
    x[:, torch.randint(0, vocab, (min(vocab, 6),), generator=g)] += 9
    room[:, :vocab] = x
    return room.cuda()[:, :vocab]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,top,n_ids,pad,scale", [
    (1, 1, 1, 1, 0, 1.0), (3, 2, 2, 2, 1, 1.0), (2, 37, 32, 1, 3, 0.5), (5, 300, 5, 3, 0, 2.0), (1, 1000, 0, 2, 0, 1.0),
    (7, 4097, 20, 1, 5, 0.7), (200, 1111, 3, 2, 0, 1.0), (1, 49152, 32, 4, 0, 1.0), (2, 32003, 1, 1, 0, 1.3),
    (400, 515, 8, 1, 2, 1.0), (1, 131075, 20, 1, 0, 1.0)])
def test_logprobs(rows, vocab, top, n_ids, pad, scale, dtype):
    x = random_logits(rows, vocab, dtype, vocab, pad)
    ids = torch.randint(-1, vocab, (rows, n_ids), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    check_logprobs(x, ids, top, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [96, 5000, 20011, 70001])
def test_logprobs_ties_masks_and_specials(vocab, dtype):
    inf, nan = float("inf"), float("nan")
    x = random_logits(16, vocab, dtype, 2)
    at = torch.arange(vocab, device="cuda")
    x[0] = 1.5                                  # all alike: the first tokens
    x[1] = -inf                                 # nothing allowed
    x[2, 3:] = -inf                             # fewer allowed than asked for
    x[3] = torch.where(at % 7 == 5, x[3], torch.full_like(x[3], -inf))
    x[4, 50] = nan
    x[5, 60], x[5, 61] = inf, inf
    x[6] = nan
    x[7] = (-at / 64.0).to(x.dtype)             # descending
    x[8] = (at / 64.0).to(x.dtype)              # ascending
    x[9] = torch.where(at % 2 == 0, 0.0, -0.0).to(x.dtype)
    x[10] = -torch.finfo(x.dtype).max / 4       # masks of a very low value
    x[10, 17] = 0
    x[11, :] = -3.0e4
    x[11, vocab - 1] = 3.0e4
    x[12] = torch.finfo(x.dtype).min            # nothing but masks of the lowest value
    x[13] = torch.finfo(x.dtype).min
    x[13, 30:33] = torch.tensor([1.0, 2.0, 2.0], device="cuda").to(x.dtype)
    x[14] = torch.finfo(x.dtype).max            # logits of the highest value
    x[14, 9:] = 0
    x[15] = torch.finfo(x.dtype).min / 3
    x[15, 40] = nan
    ids = torch.tensor([[0, 5, -1, vocab - 1]] * 16, dtype=torch.int32, device="cuda")
    check_logprobs(x, ids, 20, 1.0)


def test_logprobs_many_candidates_with_few_threads():
    """Rows made so that a handful of threads hold all of the largest logits, and more of them than are kept."""
    vocab = 120000
    for dtype, steps in (("bf16", (2048, 4096)), ("f32", (1024, 2048))):
        at = torch.arange(vocab, device="cuda")
        rows = [at.remainder(997).to(TORCH[dtype])]
        for step in steps:
            some = at % step < 40
            x = random_logits(1, vocab, dtype, 4)[0]
            rows.append(torch.where(some, torch.rand(vocab, device="cuda") + 100, x.float()).to(x.dtype))
            rows.append(torch.where(some, torch.full((vocab,), 100.0, device="cuda"), x.float()).to(x.dtype))
        x = torch.stack(rows).repeat(62, 1).contiguous()  # (one CTA a row)
        n = len(rows)
        got = logprobs(model("bf16"), x, torch.zeros(x.shape[0], 1, dtype=torch.int32, device="cuda"), 32, 1.0)
        for r in range(n):
            want = torch.sort(x[r].float(), descending=True, stable=True)[1][:32]
            assert torch.equal(got["top_id"][r].long(), want), (dtype, r)
            assert torch.equal(got["top_id"][r::n], got["top_id"][r].expand_as(got["top_id"][r::n]))


def test_logprobs_unaligned_rows_parts_left_out_and_capture():
    h = model("f32")
    flat = torch.randn(40000, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        for start in (1, 2, 3, 5):
            x = flat.to(dtype)[start:start + 3 * 4999].reshape(3, 4999)
            check_logprobs(x, torch.tensor([[4998], [0], [17]], dtype=torch.int32, device="cuda"), 7, 1.0)
    x = random_logits(6, 9000, "f32", 5)
    ids = torch.randint(0, 9000, (6, 2), dtype=torch.int32).cuda()
    full = logprobs(h, x, ids, 4, 1.0)
    ent, top = torch.zeros(6, device="cuda"), torch.zeros(6, 4, dtype=torch.int32, device="cuda")
    b.token_logprobs(h, x, entropy=ent)
    b.token_logprobs(h, x, top_id=top)
    assert torch.equal(ent, full["entropy"]) and torch.equal(top, full["top_id"])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    out = {k: torch.zeros_like(v) for k, v in full.items()}
    with torch.cuda.graph(graph, stream=side):
        b.token_logprobs(h, x, ids=ids, **out)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(out[k], full[k]) for k in out)
    x.neg_()
    graph.replay()
    full = logprobs(h, x, ids, 4, 1.0)
    assert all(torch.equal(out[k], full[k]) for k in out)


def test_logprobs_bad_ids_and_refusals():
    h = model("bf16")
    x = random_logits(2, 500, "f32", 6)
    ids = torch.tensor([[3, 500], [4, -5]], dtype=torch.int32, device="cuda")
    got = logprobs(h, x, ids, 2, 1.0)
    with pytest.raises(b.BlendError) as e:
        b.blend_device_status(h)
    assert e.value.code == b.EDEVICE
    assert math.isnan(got["logp"][0, 1]) and got["logp"][1, 1] == 0 and math.isfinite(got["logp"][0, 0])
    b.blend_device_status(h)
    lib, E, p = b.lib(), b.EINVAL, lambda t: t.data_ptr()
    out = {k: p(v) for k, v in got.items()}

    def raw(lg=p(x), ld=500, dt=b.F32, rows=2, vocab=500, scale=1.0, ids_=p(ids), n_ids=2, logp=out["logp"], top=2,
            top_id=out["top_id"], ent=out["entropy"], tl=out["top_logp"]):
        return lib.token_logprobs(h.ptr, lg, ld, dt, rows, vocab, scale, ids_, n_ids, logp, ent, top, top_id, tl, None)

    before = b.blend_launch_count()
    for i, bad in enumerate([dict(lg=None), dict(lg=p(x) + 2), dict(ld=499), dict(dt=5), dict(rows=-1), dict(vocab=0),
                             dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                             dict(ids_=None), dict(logp=None), dict(n_ids=-1), dict(top=33), dict(top=-1), dict(top_id=None),
                             dict(vocab=1, top=2), dict(ent=out["entropy"] + 1)]):
        assert raw(**bad) == E, i
    assert raw(rows=0) == b.OK and b.blend_launch_count() == before
    for bad in (lambda: b.token_logprobs(h, x.half()), lambda: b.token_logprobs(h, x, ids=ids),
                lambda: b.token_logprobs(h, x, ids=ids.long(), logp=got["logp"]),
                lambda: b.token_logprobs(h, x, entropy=got["entropy"][:1]),
                lambda: b.token_logprobs(h, x, top_logp=got["top_logp"]),
                lambda: b.token_logprobs(h, x.t(), entropy=got["entropy"])):
        with pytest.raises(ValueError):
            bad()


# ---------------------------------------------------------------- rotary positions
SCALINGS = {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=2.0),
            "bands": dict(factor=8.0, low=1.0, high=4.0, trained_len=8192),
            "yarn": dict(factor=16.0, low=1.0, high=32.0, trained_len=4096)}


def check_rope(got, x, rot, freqs, layout, dtype, magnitude=1.0):
    """An angle is off by 2^-25 of an eighth turn and 2^-33 of a turn, its sine and cosine by two steps, products and
    sums by one each: together below 2^-22 of the pair's magnitudes."""
    want = O.rope(f64(x), rot, freqs, layout, magnitude)
    n = 2 * len(freqs)
    size = np.abs(f64(x)[..., :n])
    pair = size[..., :n // 2] + size[..., n // 2:] if layout == "half" else size[..., 0::2] + size[..., 1::2]
    pair = np.concatenate([pair, pair], -1) if layout == "half" else np.repeat(pair, 2, -1)
    bound = np.zeros(want.shape)
    bound[..., :n] = abs(magnitude) * pair * 2.0 ** -22 * (1 + STEP[dtype]) + STEP[dtype] * np.abs(want[..., :n])
    inside(f64(got), want, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("hq,hkv,d,rot_dim,rows", [(4, 2, 128, 128, 9), (9, 3, 64, 32, 33), (40, 8, 128, 64, 1), (8, 8, 64, 64, 300),
                                                   (32, 1, 128, 16, 5), (4, 2, 128, 112, 1)])
def test_rope_rows(hq, hkv, d, rot_dim, rows, layout, scaling, dtype):
    h = model(dtype, hq, hkv, d)
    freqs = O.rope_freqs(5e5, rot_dim, scaling, **SCALINGS[scaling])
    magnitude = 1.25 if scaling == "yarn" else 1.0
    desc = b.rope_desc(5e5, rot_dim, layout, scaling, magnitude=magnitude, **SCALINGS[scaling])
    g = torch.Generator().manual_seed(rows)
    qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g).to(TORCH[dtype]).cuda()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    rot = np.random.default_rng(rows).integers(-(1 << 20), 1 << 20, rows)
    rot[0] = 0 if rows > 1 else 131071
    if rows > 2:
        rot[1], rot[2] = 1 << 24, -(1 << 24)
    room_q = torch.full((rows + 2, hq, d), 5.0, dtype=TORCH[dtype], device="cuda")
    room_k = torch.full((rows + 2, hkv, d), 5.0, dtype=TORCH[dtype], device="cuda")
    n = i32([max(1, rows - 1)])
    b.rope_rows(h, desc, k, room_k[:rows], i32(rot.tolist()), n, rows, q=q, q_out=room_q[:rows])
    m = int(n[0])
    assert bool((room_q[m:] == 5).all()) and bool((room_k[m:] == 5).all())
    check_rope(room_q[:m], q[:m], rot[:m], freqs, layout, dtype, magnitude)
    check_rope(room_k[:m], k[:m], rot[:m], freqs, layout, dtype, magnitude)
    if rows > 1 and magnitude == 1.0:
        assert torch.equal(room_q[0], q[0])
    # in place, both in one fused projection
    b.rope_rows(h, desc, k, k, i32(rot.tolist()), n, rows, q=q, q_out=q)
    assert torch.equal(q[:m], room_q[:m]) and torch.equal(k[:m], room_k[:m])
    b.blend_device_status(h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_rows_over_layers_matches_realign(dtype):
    """Cached keys of several layers: as rope_realign does for the plain half layout (whose table rounds cos and
    sin, so the two agree within a step), and with layers or rows interleaved."""
    h = handle(dtype, 4, 2, 128, max_pos=4096)
    L, rows = 3, 70
    k = torch.randn(L, rows, 2, 128).to(TORCH[dtype]).cuda()
    rot = np.random.default_rng(0).integers(-4000, 4000, rows)
    desc = b.rope_desc(1e4, 128)
    freqs = O.rope_freqs(1e4, 128)
    out, ref = torch.empty_like(k), torch.empty_like(k)
    b.rope_rows(h, desc, k, out, i32(rot.tolist()), i32([rows]), rows)
    b.rope_realign(h, k, ref, rows, i32(rot.tolist()), L, rows, rows)
    check_rope(out, k, rot, freqs, "half", dtype)
    assert torch.allclose(out.float(), ref.float(), rtol=2 * STEP[dtype], atol=1e-5)
    # [rows][layers] storage: layers lie within a row's stride
    woven = torch.full((rows, L, 2, 128), 5.0, dtype=TORCH[dtype], device="cuda")
    b.rope_rows(h, desc, k, woven.transpose(0, 1), i32(rot.tolist()), i32([rows]), rows)
    assert torch.equal(woven.transpose(0, 1), out)
    back = torch.empty_like(k)
    b.rope_rows(h, desc, woven.transpose(0, 1), back, i32((-rot).tolist()), i32([rows]), rows)
    # two roundings of the turned values, each within half a step of a pair's size
    size = torch.maximum(k[..., :64].float().abs(), k[..., 64:].float().abs()).repeat(1, 1, 1, 2)
    assert bool(((back.float() - k.float()).abs() <= 4 * STEP[dtype] * size + 1e-5).all())


def test_rope_rows_many_rows_and_capture():
    h = model("bf16", 32, 1, 128)
    rows = 5003
    k = torch.randn(2, rows, 1, 128).bfloat16().cuda()
    rot = torch.randint(-100000, 100000, (rows,), dtype=torch.int32).cuda()
    desc, n = b.rope_desc(1e6, 96, "pairs", "linear", factor=2.0), i32([rows])
    out, cap = torch.empty_like(k), torch.empty_like(k)
    b.rope_rows(h, desc, k, out, rot, n, rows)
    check_rope(out, k, rot.cpu().numpy(), O.rope_freqs(1e6, 96, "linear", 2.0), "pairs", "bf16")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        b.rope_rows(h, desc, k, cap, rot, n, rows)
    graph.replay()
    assert torch.equal(out, cap)
    n.fill_(7)
    cap.fill_(3)
    graph.replay()
    assert torch.equal(cap[:, :7], out[:, :7]) and bool((cap[:, 7:] == 3).all())


def test_rope_rows_checks_and_refusals():
    h = model("bf16", 4, 2, 128)
    desc = b.rope_desc(1e4, 128)
    k = torch.randn(4, 2, 128).bfloat16().cuda()
    out = torch.full_like(k, 5)
    b.rope_rows(h, desc, k, out, i32([1, (1 << 24) + 1, -(1 << 24) - 1, 2]), i32([4]), 4)
    with pytest.raises(b.BlendError) as e:
        b.blend_device_status(h)
    assert e.value.code == b.EDEVICE and bool((out[1:3] == 5).all()) and not bool((out[[0, 3]] == 5).any())
    out.fill_(5)
    b.rope_rows(h, desc, k, out, i32([1] * 4), i32([9]), 4)  # more than max_n: clamped and reported
    with pytest.raises(b.BlendError):
        b.blend_device_status(h)
    assert not bool((out == 5).all(-1).any())
    b.blend_device_status(h)
    lib, E, p = b.lib(), b.EINVAL, lambda t: t.data_ptr()
    rot, n = i32([0] * 4), i32([4])
    part = lambda **kw: b.RopeRows(**dict(dict(src=p(k), dst=p(out), src_row=256, src_layer=0, dst_row=256, dst_layer=0,
                                              heads=2, n_layers=1), **kw))

    def raw(rope=desc, parts=None, n_parts=1, max_n=4, rot_=p(rot), n_=p(n)):
        ps = parts or [part()]
        arr = (b.RopeRows * 2)(*ps)
        return lib.rope_rows(h.ptr, C.byref(rope) if rope else None, arr, n_parts, rot_, n_, max_n, None)

    D = b.rope_desc
    before = b.blend_launch_count()
    bad = [dict(rope=None), dict(rot_=None), dict(n_=None), dict(n_parts=0), dict(n_parts=3), dict(max_n=-1),
           dict(rope=D(1e4, 24)), dict(rope=D(1e4, 0)), dict(rope=D(1e4, 144)), dict(rope=D(1.0, 128)),
           dict(rope=D(float("nan"), 128)), dict(rope=D(1e4, 128, scaling="linear", factor=0.5)),
           dict(rope=D(1e4, 128, scaling="bands", factor=2.0, low=4.0, high=1.0, trained_len=10)),
           dict(rope=D(1e4, 128, scaling="yarn", factor=2.0, low=1.0, high=4.0)),
           dict(rope=D(1e4, 128, magnitude=float("inf"))),
           dict(parts=[part(src=None)]), dict(parts=[part(dst=p(out) + 8)]), dict(parts=[part(src_row=128)]),
           dict(parts=[part(dst_row=260)]), dict(parts=[part(heads=0)]), dict(parts=[part(n_layers=0)]),
           dict(parts=[part(n_layers=2, src_layer=100, dst_layer=1024)]), dict(parts=[part(dst=p(k) + 512)]),
           dict(parts=[part(n_layers=2, src_layer=256, dst_layer=256)]),
           dict(parts=[part(), part()], n_parts=2), dict(parts=[part(), part(src=p(out), dst=p(out))], n_parts=2)]
    for i, kw in enumerate(bad):
        assert raw(**kw) == E, (i, kw)
    assert raw(max_n=0) == b.OK and b.blend_launch_count() == before
    for f in (lambda: b.rope_rows(h, desc, k.float(), out, rot, n, 4), lambda: b.rope_rows(h, desc, k, out, rot, n, 5),
              lambda: b.rope_rows(h, desc, k, out, rot.long(), n, 4), lambda: b.rope_rows(h, desc, k, out, rot, n, 4, q=k),
              lambda: b.rope_rows(h, desc, k[:, :1], out, rot, n, 4), lambda: b.rope_rows(h, desc, k.cpu(), out, rot, n, 4)):
        with pytest.raises(ValueError):
            f()
