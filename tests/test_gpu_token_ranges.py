"""Token operators at the ends of the ranges that their documentation allows: logits, scales and masks far out, signs of
what is reported, gates far below 0, buffers of one row.  Bounds count roundings as in the tests of each operator."""
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as O
from rag_kv_cache_rope_gb300 import binding as b
from tests.pagedcase import TORCH, f64, i32
from tests.test_gpu_decode import Model, Step, V
from tests.test_gpu_tokens import check_logprobs, inside, linear_bounds, logprobs, model, random_logits, rows_of, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab", [(2, 70001), (1600, 5000), (3, 300)])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 20])
def test_logprobs_just_above_the_lowest_reference(rows, vocab, scale):
    """Rows whose largest logit, times log2(e), lies a little above -2^24, so that some threads find theirs below it and
    others not: all of them count.  (Both logits and scale are exact, so that z is an integer.)"""
    one = 1.0 / scale
    x = torch.empty(4, vocab, device="cuda")
    x[0] = -11629080.0
    x[0, vocab - 7] = -11629079.0
    x[1] = torch.arange(vocab, device="cuda") % 3 - 11629081.0
    for r, up in ((2, 40.0), (3, 170.0)):
        x[r] = torch.arange(vocab, device="cuda").remainder(200) - 11629250.0
        x[r, 5] += up
    ids = torch.tensor([[vocab - 7, 0, 5, vocab // 2]] * 4, dtype=torch.int32, device="cuda")
    if rows > 4:  # one CTA a row
        got = logprobs(model("bf16"), (x * one).repeat(rows // 4, 1), ids.repeat(rows // 4, 1), 9, scale)
        few = check_logprobs(x * one, ids, 9, scale)
        for k, v in few.items():
            assert torch.allclose(got[k].double(), v.repeat(rows // 4, *[1] * (v.dim() - 1)).double(), rtol=2.0 ** -20, atol=2.0 ** -16), k
        want = O.logprobs(f64(x * one), scale, ids.cpu().numpy(), 9)
        base = (vocab / 256 + 64) * 2.0 ** -24 * (math.log(vocab) + 8)
        inside(f64(got["logp"][:4]), want[0], base + 8 * 2.0 ** -24 * np.abs(want[0]))
        inside(f64(got["entropy"][:4]), want[1], 5 * base)
        assert np.array_equal(got["top_id"][:4].cpu().numpy(), want[2])
    else:
        check_logprobs(x * one, ids, 9, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_smallest_scale(dtype):
    """With a scale of 2^-64 all that is allowed is alike and what is not allowed still counts for nothing, nor does what
    lies beside a row that begins and ends within a vector; smaller scales are refused."""
    x = random_logits(3, 5001, dtype, 80, pad=2)
    x[0, 100:] = -math.inf
    x[1, ::2] = torch.finfo(x.dtype).min
    ids = torch.tensor([[0, 200], [1, 200], [5000, 7]], dtype=torch.int32, device="cuda")
    check_logprobs(x, ids, 5, 2.0 ** -64)
    out, before = torch.zeros(3, device="cuda"), b.blend_launch_count()
    for scale in (2.0 ** -65, 1e-24, 1e-30, 1e-44):
        with pytest.raises(b.BlendError) as e:
            b.token_logprobs(model("bf16"), x, entropy=out, scale=scale)
        assert e.value.code == b.EINVAL
    assert b.blend_launch_count() == before


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.5, 0.55, 2.0 ** -20, 1.0, 2.0 ** 20])
def test_logprobs_of_logits_at_both_ends_of_the_type(scale, dtype):
    """Logits further apart than the largest number: log p is a number where the scaled distance is one."""
    x = random_logits(3, 700, dtype, 81)
    top = 0.9 * torch.finfo(x.dtype).max
    x[0, 3], x[0, 4] = 0.97 * top, -0.97 * top
    x[1, 5:9] = torch.tensor([-top, top, top / 2, -top / 3], device="cuda").to(x.dtype)
    x[2] = -top
    x[2, 10], x[2, 11] = top / 4, -math.inf
    ids = torch.tensor([[3, 4, 0, 9], [5, 6, 7, 8], [0, 10, 11, 20]], dtype=torch.int32, device="cuda")
    got = logprobs(model("bf16"), x, ids, 5, scale)
    logp, entropy, top_id, top_logp = O.logprobs(f64(x), scale, ids.cpu().numpy(), 5)
    assert np.array_equal(got["top_id"].cpu().numpy(), top_id)
    # (a distance below -3.4e38 is -infinity in fp32; the distance, scale log2(e), their product and that with ln 2 round
    # once each, ln 2 by less)
    big = float(torch.finfo(torch.float32).max)
    assert (np.isinf(logp) | (np.abs(logp) < 0.999 * big) | (np.abs(logp) > 1.001 * big)).all()
    for g, w in ((got["logp"], logp), (got["top_logp"], top_logp)):
        w = np.where(w < -big, -np.inf, w)
        inside(f64(g), w, 2.0 ** -16 + 5 * 2.0 ** -24 * np.abs(np.where(np.isfinite(w), w, 0)))
    inside(f64(got["entropy"]), entropy, 2.0 ** -16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.7, 37.0])
@pytest.mark.parametrize("rows,vocab", [(2000, 501), (9, 20011)])
def test_logprobs_signs(rows, vocab, scale, dtype):
    """No log p above 0 and no entropy below it, where one token has all of the probability or nearly all; NaN stays."""
    x = (5 * torch.randn(rows, vocab, generator=torch.Generator().manual_seed(82))).to(TORCH[dtype]).cuda()
    alone = torch.arange(rows, device="cuda") % 3
    at = torch.arange(vocab, device="cuda") == 77
    x = torch.where((alone == 0)[:, None] & ~at, torch.full_like(x, -math.inf), x)
    x = torch.where((alone == 1)[:, None] & at, torch.full_like(x, 60.0), x)
    x[rows - 1, 5] = math.nan
    got = logprobs(model("bf16"), x, torch.full((rows, 1), 77, dtype=torch.int32, device="cuda"), 2, scale)
    for k in ("logp", "top_logp"):
        assert bool((got[k][:-1] <= 0).all()), k
    assert bool((got["entropy"][:-1] >= 0).all())
    assert all(bool(got[k][-1].isnan().all()) for k in ("logp", "top_logp", "entropy"))
    # what has all of the probability: 0 up to the rounding of its logit's multiple of log2(e) and of the sum
    bound = 2.0 ** -23 * (1 + scale * x[:, 77].float().abs() * 2.0 ** -20)
    one = alone[:-1] == 0
    assert bool((got["logp"][:-1, 0].abs() <= bound[:-1])[one].all()) and bool((got["entropy"][:-1] <= bound[:-1])[one].all())


@pytest.mark.parametrize("dtype,rows,n", [("f32", 5, 32), ("f32", 64, 96), ("bf16", 7, 32), ("bf16", 30, 128), ("bf16", 60, 160), ("bf16", 300, 128)])
def test_linear_swiglu_of_gates_far_below_zero(dtype, rows, n):
    """Gates and up values that are their inputs: silu(gate) * up stays right to a few steps of fp32."""
    h, k, group = model(dtype), 128, 32
    codes = torch.full((n, k), 8)
    gate = torch.arange(n) // 16 % 2 == 0
    codes[gate, 0], codes[~gate, 1] = 9, 9
    w4 = b.W4Ref(b.w4_layout(codes).cuda(), torch.ones(n, k // group, dtype=torch.bfloat16, device="cuda"), k, group)
    x = torch.zeros(rows, k, dtype=TORCH[dtype], device="cuda")
    x[:, 0] = torch.linspace(-85, 30, rows)
    x[:, 1] = torch.linspace(1, 2, rows)
    y = torch.empty(rows, n // 2, device="cuda")
    b.w4_linear(h, w4, x, y, epi="swiglu")
    want = (O.silu(f64(x[:, 0])) * f64(x[:, 1]))[:, None].repeat(n // 2, 1)
    # the exponential is within two steps of 2^-23 (its documented error), sum, quotient and product within half a step each
    inside(f64(y), want, 3.6 * 2.0 ** -23 * np.abs(want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,pad", [(1, 0), (1, 3), (2, 0), (5, 3)])
def test_rope_rows_in_place_in_a_fused_buffer_of_layers(rows, pad, dtype):
    """Queries and keys side by side in [layers][rows][heads][head dim], a single row of each layer among them, and layers
    that do not lie a whole number of rows apart."""
    h = model(dtype, 4, 2, 128)
    L, heads, d = 3, 8, 128
    step = rows * heads * d + pad * 16
    g = torch.Generator().manual_seed(83)
    flat = torch.randn(L * step, generator=g).to(TORCH[dtype]).cuda()
    buf = torch.as_strided(flat, (L, rows, heads, d), (step, heads * d, d, 1))
    first = buf.clone()
    rot = i32([1000 * i + 7 for i in range(rows)])
    rope = b.rope_desc(5e5, 64, "pairs")
    q, k = buf[:, :, :4], buf[:, :, 4:6]
    b.rope_rows(h, rope, k, k, rot, i32([rows]), rows, q=q, q_out=q)
    want = torch.empty_like(first)
    for i in range(L):
        part = first[i].contiguous()
        b.rope_rows(h, rope, part[:, 4:6], want[i, :, 4:6], rot, i32([rows]), rows, q=part[:, :4], q_out=want[i, :, :4])
    want[:, :, 6:] = first[:, :, 6:]
    assert torch.equal(buf, want) and not torch.equal(buf[:, :, :6], first[:, :, :6])
    # what does meet is refused still
    before = b.blend_launch_count()
    for bad in (buf[:, :, 3:5], buf[:, :, 5:7]):
        with pytest.raises(b.BlendError) as e:
            b.rope_rows(h, rope, k, bad, rot, i32([rows]), rows)
        assert e.value.code == b.EINVAL
    assert b.blend_launch_count() == before
    b.blend_device_status(h)


def test_rope_rows_keep_their_outputs_off_shifts_and_count():
    """Shifts and count inside an output's rows are refused; between its rows they are not touched."""
    h = model("bf16", 4, 2, 128)
    rope, rows, width = b.rope_desc(1e4, 128), 4, 2 * 128
    room = torch.full((rows, width + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    words = room.view(torch.int32).view(rows, -1)
    out = room[:, :width].view(rows, 2, 128)
    k = torch.randn(rows, 2, 128, generator=torch.Generator().manual_seed(84)).bfloat16().cuda()
    rot, n = i32([3, 4, 5, 6]), i32([rows])
    before = b.blend_launch_count()
    for bad in (dict(rot=words[0, 10:14]), dict(rot=words[0, 125:129]), dict(rot=words[1, 158:160].as_strided((4,), (1,))),
                dict(n=words[3, 127:128])):
        with pytest.raises(b.BlendError) as e:
            b.rope_rows(h, rope, k, out, bad.get("rot", rot), bad.get("n", n), rows)
        assert e.value.code == b.EINVAL and "rot or n" in str(e.value)
    assert b.blend_launch_count() == before and bool((room == 5).all())
    inside_gap, count = words[1, 130:134], words[2, 140:141]
    inside_gap.copy_(rot)
    count.copy_(n)
    b.rope_rows(h, rope, k, out, inside_gap, count, rows)
    want = torch.empty_like(k)
    b.rope_rows(h, rope, k, want, rot, n, rows)
    assert torch.equal(out, want) and torch.equal(inside_gap, rot) and torch.equal(count, n)
    b.blend_device_status(h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,top", [(16, 96, 20), (16, 5003, 20), (16, 70001, 32), (1600, 9001, 8)])
def test_logprobs_strict_masks(rows, vocab, top, dtype):
    """Fewer allowed tokens than alternatives, under masks of every kind: the allowed first, then the masked by value and
    index, NaN last."""
    low = float(torch.finfo(TORCH[dtype]).min)
    x = random_logits(16, vocab, dtype, 85)
    at = torch.arange(vocab, device="cuda")
    few = (at == 5) | (at == vocab // 2) | (at == vocab - 1)
    for r, mask in enumerate((-math.inf, low, -1e9, -3e4, -1.5e30, -1e30, low / 2)):
        x[r].masked_fill_(~few, mask)
    x[7] = torch.where(few, x[7].float(), torch.where(at % 2 == 0, low, -math.inf)).to(x.dtype)
    x[8] = torch.where(few, x[8].float(), torch.where(at % 500 == 7, -2e30, torch.where(at % 3 == 1, -math.inf, -3e30))).to(x.dtype)
    x[9] = -math.inf
    x[9, 0] = math.nan
    x[10] = math.nan
    x[10, vocab - 1], x[10, 3], x[10, 4] = 2.0, low, -math.inf
    x[11] = 0.0
    x[11, 40:43] = 1.0
    x[12] = torch.where(at % 64 == 3, torch.full_like(x[12], 4.0), torch.full_like(x[12], -math.inf))
    x[13] = torch.where(at < vocab // 3, x[13].float(), -math.inf).to(x.dtype)
    x[14] = low
    x[14, vocab - 2] = 0.0
    x[15] = (-1e30 * (1 + at % 90)).to(x.dtype)
    ids = torch.tensor([[5, vocab - 1, 3]] * 16, dtype=torch.int32, device="cuda")
    _, _, top_id, _ = O.logprobs(f64(x), 1.0, ids.cpu().numpy(), top)
    many = x.repeat(rows // 16, 1)
    got = logprobs(model("bf16"), many, ids.repeat(rows // 16, 1), top, 1.0)["top_id"].view(-1, 16, top)
    assert np.array_equal(got[0].cpu().numpy(), top_id)
    assert bool((got == got[0]).all())


def test_logprobs_strict_masks_cost_a_reading_more():
    """A grammar that allows three tokens: its rows are read twice, not over and over (three times the ordinary rows' time
    leaves room for noise; five and thirteen times it were measured with a reading for every alternative)."""
    h, rows, vocab, top = model("bf16"), 2047, 32003, 5
    x = random_logits(rows, vocab, "bf16", 86)
    out = dict(top_id=torch.empty(rows, top, dtype=torch.int32, device="cuda"), top_logp=torch.empty(rows, top, device="cuda"))
    few = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    few[[5, vocab // 2, vocab - 9]] = True

    def best(logits):
        times = []
        for _ in range(8):
            a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                b.token_logprobs(h, logits, **out)
            e.record()
            e.synchronize()
            times.append(a.elapsed_time(e))
        return min(times)

    plain = best(x)
    for mask in (-math.inf, -1e9, torch.finfo(x.dtype).min):
        assert best(x.masked_fill(~few, mask)) < 3 * plain, mask


@pytest.mark.parametrize("dtype,rows", [("bf16", 3), ("bf16", 20), ("bf16", 40), ("bf16", 130), ("f32", 3), ("f32", 20)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_inputs_at_the_ends_of_their_range(dtype, rows, group):
    """The largest inputs, whose products with the lowest code all add up, and the smallest that keep all bits."""
    h = model(dtype)
    n, k = 160, 520
    w4, values = weights(n, k, group, 87)
    w4.codes[3] = 0
    small = torch.full_like(w4.scale, 2.0 ** -30)
    x = torch.full((rows, k), 2.0 ** 123, dtype=TORCH[dtype], device="cuda")
    y = torch.empty(rows, n, device="cuda")
    big = b.W4Ref(w4.codes, small, k, group)
    b.w4_linear(h, big, x, y)
    codes = np.rint(values / np.repeat(w4.scale.double().cpu().numpy()[:, :-(-k // group)], group, 1)[:, :k])
    codes[3] = -8
    want, bound = linear_bounds(codes * 2.0 ** -30, f64(x), "f32", False)
    inside(f64(y), want, bound)
    assert f64(y)[0, 3] == -8.0 * k * 2.0 ** 93
    x = (rows_of(dtype, rows, k, 88).float() * 2.0 ** -108).to(TORCH[dtype])
    x = torch.where(x.abs() < 2.0 ** -110, torch.zeros_like(x), x)
    b.w4_linear(h, b.W4Ref(w4.codes, torch.ones_like(w4.scale), k, group), x, y)
    want, bound = linear_bounds(codes, f64(x), "f32", False)
    inside(f64(y), want, bound - 1e-30)  # (without what that allows beside numbers of usual size)


@pytest.mark.parametrize("rows,n,k", [(9, 128, 256), (30, 160, 512), (60, 200, 512), (200, 384, 512), (500, 5120, 4096)])
@pytest.mark.parametrize("group", [32, 128])
def test_linear_tiles_keep_nan_and_infinity_in_their_row(rows, n, k, group):
    """In the kernels of many rows too (whose outputs are 128 at least; the last case shares tiles between CTAs)."""
    h = model("bf16")
    w4 = b.W4Ref.empty(n, k, group)
    w4.codes.random_(0, 256, generator=torch.Generator("cuda").manual_seed(89))
    w4.scale.fill_(0.01)
    x = rows_of("bf16", rows, k, 90)
    clean, y = (torch.empty(rows, n, device="cuda") for _ in range(2))
    b.w4_linear(h, w4, x, clean)
    assert bool(clean.isfinite().all())
    bad = sorted({1, 2, rows // 2, rows - 1})
    x[bad[0], 7], x[bad[1], k - 1], x[bad[-2], 0], x[bad[-1], k // 2] = math.nan, math.inf, -math.inf, math.nan
    b.w4_linear(h, w4, x, y)
    keep = [r for r in range(rows) if r not in bad]
    assert torch.equal(y[keep], clean[keep]) and bool(y[bad[0]].isnan().all()) and not bool(y[bad].isfinite().any())
    # weights of a group that held an infinity: one output of every row
    x = rows_of("bf16", rows, k, 90)
    w4.scale[n - 3, 0] = math.nan
    b.w4_linear(h, w4, x, y)
    assert bool(y[:, n - 3].isnan().all())
    keep = [j for j in range(n) if j != n - 3]
    assert torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("rows", [9, 40, 100, 200])
def test_linear_tiles_outliers_with_weights_of_zero(rows):
    """One input far larger than the others whose weights are 0: exact zeros, so the others keep their bits."""
    h = model("bf16")
    n, k, group = 160, 512, 64
    w4, values = weights(n, k, group, 91)
    x = rows_of("bf16", rows, k, 92)
    x[:, 100] = 2.0 ** 60
    x[1] *= 2.0 ** -100
    codes = np.rint(values / np.repeat(w4.scale.double().cpu().numpy(), group, 1)).astype(np.int64) + 8
    codes[:, 100] = 8
    w4.codes.copy_(b.w4_layout(torch.from_numpy(codes)))
    values[:, 100] = 0
    y = torch.empty(rows, n, device="cuda")
    b.w4_linear(h, w4, x, y)
    xs = f64(x)
    xs[:, 100] = 0
    want, bound = linear_bounds(values, xs, "f32", False)
    inside(f64(y), want, bound)


@pytest.mark.parametrize("n_seq,group", [(3, 128), (20, 64)])
def test_generated_tokens_in_bf16_are_as_near_as_their_roundings(n_seq, group):
    """Some ten roundings a layer move their values by 2^-9 in the mean and add up like independent ones: over 2 layers the
    logits are off by 2^-9 sqrt(20) of their size in the mean, none by more than eight times that (80000 values of a
    normal distribution stay within five), and where the two highest are further apart than twice that, the token is the same."""
    m = Model("bf16", group, 1)
    st = Step(m, [(41 * s + 3) % 90 + 1 for s in range(n_seq)], 8, 2)
    st.tok.copy_(torch.arange(n_seq) * 13 % V)
    mean, clear = 2.0 ** -9 * math.sqrt(20), 0
    for _ in range(4):
        tok, pos = st.tok.cpu().numpy().copy(), st.pos.cpu().numpy().copy()
        st.run()
        want = st.oracle(tok, pos)
        size = np.sqrt((want ** 2).mean(-1, keepdims=True))
        off = np.abs(f64(st.logits) - want) / size
        assert np.sqrt((off ** 2).mean()) <= mean and off.max() <= 8 * mean, (float(np.sqrt((off ** 2).mean()) / mean), float(off.max() / mean))
        two = np.sort(want, -1)[:, -2:]
        sure = (two[:, 1] - two[:, 0]) / size[:, 0] > 16 * mean
        clear += int(sure.sum())
        assert np.array_equal(st.top[:, 0].cpu().numpy()[sure], want.argmax(1)[sure])
    assert clear > 0
    b.blend_device_status(m.h)
