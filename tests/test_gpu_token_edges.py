"""Token operators in calls that the documentation allows and ordinary tests leave out: more row blocks than one grid
axis holds, rows that lie beside their results, no tensor cores, several host threads and streams, a first call
that is captured. Bounds as in the tests of each operator."""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import token_oracle as O
from rag_kv_cache_rope_gb300 import binding as b
from tests.pagedcase import TORCH, f64, handle, i32
from tests.test_gpu_tokens import inside, linear_bounds, logprobs, model, random_logits, rows_of, weights

pytestmark = pytest.mark.gpu


def test_linear_more_row_blocks_than_65535():
    """The longest fp32 rows leave shared memory for four of them: 2^18 rows are 65536 blocks."""
    h = model("f32")
    rows, k = 1 << 18, 32768
    w4, values = weights(3, k, 128, 31)
    x = torch.zeros(rows, k, device="cuda")
    at = [0, 5, 131071, rows - 5, rows - 1]
    x[at] = rows_of("f32", len(at), k, 32)
    y = torch.full((rows, 3), 7.0, device="cuda")
    b.w4_linear(h, w4, x, y)
    want, bound = linear_bounds(values, f64(x[at]), "f32", False)
    inside(f64(y[at]), want, bound)
    y[at] = 0
    assert not bool(y.any())
    b.blend_device_status(h)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_many_rows_without_tensor_cores(group):
    h = handle("bf16", 4, 2, 128)
    b.blend_set_tensor_cores(h, False)
    w4, values = weights(200, 712, group, 33)
    x = rows_of("bf16", 41, 712, 34)
    y = torch.empty(41, 200, device="cuda")
    b.w4_linear(h, w4, x, y)
    want, bound = linear_bounds(values, f64(x), "f32", False)
    inside(f64(y), want, bound)


@pytest.mark.parametrize("rows", [1, 7, 70])
def test_linear_codes_behind_the_inputs_do_not_count(rows):
    h = model("bf16")
    w4, values = weights(160, 136, 32, 35)
    x = rows_of("bf16", rows, 136, 36)
    y, z = (torch.empty(rows, 160, device="cuda") for _ in range(2))
    b.w4_linear(h, w4, x, y)
    for i in range(136, 256):  # inputs that the last chunk has room for
        byte, shift = O.w4_place(i)
        held = w4.codes[:, byte]
        w4.codes[:, byte] = (held & (15 << (4 - shift))) | (13 << shift)
    b.w4_linear(h, w4, x, z)
    assert torch.equal(y, z)
    want, bound = linear_bounds(values, f64(x), "f32", False)
    inside(f64(z), want, bound)


@pytest.mark.parametrize("rows", [5, 40])
def test_linear_results_beside_their_inputs(rows):
    """Inputs and results as columns of one buffer do not meet; one column in common is refused."""
    h = model("bf16")
    w4, values = weights(192, 256, 64, 37)
    room = torch.full((rows, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    room[:, :256] = rows_of("bf16", rows, 256, 38)
    b.w4_linear(h, w4, room[:, :256], room[:, 256:448])
    want, bound = linear_bounds(values, f64(room[:, :256]), "bf16", False)
    inside(f64(room[:, 256:448]), want, bound)
    assert bool((room[:, 448:] == 7.0).all())
    launches = b.blend_launch_count()
    for lo in (255, 0, 64):
        with pytest.raises(b.BlendError) as e:
            b.w4_linear(h, w4, room[:, :256], room[:, lo:lo + 192])
        assert e.value.code == b.EINVAL
    assert b.blend_launch_count() == launches


def test_linear_from_several_threads_and_streams():
    """Calls at once from four host threads, each on its own stream, give what one thread gives."""
    h = model("bf16")
    cases = []
    for i, (rows, n, k, group) in enumerate([(200, 1024, 2048, 128), (60, 1280, 4096, 64), (20, 2048, 1024, 32), (3, 4096, 4096, 128)]):
        w4, _ = weights(n, k, group, 40 + i)
        x = rows_of("bf16", rows, k, 50 + i)
        y = torch.empty(rows, n, device="cuda")
        b.w4_linear(h, w4, x, y)
        cases.append((w4, x, y, [torch.empty_like(y) for _ in range(8)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []

    def run(case):
        w4, x, _, outs, stream = case
        try:
            torch.cuda.set_device(0)
            for _ in range(5):
                for out in outs:
                    b.w4_linear(h, w4, x, out, stream=stream)
        except Exception as e:  # noqa: BLE001 - handed to the test's thread
            failed.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for _, _, y, outs, _ in cases:
        assert all(torch.equal(y, out) for out in outs)
    b.blend_device_status(h)


FIRST = """
import torch
from rag_kv_cache_rope_gb300 import binding as b
from tests.pagedcase import handle, i32
from tests.test_gpu_tokens import rows_of, weights
h = handle("bf16", 4, 2, 128)
calls = []
for rows, n, k, group in ((2, 512, 1024, 128), (30, 512, 1024, 64), (60, 512, 1024, 32), (200, 512, 1024, 128)):
    w4, _ = weights(n, k, group, rows)
    x, y = rows_of("bf16", rows, k, 1), torch.full((rows, n), -7.0, device="cuda")
    calls.append((lambda out, w4=w4, x=x: b.w4_linear(h, w4, x, out), y))
    back = torch.full((n, k), -7.0, dtype=torch.bfloat16, device="cuda")
    calls.append((lambda out, w4=w4: b.w4_unpack(h, w4, out), back))
logits = torch.randn(3, 70001, device="cuda")
calls.append((lambda out: b.token_logprobs(h, logits, top_id=out), torch.full((3, 7), -7, dtype=torch.int32, device="cuda")))
rope, rot, n = b.rope_desc(1e4, 128), i32([5, 6, 7]), i32([3])
k = rows_of("bf16", 3, 256, 2).view(3, 2, 128)
calls.append((lambda out: b.rope_rows(h, rope, k, out, rot, n, 3), torch.full((3, 2, 128), -7.0, dtype=torch.bfloat16, device="cuda")))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for call, out in calls:
        call(out)
graph.replay()
torch.cuda.synchronize()
for i, (call, out) in enumerate(calls):
    again = torch.zeros_like(out)
    call(again)
    assert torch.equal(out, again), i
b.blend_device_status(h)
print("all", len(calls))
"""


def test_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all 10" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


def test_logprobs_more_ids_than_threads_and_the_same_id_twice():
    h = model("bf16")
    rows, vocab, n_ids = 3, 5003, 700
    x = random_logits(rows, vocab, "f32", 60)
    ids = torch.randint(0, vocab, (rows, n_ids), generator=torch.Generator().manual_seed(61)).int().cuda()
    ids[:, 1], ids[:, 699], ids[1, 300] = ids[:, 0], ids[:, 0], -1
    logp = torch.full((rows, n_ids), 7.0, device="cuda")
    b.token_logprobs(h, x, ids=ids, logp=logp, scale=0.5)
    lp = torch.log_softmax(x.double() * 0.5, -1)
    want = torch.gather(lp, 1, ids.long().clamp_min(0)).cpu().numpy()
    want[1, 300] = 0.0
    # the logit's product and the difference round once each, the logarithm of the sum by less than 2^-18
    big = float((x.abs().max() * 0.5 + lp.abs().max()).item())
    inside(f64(logp), want, big * 2.0 ** -22 + 2.0 ** -18)
    assert torch.equal(logp[:, 0], logp[:, 1]) and torch.equal(logp[:, 0], logp[:, 699])


def test_logprobs_outputs_apart():
    h = model("bf16")
    x = random_logits(4, 600, "f32", 62)
    room = torch.zeros(64, dtype=torch.int32, device="cuda")
    ids = room[:8].view(4, 2)
    fl = room.view(torch.float32)
    before = b.blend_launch_count()
    for bad in (dict(ids=ids, logp=fl[4:12].view(4, 2)), dict(entropy=x.view(-1)[100:104]),
                dict(top_id=room[:8].view(4, 2), top_logp=fl[7:15].view(4, 2)), dict(ids=ids, logp=fl[8:16].view(4, 2), entropy=fl[15:19]),
                dict(top_id=x.view(torch.int32).view(-1)[2392:2400].view(4, 2))):
        with pytest.raises(b.BlendError) as e:
            b.token_logprobs(h, x, **bad)
        assert e.value.code == b.EINVAL
    assert b.blend_launch_count() == before
    b.token_logprobs(h, x, ids=ids, logp=fl[8:16].view(4, 2), entropy=fl[16:20], top_id=room[20:28].view(4, 2), top_logp=fl[28:36].view(4, 2))
    assert int(room[36:].abs().max()) == 0
    # logp over its ids is refused too: nothing that is read is written
    with pytest.raises(b.BlendError):
        b.token_logprobs(h, x, ids=ids, logp=fl[:8].view(4, 2))


def test_unknown_names_are_refused():
    h = model("bf16")
    w4, _ = weights(32, 128, 32, 63)
    x, y = rows_of("bf16", 1, 128, 64), torch.empty(1, 32, device="cuda")
    with pytest.raises(ValueError):
        b.w4_linear(h, w4, x, y, epi="gelu")
    for bad in (dict(layout="thirds"), dict(scaling="dynamic")):
        with pytest.raises(ValueError):
            b.rope_desc(1e4, 128, **bad)


def test_rope_rows_of_a_fused_projection_in_place_on_two_streams():
    """Two calls at once on halves of one buffer, queries and keys in place between values, some rows not turned."""
    h = model("bf16", 4, 2, 64)
    rows = 40
    qkv = rows_of("bf16", rows, 8 * 64, 65).view(rows, 8, 64)
    first = qkv.clone()
    rot = torch.arange(rows, dtype=torch.int32, device="cuda") * 1000
    rope = b.rope_desc(5e5, 32, "pairs")
    one = first.clone()
    b.rope_rows(h, rope, one[:, 4:6], one[:, 4:6], rot, i32([rows]), rows, q=one[:, :4], q_out=one[:, :4])
    n = i32([rows // 2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, part in zip(streams, (slice(0, rows // 2), slice(rows // 2, rows))):
        p, turn = qkv[part], rot[part]
        b.rope_rows(h, rope, p[:, 4:6], p[:, 4:6], turn, n, rows // 2, q=p[:, :4], q_out=p[:, :4], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(qkv, one) and torch.equal(qkv[:, 6:], first[:, 6:]) and torch.equal(qkv[0], first[0])
    assert not torch.equal(qkv[1:, :6], first[1:, :6])
    b.blend_device_status(h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,top", [(1, 1), (131, 8), (4000, 5), (16384, 8), (16385, 1), (32768, 8), (32003, 9)])
def test_logprobs_of_many_short_rows(vocab, top, dtype):
    """As many rows as fill the GPU with CTAs of half the threads, every row's mask and ranking its own."""
    h = model("bf16")
    rows, low = 1600, float(torch.finfo(TORCH[dtype]).min)
    x = random_logits(rows, vocab, dtype, 70 + vocab)
    x[3] = 0.0
    x[4] = low
    x[5] = float("-inf")
    x[6, vocab // 2:] = float("-inf")
    x[7, ::2] = low
    x[8, vocab // 3] = float("nan")
    x[9, vocab // 4] = float("inf")
    x[10] = float("nan")
    x[11, 1:] = float("-inf")
    x[12] = 7.5
    if vocab > 200:
        x[13] = torch.arange(vocab, device="cuda").to(x.dtype) * -0.01  # the largest with few threads
    ids = torch.randint(-1, vocab, (rows, 2), dtype=torch.int32, generator=torch.Generator().manual_seed(71)).cuda()
    got = logprobs(h, x, ids, top, 1.0)
    at = list(range(14)) + list(range(100, rows, 50)) + [rows - 1]
    logp, entropy, top_id, top_logp = O.logprobs(f64(x[at]), 1.0, ids[at].cpu().numpy(), top)
    assert np.array_equal(got["top_id"][at].cpu().numpy(), top_id)
    # terms 2^t are off by |t| 2^-24 + 2^-22, sums by 2^-24 an addition: a 128th of the row and the joins
    spread = math.log(vocab) + 8
    base, step = (vocab / 128 + 64) * 2.0 ** -24 * spread, 8 * 2.0 ** -24
    inside(f64(got["logp"][at]), logp, base + step * np.abs(np.nan_to_num(logp, posinf=0, neginf=0)))
    inside(f64(got["top_logp"][at]), top_logp, base + step * np.abs(np.nan_to_num(top_logp, posinf=0, neginf=0)))
    inside(f64(got["entropy"][at]), entropy, 4 * base + step * spread)
    lse = torch.logsumexp(x[14:].double(), -1, keepdim=True)
    want = torch.where(ids[14:] >= 0, torch.gather(x[14:].double(), 1, ids[14:].long().clamp_min(0)) - lse, 0.0)
    inside(f64(got["logp"][14:]), f64(want), base + step * np.abs(f64(want)))
    b.blend_device_status(h)


@pytest.mark.parametrize("rows,n,k,group,epi,out", [
    (500, 5120, 4096, 128, "store", "bf16"), (389, 5000, 4104, 32, "add", "f32"), (20, 20480, 4096, 64, "store", "f32"),
    (60, 20576, 4360, 128, "swiglu", "bf16"), (257, 9001, 5120, 64, "store", "f32"), (500, 5120, 13824, 128, "store", "f32")])
def test_linear_tiles_that_two_ctas_share(rows, n, k, group, epi, out):
    """Tiles that do not come out even over the SMs, so that CTAs take stretches of their line; against 64 bits on the GPU
    with the packed values, which are exact in fp32."""
    h = model("bf16")
    w4 = b.W4Ref.empty(n, k, group)
    w4.codes.random_(0, 256, generator=torch.Generator("cuda").manual_seed(90))
    w4.scale.copy_(torch.rand(w4.scale.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(91)) / 64 + 1 / 128)
    w = torch.empty(n, k, device="cuda")
    b.w4_unpack(model("f32"), w4, w)
    w = w.double()
    x = rows_of("bf16", rows, k, 92, 0.3)
    want, mag = x.double() @ w.T, x.double().abs() @ w.abs().T
    err = (3 * k / 16 + k / 32 + 64) * 2.0 ** -23 * mag
    if epi == "swiglu":
        (g, u), (eg, eu) = (t.view(rows, -1, 2, 16).unbind(2) for t in (want, err))
        s = g * torch.sigmoid(g)
        es = 1.1 * eg + (2 + g.abs()) * 2.0 ** -21 * s.abs()
        err, want = ((u.abs() * es + s.abs() * eu + es * eu).reshape(rows, -1), (s * u).reshape(rows, -1))
    wide = want.shape[1]
    base = torch.randn(rows, wide, device="cuda")
    room = torch.full((rows + 1, wide + 8), 7.0, dtype=TORCH[out], device="cuda")
    y = room[:rows, :wide]
    y.copy_(base)
    again = y.clone()
    b.w4_linear(h, w4, x, y, epi=epi)
    if epi == "add":
        want = want + base.double()
    step = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    bound = err * 1.01 + step * (want.abs() + err) + 1e-30 + (step * want.abs() if epi == "add" else 0)
    assert bool(((y.double() - want).abs() <= bound).all())
    assert bool((room[rows:] == 7.0).all()) and bool((room[:, wide:] == 7.0).all())
    b.w4_linear(h, w4, x, again, epi=epi)
    assert torch.equal(y, again)
    b.blend_device_status(h)
