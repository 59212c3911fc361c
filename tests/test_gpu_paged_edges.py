"""Paged-cache calls at their edges: the reset after an error, totals and sizes at their limits, values and
queries of extreme size, and what masked tokens may hold."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from rag_kv_cache_rope_gb300 import binding as b
from pagedcase import attention_bound, f64, filled, handle, i32

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
    assert status(h) == b.OK
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    torch.cuda._sleep(1 << 30)  # about half a second on the default stream
    busy.record()
    with torch.cuda.stream(side):
        left.fill_(1)
    b.blend_wait_flag(h, zero, 10, stream=side)
    assert status(h, side) == b.ETIMEOUT and status(h, side) == b.OK
    b.paged_attention(h, c.pages, q, start, lens, 40, out, stream=side)
    assert status(h, side) == b.OK
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
