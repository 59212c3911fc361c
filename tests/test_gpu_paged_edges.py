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
