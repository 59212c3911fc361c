"""Generated tokens behind a finished cache, with the operators as a program uses them together: 4-bit
projections, rotary positions scaled for long contexts, the paged cache, 4-bit head and log probabilities, step by
step and as a captured step, against a float64 run of the same model."""
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as O
from rag_kv_cache_rope_gb300 import binding as b
from tests.pagedcase import TORCH, f64, handle, i32

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, F, V, L, EPS, THETA = 256, 4, 2, 64, 384, 1000, 2, 1e-6, 5e5
BANDS = dict(factor=8.0, low=1.0, high=4.0, trained_len=256)
QD, KVD = HQ * D, HKV * D


class Model:
    def __init__(self, dtype, group, seed):
        g = torch.Generator().manual_seed(seed)
        dt = TORCH[dtype]
        self.dtype, self.h = dtype, handle(dtype, HQ, HKV, D, max_pos=16)
        self.emb = (torch.randn(V, H, generator=g)).to(dt).cuda()

        def packed(n, k):
            w = (torch.randn(n, k, generator=g) / math.sqrt(k)).to(dt).cuda()
            ref = b.W4Ref.empty(n, k, group)
            b.w4_pack(self.h, w, ref)
            codes, scales = O.w4_quantise(w.float().cpu().numpy(), group)
            return ref, O.w4_values(codes, scales, group)

        self.layers = [{k: packed(*s) for k, s in (("qkv", (QD + 2 * KVD, H)), ("o", (H, QD)), ("gu", (2 * F, H)), ("down", (H, F)))}
                       for _ in range(L)]
        self.head = packed(V, H)
        self.rope = b.rope_desc(THETA, D // 2, "pairs", "bands", **BANDS)
        self.freqs = O.rope_freqs(THETA, D // 2, "bands", **BANDS)


class Step:
    """One decode step of n_seq sequences over pages that hold their tokens so far; buffers of its own."""

    def __init__(self, m, lens, room, seed):
        dt, n = TORCH[m.dtype], len(lens)
        self.m, self.n = m, n
        cols = (max(lens) + room + 15) // 16
        table = torch.randperm(n * cols, generator=torch.Generator().manual_seed(seed)).reshape(n, cols).int().cuda()
        g = torch.Generator().manual_seed(seed + 1)
        self.pages, self.past = [], []
        for _ in range(L):
            k, v = (torch.randn(n * cols, HKV, 16, D, generator=g).to(dt).cuda() for _ in range(2))
            self.pages.append(b.PagesRef(k, v, table))
            rows = []
            for s in range(n):
                at = torch.arange(lens[s])
                page, slot = table[s].cpu().long()[at // 16], at % 16
                rows.append([f64(t.cpu()[page, :, slot]) for t in (k, v)])
            self.past.append(rows)
        self.tok = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.pos, self.kv_len = i32(lens), i32([x + 1 for x in lens])
        self.seq, self.q_start, self.count = i32(list(range(n))), i32(list(range(n + 1))), i32([n])
        self.zeros = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.qkv = torch.empty(n, HQ + 2 * HKV, D, dtype=dt, device="cuda")
        self.att, self.act = torch.empty(n, QD, dtype=dt, device="cuda"), torch.empty(n, F, dtype=dt, device="cuda")
        self.logits = torch.empty(n, V, device="cuda")
        self.logp, self.ent = torch.empty(n, 1, device="cuda"), torch.empty(n, device="cuda")
        self.top, self.top_logp = torch.empty(n, 5, dtype=torch.int32, device="cuda"), torch.empty(n, 5, device="cuda")

    def norm(self, x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).to(TORCH[self.m.dtype])

    def run(self):
        m, h, n = self.m, self.m.h, self.n
        x = m.emb[self.tok.long()].float()
        q, k, v = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:]
        for layer, pages in zip(m.layers, self.pages):
            b.w4_linear(h, layer["qkv"][0], self.norm(x), self.qkv.view(n, -1))
            b.rope_rows(h, m.rope, k, k, self.pos, self.count, n, q=q, q_out=q)
            b.paged_append(h, pages, k, v, self.seq, self.pos, self.count, n, rot=self.zeros)
            b.paged_attention(h, pages, q, self.q_start, self.kv_len, 1, self.att)
            b.w4_linear(h, layer["o"][0], self.att, x, epi="add")
            b.w4_linear(h, layer["gu"][0], self.norm(x), self.act, epi="swiglu")
            b.w4_linear(h, layer["down"][0], self.act, x, epi="add")
        b.w4_linear(h, m.head[0], self.norm(x), self.logits)
        b.token_logprobs(h, self.logits, ids=self.tok.view(n, 1), logp=self.logp, entropy=self.ent, top_id=self.top,
                         top_logp=self.top_logp)
        # the likeliest token is the next one
        self.tok.copy_(self.top[:, 0])
        self.pos += 1
        self.kv_len += 1

    def oracle(self, tok, pos):
        """Logits of every sequence in float64; the rows' keys and values join the past."""
        m = self.m
        out = []
        for s, t in enumerate(tok):
            x = f64(m.emb[int(t)])[None]
            nrm = lambda x: x / np.sqrt((x ** 2).mean(-1, keepdims=True) + EPS)
            for i, layer in enumerate(m.layers):
                qkv = (nrm(x) @ layer["qkv"][1].T).reshape(1, HQ + 2 * HKV, D)
                at = np.array([pos[s]])
                q, k = (O.rope(y, at, m.freqs, "pairs") for y in (qkv[:, :HQ], qkv[:, HQ:HQ + HKV]))
                past = self.past[i][s]
                past[0], past[1] = np.concatenate([past[0], k]), np.concatenate([past[1], qkv[:, HQ + HKV:]])
                o = np.empty((HQ, D))
                for head in range(HQ):
                    z = past[0][:, head // (HQ // HKV)] @ q[0, head] / math.sqrt(D)
                    p = np.exp(z - z.max())
                    o[head] = (p / p.sum()) @ past[1][:, head // (HQ // HKV)]
                x = x + o.reshape(1, -1) @ layer["o"][1].T
                x = x + O.w4_linear(layer["gu"][1], nrm(x), True) @ layer["down"][1].T
            out.append((nrm(x) @ m.head[1].T)[0])
        return np.array(out)


@pytest.mark.parametrize("dtype,n_seq,group", [("f32", 3, 32), ("bf16", 3, 128), ("bf16", 20, 64)])
def test_generated_tokens(dtype, n_seq, group):
    m = Model(dtype, group, 1)
    lens = [(37 * s + 5) % 90 + 1 for s in range(n_seq)]
    st = Step(m, lens, 8, 2)
    st.tok.copy_(torch.arange(n_seq) * 7 % V)
    # fp32: sums of up to 400 terms, a dozen of them one behind the other, each off by its terms' 2^-24 or so.  bf16:
    # each of some ten roundings a layer moves its values by 2^-9 in the mean, and the logits' deviations add up
    # like independent ones over 2 layers: 2^-9 sqrt(20) of their size, four times that at worst
    rel = 1e-4 if dtype == "f32" else 4 * 2.0 ** -9 * math.sqrt(20)
    for step in range(4):
        tok, pos = st.tok.cpu().numpy().copy(), st.pos.cpu().numpy().copy()
        st.run()
        want = st.oracle(tok, pos)
        size = np.sqrt((want ** 2).mean(-1, keepdims=True))
        got = f64(st.logits)
        assert (np.abs(got - want) <= 8 * rel * size).all() if dtype == "bf16" else (np.abs(got - want) <= rel * size).all()
        logp, ent, top, top_logp = O.logprobs(st.logits.cpu().numpy(), 1.0, tok[:, None], 5)
        assert np.array_equal(st.top.cpu().numpy(), top)
        for a, e in ((st.logp, logp), (st.ent, ent), (st.top_logp, top_logp)):
            assert np.abs(f64(a) - e).max() < 2e-5
        if dtype == "f32":
            assert np.array_equal(st.top[:, 0].cpu().numpy(), want.argmax(1))
        # (the oracle goes on with the token that was taken)
    b.blend_device_status(m.h)


@pytest.mark.parametrize("n_seq", [1, 12])
def test_captured_step_repeats_the_eager_ones(n_seq):
    m = Model("bf16", 128, 3)
    lens = [20 + s for s in range(n_seq)]
    eager, cap = Step(m, lens, 8, 4), Step(m, lens, 8, 4)
    first = (torch.arange(n_seq) * 11 % V).int().cuda()
    eager.tok.copy_(first)
    got = []
    for _ in range(5):
        eager.run()
        got.append((eager.tok.clone(), eager.logits.clone(), eager.ent.clone()))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    keep = [t.clone() for p in cap.pages for t in p.t[:2]] + [cap.pos.clone(), cap.kv_len.clone()]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cap.run()  # every kernel is loaded
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        cap.run()
    for t, old in zip([t for p in cap.pages for t in p.t[:2]] + [cap.pos, cap.kv_len], keep):
        t.copy_(old)
    cap.tok.copy_(first)
    for tok, logits, ent in got:
        graph.replay()
        assert torch.equal(cap.tok, tok) and torch.equal(cap.logits, logits) and torch.equal(cap.ent, ent)
    b.blend_device_status(m.h)


def test_streams_of_their_own():
    """Two handles' calls on two streams at once give what they give one after the other."""
    ms = [Model("bf16", 64, 5), Model("bf16", 64, 5)]
    steps = [Step(m, [30, 4], 8, 6) for m in ms]
    alone = Step(ms[0], [30, 4], 8, 6)
    alone.run()
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for st, s in zip(steps, streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                st.run()
    torch.cuda.synchronize()
    for _ in range(2):
        alone.run()
    for st in steps:
        assert torch.equal(st.logits, alone.logits) and torch.equal(st.tok, alone.tok)
