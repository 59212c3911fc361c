"""What is measured of the operators behind a finished cache: products with 4-bit weights
(w4_linear) and the weights' packing (w4_pack, w4_unpack), log probabilities of tokens with
entropy and top alternatives (token_logprobs), and rotary positions of every layout and scaling
(rope_rows).

Every case is a dict of plain values; the inputs' values follow from the seed.  With `own` false
run() computes the operators in elementary torch operations, else it calls the framework.
"""
import math

import torch

own = False

SCALE_LOW, SCALE_HIGH = 0.003, 0.008  # scales of 4-bit weights: about those of N(0, 0.02) weights


# ---------------------------------------------------------------- cases
def _named(name, c):
    return dict(c, name=name) if name else c


def _linear(name, rows, n, k, group=128, dtype="bf16", out="bf16", epi="store"):
    return _named(name, dict(op="linear", rows=rows, n=n, k=k, group=group, dtype=dtype, out=out, epi=epi))


def _pack(name, n, k, group=128, dtype="bf16"):
    return _named(name, dict(op="pack", n=n, k=k, group=group, dtype=dtype))


def _logprobs(name, rows, vocab, dtype="f32", n_ids=1, top=0, scale=1.0, pad=0, keep=1):
    """pad: elements between the rows; keep: one token of `keep` is allowed, the others' logits are -inf."""
    return _named(name, dict(op="logprobs", rows=rows, vocab=vocab, dtype=dtype, n_ids=n_ids, top=top, scale=scale,
                             pad=pad, keep=keep))


def _rope(name, rows, layers=1, hq=32, hkv=8, d=128, rot=128, layout="half", scaling="none", dtype="bf16", far=32768,
          theta=5e5):
    """hq 0: keys only (cached rows that move by a shift of either sign); far: positions stay below it."""
    return _named(name, dict(op="rope", rows=rows, layers=layers, hq=hq, hkv=hkv, d=d, rot=rot, layout=layout,
                             scaling=scaling, dtype=dtype, far=far, theta=theta))


def listed():
    return [
        # a single user's decode step: the fused query, key and value projection, Llama-3-8B shape
        _linear("linear_1", 1, 6144, 4096),
        # a decode batch of eight through the gate and up projections, 14B shape
        _linear("linear_gate_up_8", 8, 27648, 5120, group=32, epi="swiglu"),
        # the head for four sequences: fp32 logits over the 14B shape's vocabulary
        _linear("linear_head_4", 4, 152064, 5120, group=64, out="f32"),
        # the query rows of four requests through the down projection, 14B shape
        _linear("linear_down_500", 500, 5120, 13824),
        # weights of one projection packed at start-up, Llama-3-8B shape, and read back
        _pack("pack_out", 4096, 4096),
        # the largest projection of the 14B shape, fine groups
        _pack("pack_gate_up", 27648, 5120, group=32),
        # the token just sampled, with twenty alternatives
        _logprobs("logprobs_1", 1, 152064, "bf16", 1, 20),
        # a decode batch under a temperature, five alternatives, a grammar that allows one token in seven
        _logprobs("logprobs_64", 64, 128256, "f32", 1, 5, 1.25, keep=7),
        # every token of a 2047-token answer scored, rows of an odd vocabulary
        _logprobs("logprobs_answer", 2047, 32003, "bf16", 1, 1),
        # the new token of a single sequence, Llama-3-8B heads, positions scaled by bands
        _rope("rope_1", 1, scaling="bands"),
        # a 16K-token context's cached keys moved to new places on eight layers, YaRN frequencies
        _rope("rope_cache_16k", 16064, 8, 0, 8, scaling="yarn", theta=1e6, far=131072),
        # prompt pieces of a model with interleaved pairs on half of the head
        _rope("rope_prompt", 4099, hq=40, layout="pairs", rot=64, scaling="linear", theta=1e4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear", "pack", "logprobs", "logprobs", "rope", "rope"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op in ("linear", "pack"):
        k, group = 8 * _log(rng, 8, 2048), rng.choice((32, 64, 128))
        n = _log(rng, 64, min(152064, (1 << (27 if op == "pack" else 29)) // k))
        if op == "pack":
            return _pack(None, n, k, group, dtype)
        kind = rng.choice(("one", "few", "few", "many"))
        rows = 1 if kind == "one" else rng.randint(2, 16) if kind == "few" else _log(rng, 17, 512)
        n = min(n, (1 << 35) // (k * rows))
        epi = rng.choice(("store", "swiglu"))
        if epi == "swiglu":
            n = max(32, n // 32 * 32)
        return _linear(None, rows, n, k, group, dtype, rng.choice(("bf16", "f32")), epi)
    if op == "logprobs":
        vocab = _log(rng, 1000, 262144)
        rows = _log(rng, 1, max(1, min(4096, (1 << 26) // vocab)))
        return _logprobs(None, rows, vocab, dtype, rng.randint(1, 8), rng.randint(0, 32), rng.choice((1.0, 0.7, 1.5)),
                         rng.choice((0, 0, 5, 64)), rng.choice((1, 1, 10)))
    hq, hkv, d = rng.choice(((32, 8, 128), (40, 8, 128), (9, 3, 64), (4, 2, 64), (8, 8, 128), (32, 1, 128), (0, 8, 128)))
    layers = rng.randint(1, 8) if hq == 0 else 1
    rows = _log(rng, 1, 16384 if hq == 0 else 8192)
    return _rope(None, rows, layers, hq, hkv, d, 16 * rng.randint(1, d // 16), rng.choice(("half", "pairs")),
                 rng.choice(("none", "linear", "base", "bands", "yarn")), dtype, _log(rng, 1000, 1 << 20),
                 rng.choice((1e4, 5e5, 1e6)))


def _esize(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    c = case
    if c["op"] == "linear":
        wide = c["n"] // 2 if c["epi"] == "swiglu" else c["n"]
        held = c["n"] * (c["k"] // 2 + 2 * -(-c["k"] // c["group"]))
        return {"bytes": held + c["rows"] * (c["k"] * _esize(c["dtype"]) + wide * _esize(c["out"])),
                "flops": 2 * c["rows"] * c["n"] * c["k"]}
    if c["op"] == "pack":
        held = c["n"] * (c["k"] // 2 + 2 * -(-c["k"] // c["group"]))
        # packed, and read back as values
        return {"bytes": 2 * held + 2 * c["n"] * c["k"] * _esize(c["dtype"]), "flops": 4 * c["n"] * c["k"]}
    if c["op"] == "logprobs":
        return {"bytes": c["rows"] * (c["vocab"] * _esize(c["dtype"]) + 8 * c["n_ids"] + 8 * c["top"] + 4),
                "flops": 6 * c["rows"] * c["vocab"]}
    values = c["rows"] * c["layers"] * (c["hq"] + c["hkv"])
    return {"bytes": 2 * values * c["d"] * _esize(c["dtype"]) + 4 * c["rows"], "flops": 3 * values * c["rot"]}


# ---------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    if c["op"] in ("linear", "pack"):
        n, k = c["n"], c["k"]
        chunks = -(-k // 128)
        codes = (n, chunks * 64)
        scales = (n, chunks * (128 // c["group"]))
        if c["op"] == "pack":
            s["w"] = normal(n, k, dtype=_dt(c["dtype"])) * 0.02
            s["codes"] = torch.empty(codes, dtype=torch.uint8, device="cuda")
            s["scale"] = torch.empty(scales, dtype=torch.bfloat16, device="cuda")
            s["out"] = torch.empty(n, k, dtype=_dt(c["dtype"]), device="cuda")
            return s
        s["codes"] = ints(0, 256, *codes).to(torch.uint8)
        x = torch.rand(scales, generator=g, device="cuda")
        s["scale"] = (SCALE_LOW + (SCALE_HIGH - SCALE_LOW) * x).to(torch.bfloat16)
        s["x"] = normal(c["rows"], k, dtype=_dt(c["dtype"]))
        wide = n // 2 if c["epi"] == "swiglu" else n
        s["y"] = torch.empty(c["rows"], wide, dtype=_dt(c["out"]), device="cuda")
        return s
    if c["op"] == "logprobs":
        rows, vocab = c["rows"], c["vocab"]
        room = torch.zeros(rows, vocab + c["pad"], dtype=_dt(c["dtype"]), device="cuda")
        s["logits"] = room[:, :vocab]
        s["logits"].copy_(2.5 * normal(rows, vocab))
        # a few likely tokens in each row
        at = ints(0, vocab // 8, rows, 8) + vocab // 8 * torch.arange(8, device="cuda")
        s["logits"].scatter_add_(1, at, (10 * torch.rand(rows, 8, generator=g, device="cuda")).to(_dt(c["dtype"])))
        ids = ints(0, vocab, rows, c["n_ids"])
        if c["keep"] > 1:
            allowed = torch.arange(vocab, device="cuda") % c["keep"] == 0
            s["logits"].masked_fill_(~allowed[None], -torch.inf)
            ids = ids // c["keep"] * c["keep"]
        s["ids"] = ids.to(torch.int32)
        s["logp"] = torch.empty(rows, c["n_ids"], device="cuda")
        s["entropy"] = torch.empty(rows, device="cuda")
        s["top_id"] = torch.empty(rows, c["top"], dtype=torch.int32, device="cuda")
        s["top_logp"] = torch.empty(rows, c["top"], device="cuda")
        return s
    rows, hq, hkv, d = c["rows"], c["hq"], c["hkv"], c["d"]
    dt = _dt(c["dtype"])
    s["n"] = torch.tensor([rows], dtype=torch.int32, device="cuda")
    if hq:
        # the rows of a fused projection: q heads, k heads, v heads
        qkv = normal(rows, hq + 2 * hkv, d, dtype=dt)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["q_out"] = torch.empty(rows, hq, d, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(rows, hkv, d, dtype=dt, device="cuda")
        s["rot"] = ints(0, c["far"], rows).to(torch.int32)
    else:
        s["k"] = normal(c["layers"], rows, hkv, d, dtype=dt)
        s["k_out"] = torch.empty_like(s["k"])
        # chunks of 512 tokens move together, forward or back
        shift = ints(1 - c["far"], c["far"], -(-rows // 512))
        s["rot"] = shift.repeat_interleave(512)[:rows].to(torch.int32).contiguous()
    return s


# ---------------------------------------------------------------- plain form
def _unpacked(codes, k):
    """fp32 values -8..7 [n][k] of packed rows.  16 words of 32 bits hold 128 inputs: word 4 t + w the inputs
    32 w + 8 t .. + 7, input e of them at bit 4 (e / 2) + 16 (e % 2)."""
    n = codes.shape[0]
    b = codes.reshape(n, -1, 4, 4, 4)  # chunk, t, w, byte
    both = torch.stack([b & 15, b >> 4], dim=-1)  # a byte's two nibbles
    both = both.reshape(n, -1, 4, 4, 2, 4)  # chunk, t, w, half of the word, position in it
    both = both.permute(0, 1, 3, 2, 5, 4)  # chunk, w, t, position, half
    return both.reshape(n, -1)[:, :k].float() - 8.0


def _weights(s):
    c = s["case"]
    w = _unpacked(s["codes"], c["k"])
    return w * s["scale"].float().repeat_interleave(c["group"], dim=1)[:, :c["k"]]


def _linear_plain(s):
    c = s["case"]
    y = torch.matmul(s["x"].float(), _weights(s).T)
    if c["epi"] == "swiglu":
        y = y.reshape(y.shape[0], -1, 2, 16)
        gate, up = y[:, :, 0], y[:, :, 1]
        y = (gate / (1.0 + torch.exp(-gate)) * up).reshape(y.shape[0], -1)
    return y.to(s["y"].dtype)


def _pack_plain(s):
    c = s["case"]
    n, k, group = c["n"], c["k"], c["group"]
    w = torch.nn.functional.pad(s["w"].float(), (0, -k % 128)).reshape(n, -1, group)
    scale = (w.abs().amax(-1) / 7.0).to(torch.bfloat16)
    sc = scale.double()[..., None]
    code = torch.where(sc > 0, torch.round(w.double() / sc).clamp(-7, 7), torch.zeros_like(sc)).float()
    u = (code + 8.0).to(torch.uint8).reshape(n, -1, 4, 4, 4, 2)  # chunk, w, t, position, half
    u = u.permute(0, 1, 3, 2, 5, 4).reshape(n, -1, 2)  # chunk, t, w, half, position
    s["codes"].copy_((u[..., 0] | (u[..., 1] << 4)).reshape(n, -1))
    s["scale"].copy_(scale.reshape(n, -1))
    return _weights(s).to(s["out"].dtype)


def _logprobs_plain(s):
    c = s["case"]
    x = s["logits"].float() * c["scale"]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    d = torch.where(e > 0, x - lse, torch.zeros_like(x))
    entropy = -(e / total * d).sum(1)
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :c["top"]]
    return {"logp": torch.gather(x, 1, s["ids"].long()) - lse, "entropy": entropy, "top_id": order.to(torch.int32),
            "top_logp": torch.gather(x, 1, order) - lse}


# what each scaling is drawn with: a model trained on 8192 positions
LINEAR, BASE, FACTOR, TRAINED, BANDS, RAMP = 4.0, 2.0, 8.0, 8192, (1.0, 4.0), (1.0, 32.0)


def _attention_factor(c):
    """YaRN's factor on cos and sin; cached keys carry it already."""
    return 0.1 * math.log(FACTOR) + 1.0 if c["scaling"] == "yarn" and c["hq"] else 1.0


def _frequencies(c):
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    theta, rot = c["theta"], c["rot"]
    if c["scaling"] == "base":
        theta = theta * BASE ** (rot / (rot - 2))
    f = torch.pow(torch.tensor(theta, dtype=torch.float64, device="cuda"), -2.0 * i / rot)
    if c["scaling"] == "linear":
        return f / LINEAR
    if c["scaling"] == "bands":
        low, high = BANDS
        turns = TRAINED * f / (2 * math.pi)  # over the trained length
        mix = ((turns - low) / (high - low)).clamp(0, 1)
        return f * (mix + (1 - mix) / FACTOR)
    if c["scaling"] == "yarn":
        slow, fast = RAMP
        at = [rot * math.log(TRAINED / (2 * math.pi * b)) / (2 * math.log(theta)) for b in (fast, slow)]
        low, high = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (ramp / FACTOR + (1 - ramp))
    return f


def _turned(c, x, rot):
    """x [..][rows][heads][d] of rows rotated by rot positions."""
    angle = rot.double()[:, None] * _frequencies(c)
    m = _attention_factor(c)
    cos, sin = (m * angle.cos()).float()[:, None], (m * angle.sin()).float()[:, None]
    n = c["rot"]
    head, rest = x[..., :n].float(), x[..., n:]
    if c["layout"] == "half":
        a, b = head[..., :n // 2], head[..., n // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).reshape(head.shape)
    return torch.cat([y.to(x.dtype), rest], dim=-1)


def _rope_plain(s):
    c = s["case"]
    got = {"k": _turned(c, s["k"], s["rot"])}
    if c["hq"]:
        got["q"] = _turned(c, s["q"], s["rot"])
    return got


# ---------------------------------------------------------------- the framework's calls
_handles = {}


def _handle(dtype, hq, hkv, d):
    """One handle per model, kept as a program keeps it."""
    from rag_kv_cache_rope_gb300 import binding as b
    key = (dtype, hq, hkv, d)
    if key not in _handles:
        dt = _dt(dtype)
        qd, kvd = hq * d, hkv * d

        def zeros(*shape):
            return torch.zeros(*shape, dtype=dt, device="cuda")

        w = {"embed": zeros(16, 16), "attn_norm": zeros(1, 16), "w_qkv": zeros(1, qd + 2 * kvd, 16),
             "w_o": zeros(1, 16, qd), "mlp_norm": zeros(1, 16), "w_gu": zeros(1, 32, 16), "w_down": zeros(1, 16, 16),
             "final_norm": zeros(16)}
        cfg = b.ModelCfg(1, 16, hq, hkv, d, 16, 16, b.F32 if dtype == "f32" else b.BF16, 1e4, 1e-6, 16)
        _handles[key] = b.blend_init(cfg, w, b.Limits(1, 1, 1, 1))
    return _handles[key]


def _rope_desc(b, c):
    kw = {}
    if c["scaling"] == "linear":
        kw = dict(factor=LINEAR)
    elif c["scaling"] == "base":
        kw = dict(factor=BASE)
    elif c["scaling"] == "bands":
        kw = dict(factor=FACTOR, low=BANDS[0], high=BANDS[1], trained_len=TRAINED)
    elif c["scaling"] == "yarn":
        kw = dict(factor=FACTOR, low=RAMP[0], high=RAMP[1], trained_len=TRAINED, magnitude=_attention_factor(c))
    return b.rope_desc(c["theta"], c["rot"], layout=c["layout"], scaling=c["scaling"], **kw)


def _run_own(s):
    from rag_kv_cache_rope_gb300 import binding as b
    c = s["case"]
    if c["op"] in ("linear", "pack"):
        h = _handle(c["dtype"], 32, 8, 128)
        if "w4" not in s:
            s["w4"] = b.W4Ref(s["codes"], s["scale"], c["k"], c["group"])
        if c["op"] == "linear":
            b.w4_linear(h, s["w4"], s["x"], s["y"], epi=c["epi"])
            return s["y"]
        b.w4_pack(h, s["w"], s["w4"])
        b.w4_unpack(h, s["w4"], s["out"])
        return s["out"]
    if c["op"] == "logprobs":
        got = {"logp": s["logp"], "entropy": s["entropy"], "top_id": s["top_id"], "top_logp": s["top_logp"]}
        b.token_logprobs(_handle("bf16", 32, 8, 128), s["logits"], ids=s["ids"], scale=c["scale"], **got)
        return got
    h = _handle(c["dtype"], c["hq"] or c["hkv"], c["hkv"], c["d"])
    if "rope" not in s:
        s["rope"] = _rope_desc(b, c)
    if not c["hq"]:
        b.rope_rows(h, s["rope"], s["k"], s["k_out"], s["rot"], s["n"], c["rows"])
        return {"k": s["k_out"]}
    b.rope_rows(h, s["rope"], s["k"], s["k_out"], s["rot"], s["n"], c["rows"], q=s["q"], q_out=s["q_out"])
    return {"k": s["k_out"], "q": s["q_out"]}


_PLAIN = {"linear": _linear_plain, "pack": _pack_plain, "logprobs": _logprobs_plain, "rope": _rope_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits
def _places(k):
    """For every input: its byte in a packed row and the shift of its nibble."""
    byte, shift = [], []
    for i in range(k):
        chunk, r = divmod(i, 128)
        word, r = divmod(r, 32)
        t, e = divmod(r, 8)
        bit = 4 * (e // 2) + 16 * (e % 2)
        byte.append(64 * chunk + 4 * (4 * t + word) + bit // 8)
        shift.append(bit % 8)
    return torch.tensor(byte, device="cuda"), torch.tensor(shift, device="cuda", dtype=torch.uint8)


def _linear64(c, s):
    byte, shift = _places(c["k"])
    group_of = torch.arange(c["k"], device="cuda") // c["group"]
    x, parts = s["x"].double(), []
    for r in range(0, c["n"], 8192):
        code = (s["codes"][r:r + 8192][:, byte] >> shift) & 15
        w = (code.double() - 8) * s["scale"][r:r + 8192].double()[:, group_of]
        parts.append(x @ w.T)
    y = torch.cat(parts, dim=1)
    if c["epi"] == "swiglu":
        unit = torch.arange(c["n"] // 2, device="cuda")
        at = unit // 16 * 32 + unit % 16
        y = y[:, at] * torch.sigmoid(y[:, at]) * y[:, at + 16]
    return y


def _pack64(c, s):
    out = torch.empty(c["n"], c["k"], dtype=torch.float64, device="cuda")
    for at in range(0, c["k"], c["group"]):
        w = s["w"][:, at:at + c["group"]].double()
        scale = (w.abs().max(dim=1, keepdim=True).values / 7).float().to(torch.bfloat16).double()
        step = torch.where(scale > 0, scale, torch.ones_like(scale))
        out[:, at:at + c["group"]] = torch.round(w / step) * scale
    return out


def _logprobs64(c, s):
    x = s["logits"].double() * c["scale"]
    lp = x - torch.logsumexp(x, dim=1, keepdim=True)
    p = lp.exp()
    entropy = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    # ranks by value, then by index
    left = s["logits"].double().clone()
    ids = torch.empty(c["rows"], c["top"], dtype=torch.int64, device="cuda")
    at = torch.arange(c["vocab"], device="cuda")
    for j in range(c["top"]):
        best = left.amax(1, keepdim=True)
        ids[:, j] = torch.where(left == best, at, c["vocab"]).amin(1)
        left.scatter_(1, ids[:, j:j + 1], -torch.inf)
    return {"logp": lp.gather(1, s["ids"].long()), "entropy": entropy, "top_id": ids.to(torch.int32),
            "top_logp": lp.gather(1, ids)}


def _rope64(c, s):
    rot, theta = c["rot"], c["theta"]
    if c["scaling"] == "base":
        theta *= BASE ** (rot / (rot - 2))
    freq = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if c["scaling"] == "linear":
            f /= LINEAR
        elif c["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > TRAINED / BANDS[0]:
                f /= FACTOR
            elif wave > TRAINED / BANDS[1]:
                mix = (TRAINED / wave - BANDS[0]) / (BANDS[1] - BANDS[0])
                f = (1 - mix) * f / FACTOR + mix * f
        elif c["scaling"] == "yarn":
            def dim(turns):
                return rot * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(theta))
            low, high = max(math.floor(dim(RAMP[1])), 0), min(math.ceil(dim(RAMP[0])), rot - 1)
            keep = 1 - min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f = f / FACTOR * (1 - keep) + f * keep
        freq.append(f)
    turn = torch.polar(torch.full((), _attention_factor(c), dtype=torch.float64, device="cuda"),
                       s["rot"].double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))

    def turned(x):
        y = x.double().clone()
        a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if c["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
        y[..., a], y[..., b] = z.real, z.imag
        return y

    got = {"k": turned(s["k"])}
    if c["hq"]:
        got["q"] = turned(s["q"])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _linear64, "pack": _pack64, "logprobs": _logprobs64, "rope": _rope64}[case["op"]](case, s)
