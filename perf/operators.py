"""What is measured of the paged-cache operators: appending K/V rows with their rotation
(paged_append), reading rows back (paged_gather), and attention with a sliding window and
sinks over pages in the model's type or in 4 bits (paged_attention).

Every case is a dict of plain values; lengths and row counts follow from it alone (_lens,
_rows), values and the order of the pages from the seed.  With `own` false run() computes
the operators in elementary torch operations in fp32, else it calls the framework.
"""
import math

import torch

own = False

THETA = 1e6


# ---------------------------------------------------------------- cases
def _case(name, op, fmt="model", dtype="bf16", hq=32, hkv=8, d=128, page=64, n_seq=1, length=1024, spread=0, rows=1,
          window=0, sink=0, with_q=False):
    """length: tokens of the longest sequence (rows of this call among them); spread: sequence s
    is shorter by (s * 193) % (spread + 1) tokens; rows: rows of this call per sequence at most."""
    c = dict(op=op, fmt=fmt, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, n_seq=n_seq, length=length, spread=spread,
             rows=rows, window=window, sink=sink, with_q=with_q)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of one sequence, Llama-3-8B heads: what a single user's decode step pays per layer
        _case("append_1", "append", length=700, with_q=True),
        # a decode step of 256 sequences into 4-bit pages, read back as the values held
        _case("append_int4_256", "append", fmt="int4", n_seq=256, length=2048, spread=1500, page=16),
        # a finished 16K-token cache (14B heads) moved into pages
        _case("append_16k", "append", hq=40, length=16064, rows=16064, page=128),
        # prompts of sixteen sequences into 4-bit pages, read back as the values held
        _case("append_int4_prompts", "append", fmt="int4", n_seq=16, length=4099, spread=1000, rows=4099, page=64),
        # a 16K-token context held in 4 bits brought back as a contiguous cache, keys realigned
        _case("gather_int4_16k", "gather", fmt="int4", hq=40, length=16064, rows=16064),
        # fp32 heads of the two-layer test model, a few short ragged sequences
        _case("gather_f32", "gather", dtype="f32", hq=4, hkv=2, d=64, page=32, n_seq=5, length=672, spread=333, rows=672),
        # the first decode step after a short context
        _case("attend_1", "attend", length=700),
        # a decode batch with a 4096-token window behind a 32-token shared prefix, Mistral-7B heads
        _case("attend_window_64", "attend", n_seq=64, length=8195, spread=5000, page=16, window=4096, sink=32),
        # one very long context, 14B heads
        _case("attend_128k", "attend", hq=40, length=131072, page=128),
        # pieces of four prompts over their window and sinks
        _case("attend_prompt", "attend", n_seq=4, length=8200, spread=1600, rows=2048, window=4096, sink=64),
        # a decode batch over a cache held in 4 bits
        _case("attend_int4_32", "attend", fmt="int4", n_seq=32, length=16384, spread=9000),
        # query pieces of eight requests (64 tokens each) over contexts held in 4 bits
        _case("attend_int4_query", "attend", fmt="int4", n_seq=8, length=8256, spread=3000, rows=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "append", "gather", "attend", "attend", "attend", "attend", "attend"))
    fmt = rng.choice(("model", "int4"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    hq, hkv, d = rng.choice(((32, 8, 128), (40, 8, 128), (9, 3, 64), (4, 2, 64), (8, 8, 128), (32, 1, 128)))
    page = rng.choice((16, 32, 64, 128))
    window = sink = 0
    if op == "attend":
        kind = rng.choice(("one", "one", "few", "piece"))
        if rng.random() < 0.5:
            window, sink = _log(rng, 1, 8192), rng.choice((0, 1, 4, 32, 100))
        n_seq = _log(rng, 1, 128)
        length = min(_log(rng, 1, 131072), (1 << (18 if dtype == "bf16" else 17)) // n_seq)
        rows = 1 if kind == "one" else min(length, rng.randint(2, 9))
        if kind == "piece":
            n_seq = min(n_seq, 4)
            length = min(length, 8192)
            rows = min(length, _log(rng, 10, 800 if dtype == "bf16" else 200))
    else:
        n_seq = _log(rng, 1, 256)
        length = _log(rng, 1, max(1, min(32768, (1 << 16) // n_seq)))
        rows = length if op == "gather" or rng.random() < 0.5 else 1
    spread = rng.randint(0, length - 1)
    return _case(None, op, fmt, dtype, hq, hkv, d, page, n_seq, length, spread, rows, window, sink,
                 op == "append" and rng.random() < 0.5)


def _lens(c):
    return [c["length"] - (s * 193) % (c["spread"] + 1) for s in range(c["n_seq"])]


def _rows(c):
    return [min(c["rows"], n) for n in _lens(c)]


def _esize(c):
    return 2 if c["dtype"] == "bf16" else 4


def _held(c):
    """Bytes a token's K or V row of one head takes in the pages."""
    return c["d"] * _esize(c) if c["fmt"] == "model" else c["d"] // 2 + c["d"] // 16


def work(case):
    c = case
    lens, rows = _lens(c), _rows(c)
    n, e, d, hq, hkv = sum(rows), _esize(c), c["d"], c["hq"], c["hkv"]
    if c["op"] == "append":
        b = n * 2 * hkv * (d * e + _held(c)) + (2 * n * hq * d * e if c["with_q"] else 0)
        if c["fmt"] == "int4":  # read back as values
            b += n * 2 * hkv * (d * e + _held(c))
        return {"bytes": b, "flops": 6 * n * d * hkv}
    if c["op"] == "gather":
        return {"bytes": n * 2 * hkv * (d * e + _held(c)), "flops": 6 * n * d * hkv}
    keys = pairs = 0
    for length, r in zip(lens, rows):
        first = length - r
        if c["window"] == 0:
            keys += length
            pairs += r * (first + 1) + r * (r - 1) // 2
        else:
            lo = max(0, first - c["window"] + 1)
            keys += min(c["sink"], lo) + length - lo
            for p in range(first, length):
                lo = max(0, p - c["window"] + 1)
                pairs += min(c["sink"], lo) + p + 1 - lo
    return {"bytes": keys * 2 * hkv * _held(c) + 2 * n * hq * d * e, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------- inputs
def _table(c, n_pages, g):
    """Pages of every sequence, in random order; -1 where a sequence has none."""
    lens, page = _lens(c), c["page"]
    cols = max((n + page - 1) // page for n in lens)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    lens_t = torch.tensor(lens, device="cuda")
    have = torch.arange(cols, device="cuda")[None, :] * page < lens_t[:, None]
    at = (have.reshape(-1).cumsum(0) - 1).reshape(have.shape).clamp(min=0)
    return torch.where(have, order[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()


def _int4_bytes(d):
    """(low, high): the dims that each byte of a K row and of a V row holds in its two nibbles."""
    k = torch.empty(d // 2, 2, dtype=torch.long)
    v = torch.empty(d // 2, 2, dtype=torch.long)
    for g in range(d // 32):
        for e in range(32):
            c, i = divmod(e, 8)
            bit = 4 * (i >> 1) + 16 * (i & 1)
            k[c * (d // 8) + 4 * g + bit // 8, bit % 8 // 4] = 32 * g + e
            r, i = divmod(e, 4)
            v[r * (d // 16) + 2 * g + i // 2, i % 2] = 32 * g + e
    return k.cuda(), v.cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    lens, rows, page, hq, hkv, d = _lens(c), _rows(c), c["page"], c["hq"], c["hkv"], c["d"]
    n = sum(rows)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    n_pages = sum((x + page - 1) // page for x in lens) + 3
    s = {"case": c, "table": _table(c, n_pages, g)}
    if c["fmt"] == "model":
        s["k"], s["v"] = normal(n_pages, hkv, page, d), normal(n_pages, hkv, page, d)
    else:
        def nibbles():
            return torch.randint(1, 16, (n_pages, hkv, page, d // 2), generator=g, device="cuda", dtype=torch.uint8)

        def scales():
            x = torch.rand(n_pages, hkv, page, d // 32, generator=g, device="cuda")
            return (0.1 + 0.25 * x).to(torch.bfloat16)

        s["k"], s["v"] = nibbles() * 16 + nibbles(), nibbles() * 16 + nibbles()
        s["k_scale"], s["v_scale"] = scales(), scales()
        s["k_bytes"], s["v_bytes"] = _int4_bytes(d)
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lens_t, rows_t = torch.tensor(lens, device="cuda"), torch.tensor(rows, device="cuda")
    seq = torch.repeat_interleave(torch.arange(c["n_seq"], device="cuda"), rows_t, output_size=n)
    nth = torch.arange(n, device="cuda") - s["q_start"][:-1].long()[seq]
    pos = (lens_t - rows_t)[seq] + nth
    s["seq"], s["pos"] = seq.to(torch.int32), pos.to(torch.int32)
    s["n"] = torch.tensor([n], dtype=torch.int32, device="cuda")
    if c["op"] == "attend":
        s["q"] = normal(n, hq, d)
        s["out"] = torch.empty(n, hq * d, dtype=dt, device="cuda")
        s["flat"] = seq * max(rows) + nth
        return s
    # rotation table of the model: cos and sin rounded to fp32 from fp64 angles
    inv = torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"),
                    -2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    ang = torch.arange(c["length"], device="cuda", dtype=torch.float64)[:, None] * inv
    s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    if c["op"] == "append":
        # the rows of a fused projection: q heads, k heads, v heads
        qkv = normal(n, hq + 2 * hkv, d)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty(n, hq, d, dtype=dt, device="cuda")
    else:
        # keys move by a whole chunk's shift, forward or back
        s["rot"] = (torch.randint(0, 2 * c["length"] - 1, (c["n_seq"],), generator=g, device="cuda")
                    - (c["length"] - 1)).to(torch.int32)[seq].contiguous()
    s["k_out"] = torch.empty(n, hkv, d, dtype=dt, device="cuda")
    s["v_out"] = torch.empty(n, hkv, d, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------- plain form
def _rotated(s, x, rot):
    """Pairs (i, i + d/2) of x [n][heads][d] (fp32) rotated by rot positions (of either sign)."""
    half = x.shape[-1] // 2
    at = rot.long().abs()
    c, sn = s["cos"][at][:, None], s["sin"][at][:, None]
    sn = torch.where(rot[:, None, None] < 0, -sn, sn)
    x1, x2 = x[..., :half], x[..., half:]
    return torch.cat([x1 * c - x2 * sn, x2 * c + x1 * sn], dim=-1)


def _quantised(x):
    """(codes -7..7, scale bf16) of each 32 dims of x [n][heads][d] (fp32)."""
    y = x.reshape(*x.shape[:-1], -1, 32)
    scale = (y.abs().amax(-1) / 7.0).to(torch.bfloat16)
    sf = scale.float()[..., None]
    code = torch.where(sf > 0, torch.round(y / sf).clamp(-7, 7), torch.zeros_like(y))
    return code.reshape(x.shape), scale


def _values(packed, scale, held):
    """fp32 values of packed rows [..., d/2] with scales [..., d/32]."""
    code = torch.empty(*packed.shape[:-1], packed.shape[-1] * 2, device=packed.device)
    code[..., held[:, 0]] = (packed & 15).float() - 8.0
    code[..., held[:, 1]] = (packed >> 4).float() - 8.0
    return (code.reshape(*scale.shape, 32) * scale.float()[..., None]).reshape(code.shape)


def _slots(s):
    c = s["case"]
    seq, pos = s["seq"].long(), s["pos"].long()
    return s["table"][seq, pos // c["page"]].long(), pos % c["page"]


def _append_plain(s):
    c = s["case"]
    dt = s["k_new"].dtype
    page, slot = _slots(s)
    k, v = _rotated(s, s["k_new"].float(), s["pos"]), s["v_new"].float()
    q = _rotated(s, s["q"].float(), s["pos"]).to(dt) if c["with_q"] else None
    if c["fmt"] == "model":
        s["k"][page, :, slot] = k.to(dt)
        s["v"][page, :, slot] = v.to(dt)
        return {"k": s["k"], "v": s["v"], "q": q}
    got = {"q": q}
    for name, x in (("k", k), ("v", v)):
        code, scale = _quantised(x)
        held = s[name + "_bytes"]
        u = (code + 8.0).to(torch.uint8)
        s[name][page, :, slot] = u[..., held[:, 0]] | (u[..., held[:, 1]] << 4)
        s[name + "_scale"][page, :, slot] = scale
        got[name] = (code.reshape(*scale.shape, 32) * scale.float()[..., None]).reshape(code.shape).to(dt)
    return got


def _gather_plain(s):
    dt = s["k_out"].dtype
    page, slot = _slots(s)
    k, v = s["k"][page, :, slot], s["v"][page, :, slot]
    if s["case"]["fmt"] == "int4":
        k = _values(k, s["k_scale"][page, :, slot], s["k_bytes"])
        v = _values(v, s["v_scale"][page, :, slot], s["v_bytes"])
    return {"k": _rotated(s, k.float(), s["rot"]).to(dt), "v": v.to(dt)}


def _sequences(s, name):
    """fp32 K or V of every sequence, [n_seq][hkv][tokens][d]."""
    t = s["table"].long().clamp(min=0)
    x = s[name][t]
    x = _values(x, s[name + "_scale"][t], s[name + "_bytes"]) if s["case"]["fmt"] == "int4" else x.float()
    x = x.permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _attend_plain(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    group, most = hq // hkv, max(_rows(c))
    start, lens = s["q_start"].long(), s["kv_len"].long()
    n_q = start[1:] - start[:-1]
    at = torch.arange(most, device="cuda")
    row = (start[:-1, None] + at).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().reshape(-1, most, hkv, group, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(-1, hkv, group * most, d)
    k, v = _sequences(s, "k"), _sequences(s, "v")
    x = torch.matmul(q, k.transpose(2, 3)).reshape(-1, hkv, group, most, k.shape[2]) / math.sqrt(d)
    p = ((lens - n_q)[:, None] + at)[:, :, None]
    j = torch.arange(k.shape[2], device="cuda")[None, None, :]
    sees = (j <= p) & (j < lens[:, None, None])
    if c["window"]:
        sees = sees & ((j > p - c["window"]) | (j < c["sink"]))
    sees = sees[:, None, None]
    x = x.masked_fill(~sees, -torch.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top == -torch.inf, torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(-1, hkv, group * most, k.shape[2]), v).reshape(-1, hkv, group, most, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 3, 1, 2, 4).reshape(-1, hq * d)[s["flat"]].to(s["q"].dtype)


# ---------------------------------------------------------------- the framework's calls
_handles = {}


def _handle(c):
    """One handle per model, kept as a program keeps it."""
    from rag_kv_cache_rope_gb300 import binding as b
    key = (c["dtype"], c["hq"], c["hkv"], c["d"])
    if key not in _handles:
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        qd, kvd = c["hq"] * c["d"], c["hkv"] * c["d"]

        def zeros(*shape):
            return torch.zeros(*shape, dtype=dt, device="cuda")

        w = {"embed": zeros(16, 16), "attn_norm": zeros(1, 16), "w_qkv": zeros(1, qd + 2 * kvd, 16),
             "w_o": zeros(1, 16, qd), "mlp_norm": zeros(1, 16), "w_gu": zeros(1, 32, 16), "w_down": zeros(1, 16, 16),
             "final_norm": zeros(16)}
        cfg = b.ModelCfg(1, 16, c["hq"], c["hkv"], c["d"], 16, 16, b.F32 if c["dtype"] == "f32" else b.BF16, THETA,
                         1e-6, 131072)
        _handles[key] = b.blend_init(cfg, w, b.Limits(1, 1, 1, 1))
    return _handles[key]


def _pages(s):
    from rag_kv_cache_rope_gb300 import binding as b
    if "pages" not in s:
        s["pages"] = b.PagesRef(s["k"], s["v"], s["table"], s.get("k_scale"), s.get("v_scale"))
    return s["pages"]


def _run_own(s):
    from rag_kv_cache_rope_gb300 import binding as b
    c = s["case"]
    h, pages = _handle(c), _pages(s)
    if c["op"] == "attend":
        b.paged_attention(h, pages, s["q"], s["q_start"], s["kv_len"], c["rows"], s["out"], window=c["window"],
                          n_sink=c["sink"])
        return s["out"]
    n = s["seq"].shape[0]
    if c["op"] == "gather":
        b.paged_gather(h, pages, s["seq"], s["pos"], s["n"], n, s["k_out"], s["v_out"], rot=s["rot"])
        return {"k": s["k_out"], "v": s["v_out"]}
    q = dict(q=s["q"], q_out=s["q_out"]) if c["with_q"] else {}
    b.paged_append(h, pages, s["k_new"], s["v_new"], s["seq"], s["pos"], s["n"], n, **q)
    got = {"k": s["k"], "v": s["v"], "q": s["q_out"] if c["with_q"] else None}
    if c["fmt"] == "int4":
        b.paged_gather(h, pages, s["seq"], s["pos"], s["n"], n, s["k_out"], s["v_out"])
        got["k"], got["v"] = s["k_out"], s["v_out"]
    return got


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _attend_plain(state) if op == "attend" else _gather_plain(state) if op == "gather" else _append_plain(state)


# ---------------------------------------------------------------- in 64 bits
def _turned64(x, rot):
    """x [n][heads][d] (fp64) as complex pairs, multiplied by exp(i rot theta^(-2 i / d))."""
    half = x.shape[-1] // 2
    freq = torch.tensor([THETA ** (-2.0 * i / (2 * half)) for i in range(half)], dtype=torch.float64, device="cuda")
    z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
    z = z * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), rot.double()[:, None, None] * freq)
    return torch.cat([z.real, z.imag], dim=-1)


def _held64(s, name, page, slot):
    """fp64 rows [n][heads][d] at (page, slot), dim by dim."""
    x = s[name][page, :, slot]
    if s["case"]["fmt"] == "model":
        return x.double()
    d, x = s["case"]["d"], x.long()
    scale = s[name + "_scale"][page, :, slot].double()
    got = torch.empty(*x.shape[:-1], d, dtype=torch.float64, device="cuda")
    for g in range(d // 32):
        for e in range(32):
            if name == "k":
                byte = (e // 8) * (d // 8) + 4 * g + 2 * (e & 1) + (e % 8) // 4
                shift = 4 * ((e % 8) // 2 % 2)
            else:
                byte, shift = (e // 4) * (d // 16) + 2 * g + (e % 4) // 2, 4 * (e % 2)
            got[..., 32 * g + e] = (((x[..., byte] >> shift) & 15) - 8).double() * scale[..., g]
    return got


def _rounded64(x):
    """The 4-bit form's values of fp64 rows: 32 dims share a bf16 scale of max / 7."""
    y = x.reshape(-1, 32)
    scale = (y.abs().max(dim=1).values / 7).float().to(torch.bfloat16).double()[:, None]
    return torch.where(scale > 0, torch.round(y / scale) * scale, torch.zeros_like(y)).reshape(x.shape)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    page, slot = _slots(s)
    if c["op"] == "gather":
        return {"k": _turned64(_held64(s, "k", page, slot), s["rot"]), "v": _held64(s, "v", page, slot)}
    if c["op"] == "append":
        k, v = _turned64(s["k_new"].double(), s["pos"]), s["v_new"].double()
        got = {"q": _turned64(s["q"].double(), s["pos"]) if c["with_q"] else None}
        for name, x in (("k", k), ("v", v)):
            if c["fmt"] == "int4":
                got[name] = _rounded64(x)
            else:
                got[name] = s[name].double()
                got[name][page, :, slot] = x
        return got
    group = c["hq"] // c["hkv"]
    outs = []
    at = 0
    for n, r, table in zip(_lens(c), _rows(c), s["table"]):
        tok = torch.arange(n, device="cuda")
        k = _held64(s, "k", table.long()[tok // c["page"]], tok % c["page"])
        v = _held64(s, "v", table.long()[tok // c["page"]], tok % c["page"])
        p = torch.arange(n - r, n, device="cuda")[:, None]
        hidden = tok[None] > p
        if c["window"]:
            hidden |= (tok[None] <= p - c["window"]) & (tok[None] >= c["sink"])
        o = torch.empty(r, c["hq"], c["d"], dtype=torch.float64, device="cuda")
        for head in range(c["hq"]):
            x = s["q"][at:at + r, head].double() @ k[:, head // group].T / c["d"] ** 0.5
            o[:, head] = torch.softmax(x.masked_fill(hidden, -torch.inf), dim=1) @ v[:, head // group]
        outs.append(o.reshape(r, -1))
        at += r
    return torch.cat(outs)
