"""Timed cases of the paged 4-bit cache: append, attention of single tokens, attention of chunks, and the decode step.

Keys and values live in a pool of pages, 4 bits a coordinate with one (step, offset) pair a vector:
x^ = m + s c, c in 0..15. A 16-token block of one head holds the 16 key code rows, the 16 value code rows,
16 key pairs and 16 value pairs (bf16 s in the low half, bf16 m in the high half of a 32-bit word);
byte j of a code row holds coordinates 2j (low nibble) and 2j + 1, and the 16-byte chunk p of token t's row holds
chunk p ^ x(t), x(t) = (t d / 256) mod (d / 32). The position rotation is applied in float32 and rounded to the
input's type, as a model applies it, before a key is quantized and before a query is used.

``own`` False: elementary torch operations in float32. ``own`` True: the framework's calls.
"""

import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, n_q=8, n_kv=8, d=128, dtype="f16", page=16, ctx_lo=0, ctx_hi=0, new_lo=1,
             new_hi=1, rot=128, interleaved=False, window=0)
    c.update(kw)
    return c


def listed():
    return [
        # the appends of one decode step of 16 sequences, two KV heads (a few KB: latency)
        _case("append_step", "append", batch=16, n_q=12, n_kv=2, ctx_lo=1000, ctx_hi=32767),
        # the first chunk of eight prompts of unlike lengths, one of them a single token, with half of each head rotated
        _case("append_ragged_d256", "append", batch=8, n_q=16, n_kv=8, d=256, dtype="bf16", new_lo=1, new_hi=4095,
              rot=128, interleaved=True),
        # one long prompt of a grouped-query layer
        _case("append_long", "append", batch=1, n_q=32, n_kv=8, ctx_lo=0, ctx_hi=0, new_lo=32768, new_hi=32768, page=64),
        # a single short conversation: the latency of one layer's attention
        _case("decode_short", "decode", batch=1, n_q=32, n_kv=8, ctx_lo=137, ctx_hi=137),
        # long contexts of a small model with two KV heads
        _case("decode_long", "decode", batch=16, n_q=12, n_kv=2, ctx_lo=32768, ctx_hi=32768, page=32),
        # a full batch at head_dim 256
        _case("decode_d256", "decode", batch=64, n_q=16, n_kv=8, d=256, dtype="bf16", ctx_lo=4096, ctx_hi=4096,
              rot=256, page=64),
        # a serving batch of unlike lengths, an idle slot among them, one query head per KV head, head_dim 64
        _case("decode_ragged_d64", "decode", batch=37, n_q=8, n_kv=8, d=64, dtype="bf16", ctx_lo=0, ctx_hi=19999,
              rot=64, page=16),
        # a whole prompt after its append
        _case("prefill_prompt", "prefill", batch=1, n_q=32, n_kv=8, new_lo=2048, new_hi=2048),
        # chunks of two prompts far into their contexts
        _case("prefill_chunk", "prefill", batch=2, n_q=12, n_kv=2, dtype="bf16", ctx_lo=12001, ctx_hi=16385, new_lo=512,
              new_hi=512, page=32),
        # a mixed batch at head_dim 256 with a sliding window: from one token to a few hundred
        _case("prefill_ragged_d256", "prefill", batch=5, n_q=16, n_kv=8, d=256, dtype="bf16", ctx_lo=0, ctx_hi=3000,
              new_lo=1, new_hi=900, rot=256, window=1024),
        # one decode step (append, then attention) of four sequences, five query heads per KV head
        _case("step_batch4", "step", batch=4, n_q=40, n_kv=8, ctx_lo=8191, ctx_hi=8191),
        # one decode step of a single sequence
        _case("step_single", "step", batch=1, n_q=12, n_kv=2, dtype="bf16", ctx_lo=500, ctx_hi=500, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128, 128, 256])
    n_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    c = dict(op=rng.choice(["append", "decode", "decode", "prefill", "step"]), n_q=n_kv * group, n_kv=n_kv, d=d,
             dtype=rng.choice(["f16", "bf16"]), page=rng.choice([16, 32, 64, 128]),
             rot=rng.choice([d, d, d // 2, 0]), interleaved=rng.random() < 0.3, window=0)
    tokens = 4_000_000 // (n_kv * d)           # token rows of one call, so that no draw outgrows the listed cases
    if c["op"] == "append":
        n = _log(rng, 1, 8 * tokens // 2)
        c["batch"] = min(n, _log(rng, 1, 64))
        c["new_hi"] = max(1, n // c["batch"])
        c["new_lo"] = rng.choice([c["new_hi"], 0, 1])
        c["ctx_lo"], c["ctx_hi"] = 0, _log(rng, 1, 4000)
    elif c["op"] == "prefill":
        c["new_hi"] = _log(rng, 1, 1500)
        c["batch"] = _log(rng, 1, max(1, 1500 // c["new_hi"]))
        c["new_lo"] = rng.choice([c["new_hi"], 0, 1])
        c["ctx_lo"], c["ctx_hi"] = 0, _log(rng, 1, 6000)
        c["window"] = rng.choice([0, 0, _log(rng, 1, 4000)])
    else:
        n = _log(rng, 64, 16 * tokens)
        c["batch"] = _log(rng, 1, min(128, n))
        c["ctx_hi"] = max(1, min(65000, n // c["batch"]))
        c["ctx_lo"] = rng.choice([c["ctx_hi"], 0, c["ctx_hi"] // 3])
        c["new_lo"] = c["new_hi"] = 1
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4000)])
    return c


def _spread(n, lo, hi, phase):
    """n whole numbers over [lo, hi], the first of them hi, in a fixed unordered sequence."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949 + phase * min(i, 1)) % 1.0)) for i in range(n)]


def _lengths(case):
    """(tokens held before the call, new tokens) of every sequence; a decode case attends over what is held."""
    ctx = _spread(case["batch"], case["ctx_lo"], case["ctx_hi"], 0.37)
    new = _spread(case["batch"], case["new_lo"], case["new_hi"], 0.11) if case["op"] != "decode" else [0] * case["batch"]
    if case["ctx_lo"] == 0 and case["batch"] > 2 and case["op"] == "decode":
        ctx[1] = 0                                          # an idle slot
    return ctx, new


# ------------------------------------------------------------------ the format
def _swizzle(d, device):
    t = torch.arange(16, device=device)[:, None]
    p = torch.arange(d // 32, device=device)[None, :]
    return p ^ ((t * d // 256) % (d // 32))                 # [16, d / 32]: the chunk held at place p of row t


def _bf16_down(x):
    u = x.contiguous().view(torch.int32)
    low = (u & 0xFFFF) != 0
    u = (u & -0x10000) + (low & (u < 0)).to(torch.int32) * 0x10000
    return u.view(torch.float32)


def _bf16_up(x):                                           # of values >= 0
    return ((x.contiguous().view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)


def _quantize(x):
    """(codes, s, m) of float32 vectors along the last axis (a divisor that is a tensor: each quotient is rounded once)."""
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m = _bf16_down(mn)
    r = mx - m
    s = torch.where(r > 0, _bf16_up(r / torch.full_like(r, 15.0)).clamp(min=torch.finfo(torch.float32).tiny), torch.zeros_like(r))
    c = torch.round((x - m) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15)
    return torch.where(s > 0, c, torch.zeros_like(c)), s, m


def _rotate(x, cos, sin, interleaved):
    """x [..., tokens, heads, d] float32 with cos, sin [..., tokens, rot / 2], rounded operation by operation."""
    h = cos.shape[-1]
    if h == 0:
        return x
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return y


# ------------------------------------------------------------------ state
def _fill_pages(pages, d, gen):
    """Random keys (a few channels far larger than the rest) and values, quantized into every page."""
    n_pages, n_kv, blocks, _ = pages.shape
    dev = pages.device
    chan = torch.ones(n_kv, 1, 1, d, device=dev)
    chan[..., torch.randperm(d, generator=gen, device=dev)[: d // 32]] = 6.0
    unit = torch.arange(16, device=dev)[:, None].expand(16, d // 32)
    sw = _swizzle(d, dev)
    step = max(1, 24_000_000 // (n_kv * blocks * 16 * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        parts, pairs = [], []
        for scale in (chan, 0.3):
            x = torch.randn(n, n_kv, blocks, 16, d, generator=gen, device=dev) * scale
            c, s, m = _quantize(x)
            c = c.to(torch.uint8)
            b = (c[..., 0::2] | (c[..., 1::2] << 4)).view(n, n_kv, blocks, 16, d // 32, 16)
            parts.append(b[..., unit, sw, :].reshape(n, n_kv, blocks, 8 * d))
            w = (m.view(torch.int32) & -0x10000) | ((s.view(torch.int32) >> 16) & 0xFFFF)
            pairs.append(w[..., 0].contiguous().view(torch.uint8).reshape(n, n_kv, blocks, 64))
        pages[i:i + n] = torch.cat(parts + pairs, -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    d, n_kv, n_q, page, dt = case["d"], case["n_kv"], case["n_q"], case["page"], _DT[case["dtype"]]
    ctx, new = _lengths(case)
    total = [a + b for a, b in zip(ctx, new)]
    per_row = max(1, -(-max(total) // page))
    need = [-(-t // page) for t in total]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    col = torch.arange(per_row, device=dev)[None, :]
    needs = torch.tensor(need, device=dev)[:, None]
    first = torch.cumsum(needs, 0) - needs
    table = torch.where(col < needs, perm[(first + col).clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    pages = torch.empty(n_pages, n_kv, page // 16, 16 * d + 128, dtype=torch.uint8, device=dev)
    _fill_pages(pages, d, gen)
    n_tok = case["batch"] if case["op"] == "decode" else sum(new)
    qkv = torch.randn(n_tok, (n_q + 2 * n_kv) * d, generator=gen, device=dev)
    qkv[:, :n_q * d] *= 1.0 / math.sqrt(1 + 35 / 32)       # scores of a standard deviation near 1.4
    qkv = qkv.to(dt)
    half = case["rot"] // 2
    ang = torch.arange(max(total) + 1, device=dev, dtype=torch.float64)[:, None] \
        * (500000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / max(1, half)))[None, :]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(
        case=case, d=d, n_kv=n_kv, n_q=n_q, page=page, op=case["op"], window=case["window"], dtype=dt,
        interleaved=case["interleaved"], pages=pages, table=table, max_ctx=max(total), batch=case["batch"],
        start=torch.tensor(ctx, dtype=torch.int32, device=dev), cu=torch.tensor(cu, dtype=torch.int32, device=dev),
        q=qkv[:, :n_q * d].view(n_tok, n_q, d), k=qkv[:, n_q * d:(n_q + n_kv) * d].view(n_tok, n_kv, d),
        v=qkv[:, (n_q + n_kv) * d:].view(n_tok, n_kv, d), n_tok=n_tok, max_new=max(new + [1]),
        rope=torch.cat([torch.cos(ang), torch.sin(ang)], 1).float().contiguous() if half else None,
        out=torch.empty(n_tok, n_q, d, dtype=dt, device=dev), lse=torch.empty(n_tok, n_q, device=dev),
        k_out=torch.empty(n_tok, n_kv, d, dtype=dt, device=dev), v_out=torch.empty(n_tok, n_kv, d, dtype=dt, device=dev))


# ------------------------------------------------------------------ the plain form
def _cos_sin(st, pos):
    if st["rope"] is None:
        e = torch.empty(*pos.shape, 0, device=pos.device)
        return e, e
    h = st["rope"].shape[1] // 2
    r = st["rope"][pos.clamp(min=0).long()]
    return r[..., :h], r[..., h:]


def _token_rows(st):
    """(sequence, position) of every token of the call."""
    i = torch.arange(st["n_tok"], device=st["cu"].device)
    row = torch.searchsorted(st["cu"][1:].long(), i, right=True)
    return row, st["start"][row] + (i - st["cu"][row])


def _unpack(raw, d):
    """Float32 keys and values [..., 16, d] of 16-token blocks [..., 16 d + 128]."""
    dev, sw = raw.device, _swizzle(d, raw.device)
    unit = torch.arange(16, device=dev)[:, None].expand(16, d // 32)
    got = []
    for side in (0, 1):
        b = raw[..., side * 8 * d:(side + 1) * 8 * d].reshape(*raw.shape[:-1], 16, d // 32, 16)[..., unit, sw, :]
        c = torch.stack([b & 15, b >> 4], -1).reshape(*raw.shape[:-1], 16, d).float()
        w = raw[..., 16 * d + side * 64:16 * d + side * 64 + 64].contiguous().view(torch.int32)
        s, m = (w << 16).view(torch.float32), (w & -0x10000).view(torch.float32)
        got.append(m.unsqueeze(-1) + s.unsqueeze(-1) * c)
    return got


def _rows_held(st):
    """Float32 keys and values [batch, n_kv, tokens, d] of every sequence's pages (tokens past its end: anything)."""
    g = st["pages"][st["table"].clamp(min=0).long()]        # [batch, pages, n_kv, blocks, bytes]
    g = g.transpose(1, 2).reshape(st["batch"], st["n_kv"], -1, 16 * st["d"] + 128)
    return [x.reshape(st["batch"], st["n_kv"], -1, st["d"]) for x in _unpack(g, st["d"])]


def _attend(st, q, pos, keys, vals):
    """q [batch, n, n_q, d] float32 at positions pos [batch, n] (below 0: none): float32 outputs and log-sum-exps."""
    bsz, n, n_q, d = q.shape
    g = n_q // st["n_kv"]
    q = q.view(bsz, n, st["n_kv"], g, d).permute(0, 2, 3, 1, 4).reshape(bsz, st["n_kv"], g * n, d)
    s = torch.matmul(q, keys.transpose(-1, -2)) / math.sqrt(d)
    t = torch.arange(keys.shape[2], device=q.device)
    ok = t <= pos[..., None]
    if st["window"]:
        ok &= t > pos[..., None] - st["window"]
    ok = ok[:, None, None].expand(-1, -1, g, -1, -1).reshape(bsz, 1, g * n, -1)
    s = s.masked_fill(~ok, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vals) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))[..., 0]
    back = lambda x, *e: x.view(bsz, st["n_kv"], g, n, *e).movedim(3, 1).reshape(bsz, n, n_q, *e)  # noqa: E731
    return back(out, d), back(lse)


def _stored(st):
    """What the new keys and values are stored as: float32 [n_tok, n_kv, d] each, and their places."""
    row, pos = _token_rows(st)
    cos, sin = _cos_sin(st, pos)
    k = _rotate(st["k"].float(), cos, sin, st["interleaved"]).to(st["dtype"]).float()
    got = []
    for x in (k, st["v"].float()):
        c, s, m = _quantize(x)
        got.append(m + s * c)
    return got, row, pos


def _plain(st):
    if st["op"] == "append":
        (k, v), _, _ = _stored(st)
        return dict(k=k.to(st["dtype"]), v=v.to(st["dtype"]))
    keys, vals = _rows_held(st)
    res = {}
    if st["op"] == "prefill":
        i = torch.arange(st["max_new"], device=keys.device)
        n = (st["cu"][1:] - st["cu"][:-1])[:, None]
        has = i[None, :] < n
        at = (st["cu"][:-1, None] + i[None, :]).clamp(max=st["n_tok"] - 1).long()
        pos = torch.where(has, st["start"][:, None] + i[None, :], -1)
        q = st["q"][at].float()
    else:
        if st["op"] == "step":
            (k, v), row, p = _stored(st)
            keys[row, :, p.long()], vals[row, :, p.long()] = k, v
            res = dict(k=k.to(st["dtype"]), v=v.to(st["dtype"]))
        pos = (st["start"] - (1 if st["op"] == "decode" else 0))[:, None]
        q = st["q"][:, None].float()
    cos, sin = _cos_sin(st, pos)
    q = _rotate(q, cos, sin, st["interleaved"]).to(st["dtype"]).float()
    out, lse = _attend(st, q, pos, keys, vals)
    if st["op"] == "prefill":
        out, lse = out[has], lse[has]
    else:
        out, lse = out[:, 0], lse[:, 0]
    return dict(out=out.to(st["dtype"]), lse=lse, **res)


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    from compressed_attention_head_b200 import sq

    if "cache" not in st:                                   # a program makes these once
        st["cache"] = sq.PagedKV4(st["pages"], st["table"], st["n_kv"], st["d"], st["page"])
        st["rot"] = sq.Rope(st["rope"], st["interleaved"]) if st["rope"] is not None else None
        if st["op"] == "prefill":
            n = sq.sq_kv4_attn_prefill_workspace(st["batch"], st["n_q"], st["n_kv"], st["d"], st["n_tok"])
        else:
            n = sq.sq_kv4_attn_workspace(st["batch"], st["n_q"], st["n_kv"], st["d"], st["max_ctx"])
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    cache, rot = st["cache"], st["rot"]
    if st["op"] == "append":
        sq.sq_kv4_append(cache, st["k"], st["v"], st["start"], st["cu"], rope=rot)
        sq.sq_kv4_read(cache, st["start"], st["cu"], st["k_out"], st["v_out"])
        return dict(k=st["k_out"], v=st["v_out"])
    if st["op"] == "decode":
        sq.sq_kv4_attn_decode(cache, st["start"], st["q"], 0.0, st["out"], st["max_ctx"], st["ws"], rope=rot,
                              window=st["window"], lse=st["lse"])
        return dict(out=st["out"], lse=st["lse"])
    if st["op"] == "prefill":
        sq.sq_kv4_attn_prefill(cache, st["start"], st["cu"], st["q"], 0.0, st["out"], st["ws"], rope=rot,
                               window=st["window"], lse=st["lse"])
        return dict(out=st["out"], lse=st["lse"])
    sq.sq_kv4_decode_step(cache, st["k"], st["v"], st["q"], st["start"], 0.0, st["out"], st["max_ctx"], st["ws"],
                          rope=rot, window=st["window"], lse=st["lse"])
    sq.sq_kv4_read(cache, st["start"], st["cu"], st["k_out"], st["v_out"])
    return dict(out=st["out"], lse=st["lse"], k=st["k_out"], v=st["v_out"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the least work
def _attended(case):
    """(query-key pairs of one head, keys read of one KV head) over all sequences."""
    ctx, new = _lengths(case)
    w = case["window"]
    pairs = held = 0
    for a, n in zip(ctx, new):
        if case["op"] == "decode":
            first, last = a - 1, a - 1
        elif case["op"] == "step":
            first, last = a, a
        else:
            first, last = a, a + n - 1
        if last < first or last < 0:
            continue
        lo = max(0, first - w + 1) if w else 0
        held += last + 1 - lo
        if w and first + 1 >= w:
            pairs += (last - first + 1) * w
        elif w and last + 1 > w:
            k = w - first - 1                               # positions whose prefix is still shorter than the window
            pairs += sum(range(first + 1, first + 1 + k)) + (last - first + 1 - k) * w
        else:
            pairs += (first + 1 + last + 1) * (last - first + 1) // 2
    return pairs, held


def work(case):
    d, n_kv, n_q = case["d"], case["n_kv"], case["n_q"]
    ctx, new = _lengths(case)
    n_tok = case["batch"] if case["op"] == "decode" else sum(new)
    rope = 4 * case["rot"] * n_tok
    b = f = 0
    if case["op"] in ("append", "step"):
        b += n_tok * n_kv * (2 * d * 2 + (d + 8) + 2 * d * 2) + rope     # inputs, what is stored, what is read back
        f += n_tok * n_kv * (3 * case["rot"] + 2 * 5 * d)
    if case["op"] != "append":
        pairs, held = _attended(case)
        b += held * n_kv * (d + 8) + n_tok * n_q * (2 * d * 2 + 4) + rope
        f += 4 * d * n_q * pairs
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_vec(x):
    """x^ of float64 vectors along the last axis: offset rounded down and step rounded up to 8 significant bits."""
    def grid(y, down):
        f, e = torch.frexp(y)
        z = f * 256.0
        return torch.ldexp((torch.floor(z) if down else torch.ceil(z)), e - 8)
    m = grid(x.amin(-1, keepdim=True), True)
    s = grid((x.amax(-1, keepdim=True) - m) / 15.0, False)
    c = torch.where(s > 0, torch.round((x - m) / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(s))
    return m + s * c


def _exact_rot(x, ang_row, interleaved):
    """One token's heads x [heads, d] (float64) turned by its table row, rounded to nothing."""
    h = ang_row.numel() // 2
    z = torch.complex(ang_row[:h], ang_row[h:])
    y = x.clone()
    if interleaved:
        w = torch.view_as_complex(x[:, :2 * h].reshape(x.shape[0], h, 2).contiguous()) * z
        y[:, :2 * h] = torch.view_as_real(w).reshape(x.shape[0], 2 * h)
    else:
        w = torch.complex(x[:, :h], x[:, h:2 * h]) * z
        y[:, :h], y[:, h:2 * h] = w.real, w.imag
    return y


def _exact_block(raw, d):
    """Keys and values [16 blocks, d] (float64) of the raw blocks [n, 16 d + 128] of one head, byte by byte."""
    n = raw.shape[0]
    i = torch.arange(d, device=raw.device)
    t = torch.arange(16, device=raw.device)[:, None]
    place = ((i // 32)[None, :] ^ ((t * d // 256) % (d // 32))) * 16 + ((i % 32) // 2)[None, :] + t * (d // 2)
    got = []
    for side in (0, 1):
        b = raw[:, side * 8 * d + place].long()
        c = (torch.where((i % 2 == 0), b & 15, b >> 4)).double()
        w = raw[:, 16 * d + 64 * side:16 * d + 64 * side + 64].reshape(n, 16, 4).long()
        bf = lambda lo, hi: (lo | (hi << 8)).to(torch.int32).bitwise_left_shift(16).view(torch.float32).double()  # noqa: E731
        got.append((bf(w[..., 2], w[..., 3])[..., None] + bf(w[..., 0], w[..., 1])[..., None] * c).reshape(n * 16, d))
    return got


def exact(case, seed):
    st = prepare(case, seed)
    d, n_q, n_kv, dt = st["d"], st["n_q"], st["n_kv"], st["dtype"]
    ctx, new = _lengths(case)
    group = n_q // n_kv
    turn = lambda x, p: _exact_rot(x.double(), st["rope"][p].double(), st["interleaved"]).to(dt).double() \
        if st["rope"] is not None else x.double()  # noqa: E731
    res = {}
    if st["op"] in ("append", "step"):
        if st["rope"] is not None:
            pos = torch.cat([torch.arange(a, a + n) for a, n in zip(ctx, new)]).to(st["rope"].device)
            r = st["rope"][pos].double()
            h = r.shape[1] // 2
            z = torch.complex(r[:, :h], r[:, h:])[:, None]
            k = st["k"].double()
            if st["interleaved"]:
                w = torch.view_as_real(torch.complex(k[..., 0:2 * h:2], k[..., 1:2 * h:2]) * z).flatten(-2)
            else:
                w = torch.complex(k[..., :h], k[..., h:2 * h]) * z
                w = torch.cat([w.real, w.imag], -1)
            k = torch.cat([w, k[..., 2 * h:]], -1).to(dt).double()
        else:
            k = st["k"].double()
        res = dict(k=_exact_vec(k), v=_exact_vec(st["v"].double()))
        if st["op"] == "append":
            return res
    out = torch.zeros(st["n_tok"], n_q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((st["n_tok"], n_q), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(st["batch"]):
        total = ctx[b] + new[b]
        first = ctx[b] if st["op"] != "decode" else ctx[b] - 1
        n = total - first if st["op"] != "decode" else 1
        if total == 0 or n == 0:
            at += 1 if st["op"] == "decode" else 0
            continue
        held = st["pages"][st["table"][b, :-(-total // st["page"])].long()]
        pos = torch.arange(first, first + n, device="cuda")
        q = torch.stack([turn(st["q"][at + j], first + j) for j in range(n)])
        for g in range(n_kv):
            keys, vals = _exact_block(held[:, g].reshape(-1, 16 * d + 128), d)
            keys, vals = keys[:total].clone(), vals[:total].clone()
            if st["op"] == "step":
                keys[-1], vals[-1] = res["k"][at, g], res["v"][at, g]
            t = torch.arange(total, device="cuda")[None, :]
            bad = t > pos[:, None]
            if st["window"]:
                bad |= t <= pos[:, None] - st["window"]
            for h in range(g * group, (g + 1) * group):
                s = (q[:, h] @ keys.T / math.sqrt(d)).masked_fill(bad, -math.inf)
                lse[at:at + n, h] = torch.logsumexp(s, -1)
                out[at:at + n, h] = torch.exp(s - lse[at:at + n, h, None]) @ vals
        at += n
    return dict(out=out, lse=lse, **res)
