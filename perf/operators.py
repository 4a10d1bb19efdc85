"""The attention block's operators around the 4-bit linear layers, as measured workloads.

Three operators of a 4-bit model's serving path:

  norm       residual addition + root-mean-square norm + 8-bit output with one
             scale per token, the input of the W4A8 and INT4-FP8 products
  append     rotary positions on queries and keys, keys and values quantised to
             4 bits and written into a paged cache
  attention  causal attention of new tokens over that cache: one token per
             sequence (decode), prompts, chunks of prompts, mixtures

`run` computes an operator in plain torch operations where `own` is false, and
calls the library where it is true.  Every step that rounds is part of the
operator's definition (act(v) rounds to the 16-bit type, f32(v) to binary32), so
codes, scales and packed words are equal whole numbers on both sides.

The cache is int32 [pages, kv_heads, page * (dim / 4 + 2)]; per page and head:
  K words  [page][dim / 8]         8 codes a word; nibble i of word j holds
                                   column 8 j + (0, 2, 4, 6, 1, 3, 5, 7)[i]
  V words  [page / 4][dim / 8][4]  the same words, four tokens side by side
  K meta   [page]                  scale bits (16-bit type) | zero point << 16
  V meta   [page]
and a value is (code - zero point) * scale.
"""
import math

import torch

own = False

EPS = 2.0 ** -17  # a power of two: the same number in 32 and in 64 bits
ROPE_BASE = 500000.0
_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# where column c of a word sits: nibble c / 2 + 4 (c % 2)
_SHIFT = [4 * (c // 2 + 4 * (c % 2)) for c in range(8)]


# ----------------------------------------------------------------------------- cases

def _norm(name, rows, cols, dtype, out, residual=True):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "out": out, "residual": residual}


def _append(name, seqs, tokens, heads, kv_heads, dim, rot, layout, page, dtype):
    return {"name": name, "op": "append", "seqs": seqs, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "rot": rot, "layout": layout, "page": page, "dtype": dtype}


def _attention(name, seqs, new, kv, heads, kv_heads, dim, page, window, dtype):
    return {"name": name, "op": "attention", "seqs": seqs, "new": new, "kv": kv, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "dtype": dtype}


def listed():
    return [
        # one token of one sequence through a 4096-wide layer: latency
        _norm("norm_one_token", 1, 4096, "f16", "int8"),
        # a prompt of 4096 tokens
        _norm("norm_prompt", 4096, 4096, "f16", "int8"),
        # an odd batch of wide rows into the fp8 product
        _norm("norm_odd_fp8", 777, 8192, "bf16", "fp8"),
        # one step of 64 sequences being answered, Llama-3-8B heads
        _append("append_decode", 64, 64, 32, 8, 128, 128, "half", 16, "bf16"),
        # two prompts of 4096 tokens
        _append("append_prompt", 2, 8192, 32, 8, 128, 128, "half", 64, "f16"),
        # ragged prompts, opt-125m heads, half of each head rotated in interleaved pairs
        _append("append_partial", 7, 1021, 12, 12, 64, 32, "interleaved", 16, "bf16"),
        # one answer, a short context: latency
        _attention("decode_short", 1, 1, 137, 32, 8, 128, 16, 0, "f16"),
        # a full batch of answers, contexts of 4096 to 8192 tokens
        _attention("decode_batch", 64, 1, 8192, 32, 8, 128, 16, 0, "bf16"),
        # Llama-2-7B heads (each query head has keys of its own)
        _attention("decode_mha", 16, 1, 2050, 32, 32, 128, 32, 0, "f16"),
        # two answers over very long contexts
        _attention("decode_long", 2, 1, 131072, 32, 8, 128, 128, 0, "f16"),
        # a whole prompt
        _attention("prompt", 1, 4096, 4096, 32, 8, 128, 64, 0, "f16"),
        # a mixed batch: chunks of prompts over earlier context, sliding window
        _attention("chunks_window", 5, 700, 3700, 32, 8, 128, 16, 1000, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attention", "attention"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "norm":
        cols = rng.choice([768, 2048, 4096, 5120, 8192, 11008, 14336, 8 * _log(rng, 8, 2048)])
        rows = _log(rng, 1, max(1, (4096 * 4096) // cols))
        return {k: v for k, v in _norm("", rows, cols, dtype, rng.choice(["int8", "fp8"]),
                                       rng.random() < 0.75).items() if k != "name"}
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 12, 32])
    heads = kv_heads * (rng.choice([1, 4, 4, 7, 8]) if kv_heads < 12 else 1)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        most = max(2, 8192 * 48 * 128 // ((heads + 2 * kv_heads) * dim))
        tokens = _log(rng, 1, most)
        seqs = rng.choice([1, tokens, _log(rng, 1, tokens)]) if tokens <= 512 else _log(rng, 1, 32)
        rot = rng.choice([dim, dim, dim // 2, 16])
        return {k: v for k, v in _append("", seqs, tokens, heads, kv_heads, dim, rot,
                                         rng.choice(["half", "interleaved"]), page, dtype).items() if k != "name"}
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    kind = rng.choice(["decode", "decode", "few", "prompt"])
    if kind == "prompt":
        new = _log(rng, 64, 4096)
        kv = new + rng.choice([0, _log(rng, 1, 4096)])
        # at most the whole prompt's products, and a score matrix that the plain form can hold
        most = 4096 * 4096 * 32
        new = min(new, max(64, most // (kv * heads)))
        seqs = rng.randint(1, max(1, min(most // (new * kv * heads), 16)))
    else:
        new = 1 if kind == "decode" else rng.randint(2, 16)
        kv = _log(rng, 16, 65536)
        most = max(1, 64 * 8192 * 8 * 128 // (kv * kv_heads * dim * (1 if new == 1 else 4)))
        seqs = _log(rng, 1, min(most, 128))
    return {k: v for k, v in _attention("", seqs, new, kv, heads, kv_heads, dim, page, window,
                                        dtype).items() if k != "name"}


def _lengths(case):
    """(new tokens, context with them) of each sequence: the first has the most, the others are spread below it."""
    if case["op"] == "append":
        n, t = case["seqs"], case["tokens"]
        new = [t // n + (1 if b < t % n else 0) for b in range(n)]
        return new, [m + (b * 1237) % 2048 for b, m in enumerate(new)]
    new, kv = [], []
    for b in range(case["seqs"]):
        k = case["kv"] - (b * 7919) % (case["kv"] // 2 + 1)
        m = case["new"] - (b * 613) % (case["new"] // 2 + 1) if case["new"] > 16 else case["new"]
        new.append(min(m, k))
        kv.append(k)
    return new, kv


def work(case):
    if case["op"] == "norm":
        m, k = case["rows"], case["cols"]
        b = 2 * m * k + 2 * k + m * k + 4 * m
        b += 4 * m * k if case["residual"] else 0  # the residual in and out
        b += 4 * m if case["out"] == "fp8" else 0
        return {"bytes": b, "flops": 8 * m * k}
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    new, kv = _lengths(case)
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": 2 * t * (hq + 2 * hk) * d + 4 * t * case["rot"] + 12 * t + 2 * t * hq * d + t * hk * (d + 8),
                "flops": 3 * t * (hq + hk) * case["rot"] + 8 * t * 2 * hk * d}
    pairs = read = 0
    w = case["window"]
    for n, k in zip(new, kv):
        first = k - n  # position of the first new token
        if w:
            pairs += sum(min(p + 1, w) for p in range(first, k))
            read += min(k, n + w - 1)
        else:
            pairs += n * first + n * (n + 1) // 2
            read += k
    t = sum(new)
    return {"bytes": 4 * t * hq * d + read * hk * (d + 8) + 4 * sum(-(-k // case["page"]) for k in kv),
            "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------------------- the format, in plain torch

def _divide(a, b):
    """a / b in binary32, correctly rounded (a quotient of two binary32 numbers taken in 64 bits and rounded again is)."""
    return (a.double() / b.double()).float()


def _quantise4(x):
    """Codes, scale and zero point of the last axis of x (16-bit type)."""
    f = x.float()
    lo, hi = f.amin(-1).clamp(max=0), f.amax(-1).clamp(min=0)
    s = _divide(hi - lo, torch.full_like(lo, 15.0)).to(x.dtype)
    d = torch.where(s > 0, s, 1).float()
    z = torch.round(_divide(-lo, d)).clamp(0, 15)
    c = (torch.round(_divide(f, d[..., None])) + z[..., None]).clamp(0, 15)
    live = s > 0
    return (c * live[..., None]).to(torch.int32), s, (z * live).to(torch.int32)


def _words(codes):
    """[..., D] codes as [..., D / 8] packed words."""
    sh = torch.tensor(_SHIFT, dtype=torch.int64, device=codes.device)
    w = (codes.to(torch.int64).unflatten(-1, (-1, 8)) << sh).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _meta(s, z):
    return (s.view(torch.int16).to(torch.int32) & 0xFFFF) | (z << 16)


def _sections(cache, dim, page):
    """The K words, V words, K meta and V meta of a cache, as views."""
    n = page * dim // 8
    head = cache.shape[:2]
    return (cache[..., :n].view(*head, page, dim // 8), cache[..., n:2 * n].view(*head, page // 4, dim // 8, 4),
            cache[..., 2 * n:2 * n + page], cache[..., 2 * n + page:])


def _store(cache, dim, page, slots, k, v):
    """Quantise k, v [T, kv_heads, dim] into the slots [T] of a cache."""
    p, t = slots // page, slots % page
    kw, vw, km, vm = _sections(cache, dim, page)
    c, s, z = _quantise4(k)
    kw[p, :, t] = _words(c)
    km[p, :, t] = _meta(s, z)
    c, s, z = _quantise4(v)
    vw[p, :, t // 4, :, t % 4] = _words(c)
    vm[p, :, t] = _meta(s, z)


def _values(words, meta, dtype):
    """[..., D] values of words [..., D / 8] and meta [...]."""
    sh = torch.tensor(_SHIFT, dtype=torch.int32, device=words.device)
    c = ((words[..., None] >> sh) & 15).flatten(-2).float()
    s = (meta & 0xFFFF).to(torch.int16).view(dtype).float()
    return (c - (meta >> 16)[..., None].float()) * s[..., None]


def _rotate(x, cs, rot, layout):
    """x [T, H, D] turned by its tokens' cos and sin (cs [T, rot]); each step rounds to binary32, the result to x's type."""
    f = x[..., :rot].float()
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (f[..., :rot // 2], f[..., rot // 2:]) if layout == "half" else (f[..., 0::2], f[..., 1::2])
    p, q = a * c - b * s, b * c + a * s
    r = torch.cat((p, q), -1) if layout == "half" else torch.stack((p, q), -1).flatten(-2)
    return torch.cat((r.to(x.dtype), x[..., rot:]), -1)


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case)
    if case["op"] == "norm":
        m, k = case["rows"], case["cols"]
        # hidden states: a few channels much larger than the others
        loud = 1 + 12 * (torch.rand(k, generator=g, device="cuda") < 0.004)
        st["x"] = (0.5 * randn(m, k)).to(dt)
        st["residual_in"] = (randn(m, k) * loud).to(dt) if case["residual"] else None
        st["weight"] = (1 + 0.1 * randn(k)).to(dt)
        return st
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    new, kv = _lengths(case)
    # pages of the sequences, in no order, in a pool that other sequences use too
    per = [-(-n // page) for n in kv]
    pool = sum(per) + 8
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    starts = torch.tensor([0] + per).cumsum(0).cuda()
    width = max(per)
    col = torch.arange(width, device="cuda")
    at = starts[:-1, None] + col
    tables = torch.where(at < starts[1:, None], order[at.clamp(max=pool - 1)], torch.full_like(order[:1], -1))
    cache = torch.zeros(pool, hk, page * (d // 4 + 2), dtype=torch.int32, device="cuda")
    st["cache"] = cache
    lens = torch.tensor(kv, dtype=torch.int32)
    newt = torch.tensor(new, dtype=torch.int32)
    total = sum(new)
    shift = 0.8 * randn(hk, d)  # keys have an offset of their own in each channel
    if case["op"] == "append":
        qkv = randn(total, (hq + 2 * hk), d)
        qkv[:, hq:hq + hk] += shift
        st["qkv"] = qkv.to(dt)  # as a fused product gives it
        row = torch.arange(total)
        b = torch.repeat_interleave(torch.arange(len(new)), newt.long())
        first = newt.cumsum(0) - newt
        pos = (row - first[b] + lens[b] - newt[b]).to(torch.int32).cuda()
        st["positions"] = pos
        st["slots"] = tables[b.cuda(), pos.long() // page].long() * page + pos % page
        rot = case["rot"]
        inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ang = torch.arange(max(kv), dtype=torch.float64, device="cuda")[:, None] * inv
        st["rope"] = torch.cat((ang.cos(), ang.sin()), -1).float()
        return st
    # the whole context is in the cache already, the new tokens with it
    step = max(1, (1 << 27) // (page * hk * d))
    for p in range(0, pool, step):
        n = min(step, pool - p)
        slots = torch.arange(p * page, (p + n) * page, device="cuda")
        _store(cache, d, page, slots, (randn(n * page, hk, d) + shift).to(dt), randn(n * page, hk, d).to(dt))
    st["q"] = (1.5 * randn(total, hq, d)).to(dt)
    st["tables"] = tables
    st["lens"] = lens.cuda()
    st["cu_q"] = torch.cat((torch.zeros(1, dtype=torch.int32), newt.cumsum(0).to(torch.int32))).cuda()
    st["max_new"], st["max_kv"] = max(new), max(kv)
    st["scale"] = 1.0 / math.sqrt(d)
    return st


# ----------------------------------------------------------------------------- the operators

def _plain_norm(st):
    x, w = st["x"], st["weight"]
    h = x if st["residual_in"] is None else (x.float() + st["residual_in"].float()).to(x.dtype)
    v = (h.double().square().mean(-1, keepdim=True) + EPS).float()
    r = _divide(torch.ones_like(v), v.double().sqrt().float())
    y = ((h.float() * r) * w.float()).to(x.dtype)
    top = 127.0 if st["out"] == "int8" else 448.0
    amax = y.float().abs().amax(-1, keepdim=True)
    s = _divide(amax, torch.full_like(amax, top)).to(x.dtype).float()
    q = torch.where(s > 0, _divide(y.float(), torch.where(s > 0, s, 1)), 0)
    out = {"s1": s[:, 0]}
    if st["residual_in"] is not None:
        out["residual"] = h
    if st["out"] == "int8":
        out["a8"] = torch.round(q).clamp(-128, 127).to(torch.int8)
    else:
        out["a8"] = q.clamp(-448, 448).to(torch.float8_e4m3fn)
        out["asum"] = out["a8"].double().sum(-1).float()
    return out


def _plain_append(st):
    hq, hk, rot = st["heads"], st["kv_heads"], st["rot"]
    cs = st["rope"][st["positions"].long()]
    q, k, v = st["qkv"].split((hq, hk, hk), 1)
    q = _rotate(q, cs, rot, st["layout"])
    _store(st["cache"], st["dim"], st["page"], st["slots"], _rotate(k, cs, rot, st["layout"]), v)
    return {"q": q, "cache": st["cache"]}


def _plain_attention(st):
    q, page, d, hk = st["q"], st["page"], st["dim"], st["kv_heads"]
    dt, seqs, n, m = q.dtype, st["lens"].shape[0], st["max_kv"], st["max_new"]
    group = st["heads"] // hk
    # the dense keys and values of every sequence, padded to the longest
    pages = st["cache"][st["tables"][:, :-(-n // page)].clamp(min=0).long()].transpose(1, 2)
    kw, vw, km, vm = _sections(pages.flatten(1, 2), d, page)
    shape = (seqs, hk, -1, d)
    k = _values(kw, km, dt).reshape(shape)
    v = _values(vw.transpose(3, 4).flatten(2, 3), vm, dt).reshape(shape)
    # queries by sequence, padded to the most new tokens
    cu = st["cu_q"].long()
    first, cnt, lens = cu[:-1, None], cu[1:, None] - cu[:-1, None], st["lens"].long()[:, None]
    i = torch.arange(m, device="cuda")
    rows = q[(first + i).clamp(max=q.shape[0] - 1)].float().view(seqs, m, hk, group, d).permute(0, 2, 3, 1, 4)
    t = (rows.reshape(seqs, hk, group * m, d) @ k.transpose(2, 3)).mul_(st["scale"]).view(seqs, hk, group, m, -1)
    at = (lens - cnt + i)[:, :, None]
    j = torch.arange(t.shape[-1], device="cuda")
    seen = (j <= at) & (i < cnt)[:, :, None]
    if st["window"]:
        seen &= j > at - st["window"]
    seen = seen[:, None, None]
    t = t.masked_fill_(~seen, -math.inf)
    top = t.amax(-1, keepdim=True)
    p = t.sub_(torch.where(top > -math.inf, top, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(seqs, hk, group * m, -1) @ v).view(seqs, hk, group, m, d) / torch.where(total > 0, total, 1)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, m, hk * group, d)
    return o[(i < cnt)].to(dt)  # the rows of each sequence in turn


def _own(st):
    import bit_weight_only_awq_amd as awq
    if st["op"] == "norm":
        res = st["residual_in"]
        if st["out"] == "int8":
            a8, s1, h = awq.rmsnorm_quant(st["x"], st["weight"], EPS, residual=res)
            out = {"s1": s1, "a8": a8}
        else:
            a8, s1, asum, h = awq.rmsnorm_quant_fp8(st["x"], st["weight"], EPS, residual=res)
            out = {"s1": s1, "a8": a8.view(torch.float8_e4m3fn), "asum": asum}
        if res is not None:
            out["residual"] = h
        return out
    if st["op"] == "append":
        q, k, v = st["qkv"].split((st["heads"], st["kv_heads"], st["kv_heads"]), 1)
        q = awq.kv4_append(q, k, v, st["rope"], st["positions"], st["slots"], st["cache"],
                           interleaved=st["layout"] == "interleaved")
        return {"q": q, "cache": st["cache"]}
    return awq.kv4_attention(st["q"], st["cache"], st["tables"], st["lens"], scale=st["scale"], cu_q=st["cu_q"],
                             max_q=st["max_new"], max_kv=st["max_kv"], window=st["window"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[state["op"]](state)


# ----------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits.  Where a definition rounds to 32 or 16 bits on the way to a
    scale or a code, it does so here too.  Codes and packed words have no value but themselves: None."""
    st = prepare(case, seed)
    dt = _DT[case["dtype"]]

    def f32(a):
        return a.float().double()

    def act(a):
        return a.float().to(dt).double()

    if case["op"] == "norm":
        h = st["x"].double()
        if case["residual"]:
            h = act(h + st["residual_in"].double())
        r = f32(1 / f32(torch.sqrt(f32((h * h).sum(1) / case["cols"] + EPS))))
        y = act(f32(h * r[:, None]) * st["weight"].double())
        top = 127 if case["out"] == "int8" else 448
        s = act(f32(y.abs().max(1).values / top))
        out = {"s1": s, "a8": None}
        if case["residual"]:
            out["residual"] = h
        if case["out"] == "fp8":
            code = f32(y / s[:, None]).clamp(-448, 448).nan_to_num(0.0).float().to(torch.float8_e4m3fn).double()
            out["a8"], out["asum"] = code, code.sum(1)
        return out
    if case["op"] == "append":
        rot, hq = case["rot"], case["heads"]
        q = st["qkv"][:, :hq].double()
        inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ang = st["positions"].double()[:, None] * inv
        turn = torch.polar(torch.ones_like(ang), ang)[:, None]
        if case["layout"] == "half":
            w = torch.complex(q[..., :rot // 2], q[..., rot // 2:rot]) * turn
            turned = torch.cat((w.real, w.imag), -1)
        else:
            w = torch.complex(q[..., :rot:2], q[..., 1:rot:2]) * turn
            turned = torch.view_as_real(w).flatten(-2)
        return {"q": torch.cat((turned, q[..., rot:]), -1), "cache": None}
    # attention, one sequence and one head of the cache at a time
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    group, n8 = case["heads"] // hk, page * d // 8
    new, kv = _lengths(case)
    out = torch.zeros(sum(new), case["heads"], d, dtype=torch.float64, device="cuda")
    nib = [0, 2, 4, 6, 1, 3, 5, 7]
    row = 0
    for b, (m, n) in enumerate(zip(new, kv)):
        ids = st["tables"][b, :-(-n // page)].long()
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")
        hidden = key > pos
        if case["window"]:
            hidden |= key <= pos - case["window"]
        for h in range(hk):
            body = st["cache"][ids, h]
            both = []
            for part in (0, 1):
                w = body[:, part * n8:(part + 1) * n8]
                w = w.reshape(-1, page, d // 8) if part == 0 else \
                    w.reshape(-1, page // 4, d // 8, 4).permute(0, 1, 3, 2).reshape(-1, page, d // 8)
                val = torch.empty(*w.shape, 8, dtype=torch.float64, device="cuda")
                for i in range(8):
                    val[..., nib[i]] = ((w.long() >> (4 * i)) % 16).double()
                meta = body[:, 2 * n8 + part * page:2 * n8 + (part + 1) * page].long()
                s = (meta % 65536).to(torch.int32).to(torch.int16).view(dt).double()
                val = (val.flatten(-2) - (meta // 65536).double()[..., None]) * s[..., None]
                both.append(val.reshape(-1, d)[:n])
            for e in range(group):
                t = st["q"][row:row + m, h * group + e].double() @ both[0].t() * st["scale"]
                out[row:row + m, h * group + e] = torch.softmax(t.masked_fill(hidden, -math.inf), 1) @ both[1]
        row += m
    return out
