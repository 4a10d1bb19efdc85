"""A mixture-of-experts layer's operators in 4-bit weights and block-scaled FP8, as measured workloads.

Five operators of a quantised model's serving path:

  route    each token's top experts, their softmax weights, and the plan: the
           chosen (token, place) slots in the order of their experts
  experts  matrix products grouped by expert over ragged runs of rows, weights
           in the AWQ 4-bit format of the dense layers
  combine  the weighted sum of each token's experts' rows
  quant    16-bit activations as E4M3 codes with one scale for each run of 128
           values of a row
  product  matrix products of such codes with E4M3 weights that have one scale
           for each block of 128 x 128, one weight matrix or one per expert

`run` computes an operator in plain torch operations where `own` is false, and
calls the library where it is true.

Definitions.  route: of the logits l[t, e] (infinity counted as the largest
finite binary32 number; minus infinity and NaN never chosen) the k largest, ties to the
lower expert; weight exp(l - max) over the sum of all eligible experts', or of
the chosen ones'.  Slot t k + j holds the token's j-th choice; `rows` lists the
slots by expert, then by slot, `offsets` where each expert's begin, `places`
where each slot went.  quant: s = f32(max |x| / 448), codes
e4m3(clamp(f32(x / s), -448, 448)) (s = 0: codes 0).  product: the sum over the
blocks b of 128 along K of sa[m, b] sw[n / 128, b] sum_k a[m, k] w[n, k].
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_ORDER = (0, 2, 4, 6, 1, 3, 5, 7)  # nibble i of a packed word holds column 8 j + _ORDER[i]
_TOP = 448.0                       # the largest E4M3 number


# ----------------------------------------------------------------------------- cases

def _route(name, tokens, experts, top, renormalize, dtype):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top": top,
            "renormalize": renormalize, "dtype": dtype}


def _experts(name, tokens, experts, top, k, n, group, zeros, gather, dtype):
    return {"name": name, "op": "experts", "tokens": tokens, "experts": experts, "top": top, "k": k, "n": n,
            "group": group, "zeros": zeros, "gather": gather, "dtype": dtype}


def _combine(name, tokens, top, n, dtype):
    return {"name": name, "op": "combine", "tokens": tokens, "top": top, "n": n, "dtype": dtype}


def _quant(name, rows, cols, dtype):
    return {"name": name, "op": "quant", "rows": rows, "cols": cols, "dtype": dtype}


def _product(name, tokens, experts, top, k, n, gather, dtype):
    return {"name": name, "op": "product", "tokens": tokens, "experts": experts, "top": top, "k": k, "n": n,
            "gather": gather, "dtype": dtype}


def listed():
    return [
        # one answer's next token: latency
        _route("route_one_token", 1, 64, 8, True, "bf16"),
        # a prompt, an odd number of tokens, many experts
        _route("route_prompt", 8191, 128, 8, False, "f32"),
        # one answer's next token through gate and up of 8 experts (two of them chosen), Llama-3-8B widths
        _experts("experts_one_token", 1, 8, 2, 4096, 28672, 128, True, True, "f16"),
        # a batch of 32 answers through down: rows in the order of their experts already
        _experts("experts_batch", 32, 8, 2, 14336, 4096, 128, True, False, "bf16"),
        # a prompt of 4096 tokens through gate and up
        _experts("experts_prompt", 4096, 8, 2, 4096, 28672, 128, True, True, "f16"),
        # one step of 64 answers, two experts each
        _combine("combine_batch", 64, 2, 4096, "f16"),
        # a prompt, eight experts each
        _combine("combine_prompt", 4095, 8, 4096, "bf16"),
        # one token: latency
        _quant("quant_one_token", 1, 4096, "f16"),
        # a prompt's MLP activations
        _quant("quant_prompt", 4096, 14336, "bf16"),
        # one token through a dense layer
        _product("product_one_token", 1, 0, 1, 4096, 14336, False, "bf16"),
        # a prompt through a dense layer
        _product("product_prompt", 4096, 0, 1, 4096, 14336, False, "bf16"),
        # an odd prompt through 64 small experts, eight each: about 97 rows an expert, ragged
        _product("product_experts", 777, 64, 8, 2048, 2048, True, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "combine", "quant", "product", "product"])
    dtype = rng.choice(["f16", "bf16"])
    experts = rng.choice([4, 8, 8, 16, 60, 64, 128])
    top = min(rng.choice([1, 2, 2, 4, 6, 8]), experts)
    if op == "route":
        case = _route("", _log(rng, 1, 8191 * 128 // max(experts, 32)), experts, top, rng.random() < 0.5,
                      rng.choice(["f16", "bf16", "f32"]))
    elif op == "combine":
        n = rng.choice([768, 2048, 4096, 8192, 8 * _log(rng, 8, 1024)])
        case = _combine("", _log(rng, 1, 4095 * 8 * 4096 // (top * n)), top, n, dtype)
    elif op == "quant":
        cols = rng.choice([768, 2048, 4096, 11008, 14336, 16 * _log(rng, 4, 1024)])
        case = _quant("", _log(rng, 1, 4096 * 14336 // cols), cols, dtype)
    elif op == "experts":
        group = rng.choice([32, 64, 128, 128])
        k = rng.choice([768, 2048, 4096, 14336, group * _log(rng, 2, 64)])
        n = rng.choice([768, 1408, 4096, 14336, 8 * _log(rng, 8, 1024)])
        experts = min(experts, max(4, 8 * 4096 * 28672 // (k * n)))
        top = min(top, experts)
        tokens = _log(rng, 1, max(2, min(8192, 4096 * 2 * 4096 * 28672 // (top * k * n))))
        case = _experts("", tokens, experts, top, k, n, group, rng.random() < 0.7, rng.random() < 0.5, dtype)
    else:
        k = rng.choice([768, 2048, 4096, 11008, 14336, 16 * _log(rng, 8, 512)])
        n = rng.choice([768, 1408, 4096, 14336, 8 * _log(rng, 8, 1024)])
        experts = rng.choice([0, 0, experts])
        experts = min(experts, max(4, 8 * 4096 * 14336 // (k * n)))
        top = min(top, experts) if experts else 1
        tokens = _log(rng, 1, max(2, min(16384, 4096 * 4096 * 14336 // (top * k * n))))
        case = _product("", tokens, experts, top, k, n, experts > 0 and rng.random() < 0.5, dtype)
    return {name: v for name, v in case.items() if name != "name"}


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top"]
        # logits in; weights, experts, rows and places out
        return {"bytes": t * e * (4 if case["dtype"] == "f32" else 2) + 16 * t * k + 4 * (e + 1), "flops": 4 * t * e}
    if op == "combine":
        t, k, n = case["tokens"], case["top"], case["n"]
        return {"bytes": 2 * t * k * n + 2 * t * n + 8 * t * k, "flops": 2 * t * k * n}
    if op == "quant":
        m, k = case["rows"], case["cols"]
        return {"bytes": 3 * m * k + 4 * m * -(-k // 128), "flops": 4 * m * k}
    t, e, k, n = case["tokens"], case["experts"], case["k"], case["n"]
    rows = t * case["top"]
    live = e * (1 - (1 - case["top"] / e) ** t) if e else 1  # the experts that some token chose, when all are alike
    read = t if case["gather"] else rows
    if op == "experts":
        g = case["group"]
        weights = k * n // 2 + 2 * (k // g) * n + ((k // g) * n // 2 if case["zeros"] else 0)
        b = live * weights + 2 * read * k + 2 * rows * n
    else:
        blocks = -(-k // 128)
        b = live * (k * n + 4 * blocks * -(-n // 128)) + read * (k + 4 * blocks) + 2 * rows * n
    return {"bytes": int(b) + (8 * rows if e else 0), "flops": 2 * rows * k * n}


# ----------------------------------------------------------------------------- formats, in plain torch

def _divide(a, b):
    """a / b in binary32, correctly rounded (a quotient of two binary32 numbers taken in 64 bits and rounded again is)."""
    return (a.double() / b.double()).float()


def _block_codes(x):
    """E4M3 codes of x [M, K] and the scales [M, ceil(K / 128)] of its runs of 128."""
    m, k = x.shape
    f = x.float()
    pad = torch.nn.functional.pad(f, (0, -k % 128)).unflatten(1, (-1, 128))
    amax = pad.abs().amax(-1)
    s = _divide(amax, torch.full_like(amax, _TOP))
    q = torch.where(s > 0, 1, 0)[..., None] * _divide(pad, torch.where(s > 0, s, 1)[..., None])
    return q.clamp(-_TOP, _TOP).to(torch.float8_e4m3fn).flatten(1)[:, :k].contiguous(), s


def _columns(words):
    """[..., N / 8] packed words as [..., N] whole numbers 0..15."""
    shift = torch.empty(8, dtype=torch.int32, device=words.device)
    for i, c in enumerate(_ORDER):
        shift[c] = 4 * i
    return ((words[..., None] >> shift) & 15).flatten(-2)


def _plan(ids, experts):
    """offsets, rows and places of the slots' experts ids [T, k] (-1: none)."""
    flat = torch.where(ids < 0, experts, ids).flatten()
    order = torch.sort(flat, stable=True).indices
    offsets = (flat[None, :] < torch.arange(experts + 1, device=flat.device)[:, None]).sum(1)
    at = torch.empty_like(order)
    at[order] = torch.arange(len(order), device=order.device)
    live = flat[order] < experts
    return (offsets.to(torch.int32), torch.where(live, order, -1).to(torch.int32),
            torch.where(flat < experts, at, -1).to(torch.int32))


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def hidden(m, k):
        """Hidden states: a few channels much larger than the others."""
        return randn(m, k) * (1 + 12 * (rand(k) < 0.004))

    st = dict(case)
    if op == "quant":
        st["x"] = hidden(case["rows"], case["cols"]).to(dt)
        return st
    t, e, top = case["tokens"], case.get("experts", 0), case["top"]
    if op == "route":
        # experts differ in popularity
        st["logits"] = (1.5 * randn(t, e) + 0.7 * randn(e)).to(dt)
        return st
    if op == "combine":
        st["y"] = randn(t * top, case["n"]).to(dt)
        st["weights"] = torch.softmax(randn(t, top), 1)
        ids = torch.rand(t, 8, generator=g, device="cuda").argsort(1)[:, :top]
        st["places"] = _plan(ids, 8)[2]
        return st
    k, n = case["k"], case["n"]
    rows = t * top
    if e:
        ids = (1.5 * randn(t, e) + 0.7 * randn(e)).topk(top, 1).indices
        offsets, order, _ = _plan(ids, e)
        st["offsets"], st["rows"] = offsets, order if case["gather"] else None
        st["counts"] = offsets.diff().tolist()  # (for the plain form's loop)
    x = hidden(t if case["gather"] else rows, k)
    if op == "experts":
        gr = case["group"]
        st["x"] = x.to(dt)

        def words(*shape):
            return torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)

        st["qweight"] = torch.stack([words(k, n // 8) for _ in range(e)])
        st["qzeros"] = words(e, k // gr, n // 8) if case["zeros"] else None
        st["scales"] = ((0.5 + rand(e, k // gr, n)) / (4.6 * k ** 0.5)).to(dt)
        return st
    st["a"], st["sa"] = _block_codes(x.to(torch.bfloat16))
    kb, nb = -(-k // 128), -(-n // 128)
    w = torch.empty(max(e, 1), n, k, dtype=torch.float8_e4m3fn, device="cuda")
    sw = torch.empty(max(e, 1), nb, kb, device="cuda")
    for i in range(max(e, 1)):
        f = torch.nn.functional.pad(randn(n, k) * k ** -0.5, (0, -k % 128, 0, -n % 128))
        f = f.view(nb, 128, kb, 128)
        sw[i] = f.abs().amax((1, 3)) / _TOP
        w[i] = (f / sw[i][:, None, :, None]).clamp(-_TOP, _TOP).reshape(nb * 128, kb * 128)[:n, :k].to(w.dtype)
    st["w"], st["sw"] = (w, sw) if e else (w[0], sw[0])
    return st


# ----------------------------------------------------------------------------- the operators

def _plain_route(st):
    e, top = st["experts"], st["top"]
    l = st["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=torch.finfo(torch.float32).max)
    v, ids = torch.sort(l, dim=1, descending=True, stable=True)
    v, ids = v[:, :top], ids[:, :top]
    live = v > -math.inf
    best = torch.where(live[:, :1], v[:, :1], 0)
    w = torch.exp(v - best)
    total = w.sum(1, keepdim=True) if st["renormalize"] else torch.exp(l - best).sum(1, keepdim=True)
    w = torch.where(live, w / torch.where(total > 0, total, 1), 0)
    ids = torch.where(live, ids, -1)
    offsets, rows, places = _plan(ids, e)
    return {"weights": w, "experts": ids.to(torch.int32), "offsets": offsets, "rows": rows, "places": places}


def _plain_combine(st):
    t, top = st["tokens"], st["top"]
    p = st["places"].view(t, top).long()
    out = torch.zeros(t, st["n"], device="cuda")
    for j in range(top):
        w = torch.where(p[:, j] < 0, 0, st["weights"][:, j])
        out += w[:, None] * st["y"][p[:, j].clamp(min=0)].float()
    return out.to(st["y"].dtype)


def _plain_quant(st):
    a, s = _block_codes(st["x"])
    return {"codes": a, "scales": s}


def _grouped(st, x, weight):
    """x's rows through their experts' weights (weight(e): [K, N] in binary32)."""
    if st["rows"] is not None:
        x = x[st["rows"].long() // st["top"]]
    out, at = [], 0
    for e, c in enumerate(st["counts"]):
        if c:
            out.append(x[at:at + c] @ weight(e))
        at += c
    return torch.cat(out).to(_DT[st["dtype"]])


def _plain_experts(st):
    gr = st["group"]

    def weight(e):
        q = _columns(st["qweight"][e]).float().unflatten(0, (-1, gr))
        z = 8.0 if st["qzeros"] is None else _columns(st["qzeros"][e]).float()[:, None]
        return ((q - z) * st["scales"][e].float()[:, None]).flatten(0, 1)

    return _grouped(st, st["x"].float(), weight)


def _plain_product(st):
    k, n = st["k"], st["n"]
    x = st["a"].float() * st["sa"].repeat_interleave(128, 1)[:, :k]

    def weight(w, sw):
        return (w.float() * sw.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]).t()

    if not st["experts"]:
        return (x @ weight(st["w"], st["sw"])).to(_DT[st["dtype"]])
    return _grouped(st, x, lambda e: weight(st["w"][e], st["sw"][e]))


def _own(st):
    import bit_weight_only_awq_amd as awq
    op = st["op"]
    if op == "route":
        w, ids, offsets, rows, places = awq.moe_route(st["logits"], st["top"], renormalize=st["renormalize"])
        return {"weights": w, "experts": ids, "offsets": offsets, "rows": rows, "places": places}
    if op == "combine":
        return awq.moe_combine(st["y"], st["weights"], st["places"])
    if op == "quant":
        a, s = awq.quant_act_fp8_block(st["x"])
        return {"codes": a.view(torch.float8_e4m3fn), "scales": s}
    if op == "experts":
        return awq.moe_gemm_w4a16(st["x"], st["qweight"], st["scales"], st["qzeros"], st["offsets"], rows=st["rows"],
                                  top_k=st["top"], group_size=st["group"])
    if st["experts"]:
        return awq.moe_gemm_fp8_block(st["a"], st["w"], st["sa"], st["sw"], st["offsets"], rows=st["rows"],
                                      top_k=st["top"], dtype=_DT[st["dtype"]])
    return awq.gemm_fp8_block(st["a"], st["w"], st["sa"], st["sw"], dtype=_DT[st["dtype"]])


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "combine": _plain_combine, "quant": _plain_quant, "experts": _plain_experts,
            "product": _plain_product}[state["op"]](state)


# ----------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits.  The plan of a routing has no value but itself: None."""
    st = prepare(case, seed)
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "route":
        l = st["logits"].double()
        chosen = torch.zeros_like(l, dtype=torch.bool)
        w = torch.exp(l - l.max(1, keepdim=True).values)
        picks = []
        for _ in range(case["top"]):
            # the lowest of the experts that are left with the largest logit
            rest = l.masked_fill(chosen, -math.inf)
            is_max = rest == rest.max(1, keepdim=True).values
            i = torch.where(is_max, torch.arange(l.shape[1], device="cuda"), l.shape[1]).min(1, keepdim=True).values
            chosen.scatter_(1, i, True)
            picks.append(w.gather(1, i))
        w_top = torch.cat(picks, 1)
        whole = w_top.sum(1, keepdim=True) if case["renormalize"] else w.sum(1, keepdim=True)
        return {"weights": w_top / whole, "experts": None, "offsets": None, "rows": None, "places": None}
    if op == "combine":
        y, p = st["y"].double(), st["places"].long()
        terms = y[p].unflatten(0, (-1, case["top"])) * st["weights"].double()[..., None]
        return terms.sum(1)
    if op == "quant":
        x = st["x"].double()
        out, scales = torch.empty_like(x), []
        for b in range(0, case["cols"], 128):
            run_ = x[:, b:b + 128]
            s = (run_.abs().max(1, keepdim=True).values / 448).float().double()
            scales.append(s)
            q = (run_ / s).nan_to_num(0.0).float().clamp(-448, 448)
            out[:, b:b + 128] = q.to(torch.float8_e4m3fn).double()
        return {"codes": out, "scales": torch.cat(scales, 1)}
    k, n, e = case["k"], case["n"], case["experts"]
    if op == "product":
        x = st["a"].double()
        for b in range(0, k, 128):
            x[:, b:b + 128] *= st["sa"][:, b // 128:b // 128 + 1].double()
        block_n = torch.arange(n, device="cuda") // 128
        block_k = torch.arange(k, device="cuda") // 128

        def weight(i):
            w, s = (st["w"][i], st["sw"][i]) if e else (st["w"], st["sw"])
            return w.double() * s.double()[block_n][:, block_k]  # [N, K]
    else:
        x = st["x"].double()

        def weight(i):
            w = torch.empty(n, k, dtype=torch.float64, device="cuda")
            words = st["qweight"][i].long() & 0xFFFFFFFF
            per = torch.arange(k, device="cuda") // case["group"]
            for nibble, c in enumerate(_ORDER):
                q = (words // 16 ** nibble) % 16
                z = 8 if st["qzeros"] is None else (((st["qzeros"][i].long() & 0xFFFFFFFF) // 16 ** nibble) % 16)[per]
                w[c::8] = ((q - z).double() * st["scales"][i][:, c::8].double()[per]).t()
            return w
    if not e:
        return x @ weight(0).t()
    out = torch.empty(case["tokens"] * case["top"], n, dtype=torch.float64, device="cuda")
    ends = st["offsets"].tolist()
    for i in range(e):
        lo, hi = ends[i], ends[i + 1]
        if lo == hi:
            continue
        mine = x[lo:hi] if st["rows"] is None else x[torch.div(st["rows"][lo:hi].long(), case["top"],
                                                               rounding_mode="floor")]
        out[lo:hi] = mine @ weight(i).t()
    return out
