"""Attention over the 4-bit paged cache, against the oracle in 64 bits.

Bound on each output element, from the roundings the header states (u = half a
step of the type): the output's own, u_out |y|; the softmax numerators' one to
11 bits, 2^-11 sum p |v|, and where they fall below fp16's normal range (2^-28
of the largest value scale) 2^-39 of it a token; the scores', which move p by
twice their error: 2^-24 a term for the sums of D products of codes up to 15
and of the zero points' part (2 * 15 sum |q| s scale, over D + 32 roundings);
exp2's two units; and the fp32 sums over the tokens, n / 4 + 256 roundings of
terms up to 30 s' each."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def t16(bits, dtype):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(DT[dtype])


def b16(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


class Case:
    """A cache with sequences of the given lengths on shuffled pages; every word that no row may use is garbage."""

    def __init__(self, lens, new, hq, hkv, D, P, dtype, seed=0, k_size=1.0, v_size=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.dtype, self.P, self.hq, self.D = dtype, P, hq, D
        self.lens, self.new = np.array(lens, dtype=np.int32), np.array(new, dtype=np.int32)
        per = [-(-n // P) for n in lens]
        pages = sum(per) + 1
        order = rng.permutation(pages)
        width = max(per + [1]) + spare
        self.tables = rng.integers(-2 ** 31, 2 ** 31, (len(lens), width)).astype(np.int32)  # unused entries: anything
        cache = rng.integers(-2 ** 31, 2 ** 31, (pages, hkv, block.head_words(D, P))).astype(np.int64).astype(np.int32)
        nan = 0x7E00 if dtype == "f16" else 0x7FC0
        cache[:, :, 2 * P * D // 8:] = np.int32((np.uint32(0x7E00) << 16 | nan).astype(np.uint32).view(np.int32))
        at = 0
        for b, n in enumerate(lens):
            self.tables[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            if n:
                tok = np.arange(n)
                slots = self.tables[b, tok // P].astype(np.int64) * P + tok % P
                k = rng.standard_normal((n, hkv, D)) * k_size + 0.5 * rng.standard_normal((1, hkv, D))
                v = rng.standard_normal((n, hkv, D)) * v_size * 10.0 ** rng.uniform(-1, 1, (n, 1, 1))
                block.store(cache, P, slots, block.encode(k, dtype), block.encode(v, dtype), dtype)
        self.cache = cache
        self.cu = np.concatenate(([0], np.cumsum(self.new))).astype(np.int32)
        self.q = block.encode(rng.standard_normal((int(self.cu[-1]), hq, D)) * 1.5, dtype)

    def gpu(self, window=0, scale=None, max_kv=None, max_q=None, out=None, q=None):
        put = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
        qd = t16(self.q, self.dtype).to(dev()) if q is None else q
        decode = bool((self.new == 1).all())
        return awq.kv4_attention(qd, put(self.cache), put(self.tables), put(self.lens), scale=scale,
                                 cu_q=None if decode else put(self.cu),
                                 max_q=1 if decode else int(self.new.max()) if max_q is None else max_q,
                                 max_kv=int(self.lens.max()) if max_kv is None else max_kv, window=window, out=out)

    def check(self, window=0, scale=None, **kw):
        y = self.gpu(window, scale, **kw)
        sc = self.D ** -0.5 if scale is None else float(np.float32(scale))
        want, spread, unit = block.attention(self.q, self.cache, self.P, self.tables, self.lens, self.cu, sc, window,
                                             self.dtype)
        got = block.decode(b16(y), self.dtype)
        u = 2.0 ** -11 if self.dtype == "f16" else 2.0 ** -8
        n = max(int(self.lens.max()), 1)
        sv, sq, smax = unit[..., :1], unit[..., 1:2], unit[..., 2:]
        score = 2.0 ** -24 * (self.D + 32) * 30 * sq
        bound = (u * np.abs(want) + (1 + u) * ((2.0 ** -11 + 2 * score + 2.0 ** -21) * spread
                 + 2.0 ** -24 * (n / 4 + 256) * 30 * sv + 2.0 ** -39 * 15 * n * smax)
                 + (2.0 ** -25 if self.dtype == "f16" else 0))
        # a row that sees a token stored as not finite is NaN, and no other
        assert np.array_equal(np.isnan(got), np.isnan(want)) and not np.isinf(got).any()
        bad = np.abs(got - want) > bound
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - want)[bad][:5], bound[bad][:5], want[bad][:5])
        return y


HEADS = [(1, 1), (4, 1), (8, 8), (32, 8), (7, 1), (14, 2), (16, 1), (17, 1), (40, 2), (71, 1)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_decode_heads(hq, hkv, D, dtype):
    Case([1, 40, 0, 131], [1] * 4, hq, hkv, D, 16, dtype, seed=hq + D).check()


@pytest.mark.parametrize("D,dtype", [(128, "f16"), (64, "bf16")])
@pytest.mark.parametrize("P", [16, 32, 64, 256, 1024])
def test_decode_lengths_around_tiles(P, D, dtype):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257]
    Case(lens, [1] * len(lens), 8, 2, D, P, dtype, seed=P).check()


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
def test_decode_split_over_workgroups(D, dtype):
    """One long and several shorter sequences: partial sums through the workspace, again and again."""
    c = Case([2900, 700, 0, 130, 1], [1] * 5, 4, 1, D, 32, dtype, seed=3)
    y = c.check(max_kv=4096)
    for _ in range(3):
        assert torch.equal(c.gpu(max_kv=4096), y)
    assert torch.equal(c.gpu(max_kv=2900).isfinite(), y.isfinite())
    c.check(max_kv=1)      # a bound that is too low costs speed, not correctness
    c.check(max_kv=10 ** 6)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 1000])
def test_decode_window(window, dtype):
    Case([1, 16, 33, 100, 101, 300, 640], [1] * 7, 4, 2, 64, 16, dtype, seed=window).check(window=window)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,D,P,window", [(4, 1, 64, 16, 0), (8, 2, 128, 32, 0), (3, 3, 128, 16, 20),
                                               (14, 2, 64, 64, 7), (1, 1, 64, 16, 0)])
def test_several_new_tokens(hq, hkv, D, P, window, dtype):
    """Decode and several tokens mixed; more new tokens than context (rows that see nothing)."""
    lens, new = [50, 3, 130, 64, 7, 0, 200], [4, 5, 1, 16, 7, 2, 0]
    Case(lens, new, hq, hkv, D, P, dtype, seed=D + P).check(window=window)


@pytest.mark.parametrize("hq,hkv,D,P,window,dtype", [
    (4, 1, 128, 16, 0, "f16"), (2, 2, 64, 32, 0, "bf16"), (8, 2, 128, 64, 50, "bf16"), (4, 4, 64, 16, 130, "f16"),
    (7, 1, 128, 128, 0, "f16")])
def test_prompts(hq, hkv, D, P, window, dtype):
    """Whole prompts and chunks over earlier context, of lengths around the tiles'."""
    lens, new = [127, 300, 128, 65, 513], [127, 77, 128, 65, 33]
    Case(lens, new, hq, hkv, D, P, dtype, seed=hq * D).check(window=window)


def test_rows_past_max_q_are_left():
    c = Case([40, 40], [6, 3], 2, 1, 64, 16, "f16", seed=1)
    full = c.check()
    out = torch.full_like(full, 7.0)
    c.gpu(max_q=4, out=out)
    assert torch.equal(out[:4], full[:4]) and torch.equal(out[6:], full[6:]) and bool((out[4:6] == 7).all())


@pytest.mark.parametrize("new", [1, 40])
def test_missing_pages_hide_their_tokens(new):
    """Table entries that name no page of the cache, inside a sequence."""
    c = Case([200, 90], [new, new], 4, 2, 64, 16, "f16", seed=2)
    c.tables[0, 3] = -1
    c.tables[0, 7] = c.cache.shape[0]
    c.tables[1, :] = np.int32(2 ** 31 - 1)
    y = c.check()
    assert not y[new:].any()


@pytest.mark.parametrize("new", [1, 3, 50])
def test_nan_reaches_only_rows_that_see_it(new):
    c = Case([120, 60], [new, new], 2, 1, 64, 16, "f16", seed=4)
    ref = b16(c.gpu())
    tok = 120 - new // 2 - 1  # seen by the rows from here on
    page, at = c.tables[0, tok // 16], tok % 16
    c.cache[page, 0, block.word_at("vm", 16, 64, at)] = 0x7E00
    got = b16(c.gpu())
    first = tok - (120 - new)
    assert np.isnan(block.decode(got[first:new], "f16")).all()
    assert np.array_equal(got[:first], ref[:first]) or np.abs(
        block.decode(got[:first], "f16") - block.decode(ref[:first], "f16")).max() < 2e-2
    assert np.array_equal(got[new:], ref[new:])


def test_nan_in_a_query_stays_in_its_row():
    c = Case([120, 60], [5, 5], 2, 1, 64, 16, "f16", seed=5)
    ref = c.check()
    c.q[3, 1, 9] = 0x7E00
    got = c.gpu()
    keep = torch.ones_like(ref, dtype=torch.bool)
    keep[3, 1] = False
    assert torch.equal(got[keep], ref[keep]) and bool(got[3, 1].isnan().all())


@pytest.mark.parametrize("dtype,k_size,v_size", [("f16", 1e-5, 1e-5), ("f16", 3000.0, 3000.0),
                                                 ("f16", 300.0, 300.0), ("bf16", 1e-25, 1e-25),
                                                 ("bf16", 1e25, 1e25), ("f16", 40.0, 1.0)])
def test_magnitudes(dtype, k_size, v_size):
    """Scales far from one; scores so large that a row sees one token only."""
    scale = 0.125 / max(k_size, 1.0) if k_size != 40.0 else None
    for new in (1, 40):
        Case([90, 61], [new, new], 4, 2, 64, 16, dtype, seed=6, k_size=k_size, v_size=v_size).check(scale=scale)


def test_large_and_zero_queries():
    for dtype, big in (("f16", 2.0 ** 13), ("bf16", 2.0 ** 60)):
        c = Case([70], [4], 2, 1, 64, 16, dtype, seed=7)
        c.q[0] = 0
        c.q[1] = block.encode(block.decode(c.q[1], dtype) * 2.0 ** -12, dtype)
        c.q[2] = block.encode(block.decode(c.q[2], dtype) * big, dtype)
        c.check(scale=0.01 / big)


def test_out_over_q():
    for lens, new in (([1500], [1]), ([300, 90], [70, 20])):
        c = Case(lens, new, 8, 2, 128, 16, "f16", seed=8)
        ref = c.gpu()
        q = t16(c.q, "f16").to(dev())
        assert torch.equal(c.gpu(q=q, out=q), ref) and torch.equal(q, ref)


def test_workspace_left_zero():
    c = Case([3000, 20], [1, 1], 4, 2, 128, 16, "f16", seed=9)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.gpu()
    s.synchronize()
    ws = awq.ops.WORKSPACE.get
    with torch.cuda.stream(s):
        buf = ws(dev(), 1)
    torch.cuda.synchronize()
    assert not buf.any()


def test_two_streams():
    """Split calls on two unsynchronised streams, each with its own workspace."""
    cases = [Case([2000, 700], [1, 1], 4, 2, 64, 16, "f16", seed=s) for s in (10, 11)]
    ref = [c.gpu() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cases, streams)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i].append(c.gpu())
    torch.cuda.synchronize()
    for r, ys in zip(ref, got):
        assert all(torch.equal(y, r) for y in ys)


def test_append_then_attend_under_a_graph():
    """One decode step (append, then attention) captured and replayed, eager work between; each equal to the eager result."""
    c = Case([700, 90, 33], [1, 1, 1], 8, 2, 128, 16, "f16", seed=12)
    g0 = torch.Generator().manual_seed(1)
    cache = torch.from_numpy(c.cache).to(dev())
    tables, lens = torch.from_numpy(c.tables).to(dev()), torch.from_numpy(c.lens).to(dev())
    pos = lens - 1
    slots = (tables.gather(1, (pos // 16).long()[:, None])[:, 0].long() * 16 + pos % 16)
    qkv = torch.randn(3, 12, 128, generator=g0).half().to(dev())
    x, w = torch.randn(3, 1024, generator=g0).half().to(dev()), torch.ones(1024, dtype=torch.half, device=dev())
    rope = awq.rope_table(1024, 128, device=dev())
    out = torch.empty(3, 8, 128, dtype=torch.half, device=dev())
    qo = torch.empty_like(out)
    a8, s1 = torch.empty(3, 1024, dtype=torch.int8, device=dev()), torch.empty(3, device=dev())
    h = torch.empty_like(x)

    def step():
        awq.rmsnorm_quant(x, w, residual=out.view(3, 1024), residual_out=h, a8=a8, s1=s1)
        q, k, v = qkv.split((8, 2, 2), 1)
        awq.kv4_append(q, k, v, rope, pos, slots, cache, out=qo)
        awq.kv4_attention(qo, cache, tables, lens, max_kv=2048, out=out)

    def results():
        return [t.clone() for t in (out, qo, cache, a8, s1, h)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    out.zero_()
    step()
    torch.cuda.synchronize()
    first = results()
    step()
    torch.cuda.synchronize()
    second = results()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for rep in range(4):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), first)), rep
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), second)), rep
        other = Case([900], [1], 4, 1, 64, 16, "f16", seed=rep)
        other.check()
