"""Value scales far from each other in one call of the attention over the 4-bit
cache: what a row does not see, or sees with next to no probability, must not
cost it bits, whichever kernel the call takes.

Bound on each output element, from the roundings the header states (u = half a
step of the type): the output's own, u |y|; the softmax numerators' one to 11
bits, 2^-11 sum p |v|, and for those below 2^-19 of the row's largest 2^-30 of
that largest, each times a code of up to 15; the scores', which move p by twice
their error: 2^-24 a term for the sums of D products of codes up to 15 and of
the zero points' part (2 * 15 sum |q| s scale, over D + 32 roundings); exp2's
two units; and the fp32 sums, n / 4 + 256 roundings of terms up to 30 s' each.
Everything in it is the row's own: tokens it does not see have no part in it."""
import numpy as np
import pytest

from gpu_helpers import dev  # noqa: F401
from oracle import block
from test_gpu_kv4_attention import Case, b16

pytestmark = pytest.mark.gpu
LONG = 131072  # with more than 128 rows: the prompts' kernel, whatever the batch
EXP = {"f16": 10, "bf16": 7}  # where a pattern's exponent starts


def slot_of(c, b, token):
    return int(c.tables[b, token // c.P]), token % c.P


def boost(c, b, token, log2):
    """Token `token` of sequence b: every head's value scale times 2^log2."""
    page, at = slot_of(c, b, token)
    i = block.word_at("vm", c.P, c.D, at)
    c.cache[page, :, i] += np.int32(log2 << EXP[c.dtype])


def check(c, window=0, **kw):
    got = block.decode(b16(c.gpu(window=window, **kw)), c.dtype)
    args = (c.q, c.cache, c.P, c.tables, c.lens, c.cu, c.D ** -0.5, window, c.dtype)
    want, spread, unit = block.attention(*args)
    most, seen, total = np.moveaxis(block.products(*args), 2, 0)[..., None]
    u = 2.0 ** -11 if c.dtype == "f16" else 2.0 ** -8
    n = max(int(c.lens.max()), 1)
    score = 2.0 ** -24 * (c.D + 32) * 30 * unit[..., 1:2]
    bound = (u * np.abs(want) + (1 + u) * ((2.0 ** -11 + 2 * score + 2.0 ** -21) * spread
             + 2.0 ** -24 * (n / 4 + 256) * 30 * total + 2.0 ** -30 * 15 * most * seen)
             + (2.0 ** -25 if c.dtype == "f16" else 0))
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


def case(new, dtype, D, seed):
    # (fp16: so small that a token boosted by 2^20 still fits the type)
    return Case([320, 160], [new, min(new, 160)], 2, 1, D, 16, dtype, seed=seed, v_size=2.0 ** -10)


RATIOS = [("f16", 12), ("f16", 20), ("bf16", 12), ("bf16", 20), ("bf16", 33), ("bf16", 60)]
# rows of each of the kernels: up to four, tiles of 16 rows, the prompts'
NEW = [(2, None), (40, None), (150, LONG)]


@pytest.mark.parametrize("new,max_kv", NEW)
@pytest.mark.parametrize("dtype,log2", RATIOS)
def test_hidden_by_the_diagonal(dtype, log2, new, max_kv):
    for D in (64, 128):
        c = case(new, dtype, D, seed=log2 + D)
        boost(c, 0, 320 - new // 2, log2)
        boost(c, 1, 160 - min(new, 160) // 2, log2)
        check(c, max_kv=max_kv)


@pytest.mark.parametrize("new,max_kv", NEW)
@pytest.mark.parametrize("dtype,log2", RATIOS)
def test_hidden_by_the_window(dtype, log2, new, max_kv):
    """Tokens that leave the window of the later rows."""
    for D in (64, 128):
        c = case(new, dtype, D, seed=log2 + D + 1)
        for t in (320 - new - 30, 320 - new - 49, 320 - new):
            boost(c, 0, t, log2)
        check(c, window=50, max_kv=max_kv)


@pytest.mark.parametrize("new,max_kv", [(1, None), *NEW])
@pytest.mark.parametrize("dtype,log2", RATIOS)
def test_seen_with_next_to_no_probability(dtype, log2, new, max_kv):
    """A token whose key is opposed to every query: its probability is below 2^-80 of the others'."""
    for D in (64, 128):
        c = case(new, dtype, D, seed=log2 + D + 2)
        q = block.decode(c.q, dtype)
        q[..., 0] = 40.0
        c.q = block.encode(q, dtype)
        rng = np.random.default_rng(log2)
        for t in (0, 77, 169):
            k = rng.standard_normal((1, 1, D))
            k[..., 0] = -25.0
            page, at = slot_of(c, 0, t)
            block.store(c.cache, c.P, [page * c.P + at], block.encode(k, dtype),
                        block.encode(rng.standard_normal((1, 1, D)) * 2.0 ** -10, dtype), dtype)
            boost(c, 0, t, log2)
        check(c, max_kv=max_kv)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_first_row_beside_a_loud_second_token(dtype):
    """A whole prompt: row 0 sees token 0 alone, and every other row token 1 too."""
    for log2 in (20,) if dtype == "f16" else (20, 33, 60):
        c = Case([300], [300], 1, 1, 64, 16, dtype, seed=log2, v_size=2.0 ** -10)
        boost(c, 0, 1, log2)
        check(c, max_kv=LONG)


@pytest.mark.parametrize("dtype,step", [("f16", 3), ("bf16", 14)])
def test_scales_that_rise_with_the_tokens(dtype, step):
    """The largest product grows from one tile of 64 tokens to the next, for some rows only."""
    c = Case([320], [200], 2, 1, 64, 16, dtype, seed=step, v_size=2.0 ** -10)
    for t in range(320):
        boost(c, 0, t, step * (t // 64))
    check(c, max_kv=LONG)
    check(c, window=70, max_kv=LONG)


@pytest.mark.parametrize("new,max_kv", [(1, None), *NEW])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("which", ["values", "every third token"])
def test_scales_below_zero(which, dtype, new, max_kv):
    """(code - z) s holds for any s: a cache that something else has filled may have them."""
    for D in (64, 128):
        c = Case([320, 160], [new, min(new, 160)], 2, 1, D, 16, dtype, seed=D + new)
        for b, n in enumerate(c.lens):
            for t in range(0, n, 1 if which == "values" else 3):
                page, at = slot_of(c, b, t)
                c.cache[page, :, block.word_at("vm", 16, D, at)] ^= 0x8000
                if which != "values":
                    c.cache[page, :, block.word_at("km", 16, D, at)] ^= 0x8000
        check(c, max_kv=max_kv)
