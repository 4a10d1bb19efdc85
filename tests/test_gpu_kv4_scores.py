"""Attention over the 4-bit cache at scores where binary32 has no fractions left.

A score's error is 2^-24 a term for the sums of D products of codes up to 15 and
of the zero points' part: 30 sum |q| s scale, over D + 32 roundings.  A row whose
best score is ahead of the next by twice that, and 40, is the value of its best
token, to the roundings of the output and of the numerators; rows without such
a lead are left out.  From 2^25 on (times log2 e) a row is NaN: it is never
finite and wrong."""
import numpy as np
import pytest

from oracle import block
from test_gpu_kv4_attention import Case, b16

pytestmark = pytest.mark.gpu
LONG = 131072  # with more than 128 rows: the prompts' kernel
LOG2E = 1.4426950408889634
KERNELS = [(1, None), (40, None), (150, LONG)]


def check(c, scale, **kw):
    got = block.decode(b16(c.gpu(scale=scale, **kw)), c.dtype)
    u = 2.0 ** -11 if c.dtype == "f16" else 2.0 ** -8
    sums = 2.0 ** -24 * (int(c.lens.max()) / 4 + 256) * 30
    sure, scale = 0, float(np.float32(scale))
    for r, e, row, t, _, V, ks, vs in block._rows(c.q, c.cache, c.P, c.tables, c.lens, c.cu, scale, 0, c.dtype):
        t, out = t * LOG2E, got[r, e]
        first = int(t.argmax())
        error = 2.0 ** -24 * (c.D + 32) * 30 * scale * ks.max() * np.abs(row).sum() * LOG2E
        lead = t[first] - np.sort(t)[-2] if len(t) > 1 else np.inf
        if np.abs(t[first]) > 2.0 ** 25.2:
            assert np.isnan(out).all(), (r, e)
        elif np.abs(t[first]) < 2.0 ** 24.8:
            assert np.isfinite(out).all(), (r, e)
            if lead > 2 * error + 40:
                # (the others' weights together are below n 2^-40)
                v, rest = V[first], len(t) * 2.0 ** -40 * np.abs(V).max()
                assert (np.abs(out - v) <= (u + 2.0 ** -11 + 2.0 ** -20) * np.abs(v) + sums * vs[first] + rest
                        + (2.0 ** -25 if c.dtype == "f16" else 0)).all(), (r, e)
                sure += 1
    return sure


@pytest.mark.parametrize("new,max_kv", KERNELS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scores_up_to_the_limit_and_past_it(dtype, new, max_kv):
    for D in (64, 128):
        c = Case([260, 170], [new, new], 2, 1, D, 16, dtype, seed=D + new)
        sure = 0
        for log2 in (14, 18, 20, 22, 24, 26, 28, 30, 34, 60):  # (of the scale; scores before it are some 2^4)
            sure += check(c, 2.0 ** (log2 - 4), max_kv=max_kv)
        assert sure > c.q.shape[0] * c.hq


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("new,max_kv", KERNELS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_far_scores_of_some_tokens(dtype, new, max_kv, sign):
    """Tokens at -2^27 beside ordinary ones change nothing; at 2^27 they make the rows that see them NaN."""
    L, D = 460, 64
    c = Case([L], [new], 2, 1, D, 16, dtype, seed=new)
    q = block.decode(c.q, dtype)
    q[..., 0] = 2.0 ** 12
    c.q = block.encode(q, dtype)
    rng = np.random.default_rng(new)
    for t in range(L):
        k = rng.standard_normal((1, 1, D))
        k[..., 0] = 0
        # (the first tokens, whole tiles of them, and some among the others)
        if t < 200 and sign < 0 or t % 37 == 5 and (sign < 0 or t > L - new // 2):
            k[..., 0] = sign * 2.0 ** 15
        page = int(c.tables[0, t // 16])
        block.store(c.cache, 16, [page * 16 + t % 16], block.encode(k, dtype),
                    block.encode(rng.standard_normal((1, 1, D)), dtype), dtype)
    got = block.decode(b16(c.gpu(scale=1.0, max_kv=max_kv)), dtype)
    args = (c.q, c.cache, c.P, c.tables, c.lens, c.cu, 1.0, 0, dtype)
    want, spread, unit = block.attention(*args)
    near = np.zeros(want.shape[:2], dtype=bool)
    sq = np.zeros(want.shape[:2])
    for r, e, row, _, _, _, ks, _ in block._rows(*args):
        quiet = ks < 100  # (a token at 2^27 has a scale of 2^15 / 15)
        near[r, e] = sign < 0 or quiet.all()
        sq[r, e] = ks[quiet].max() * np.abs(row).sum()
    u = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    most, seen, total = np.moveaxis(block.products(*args), 2, 0)[..., None]
    score = 2.0 ** -24 * (D + 32) * 30 * sq[..., None]
    bound = (u * np.abs(want) + (1 + u) * ((2.0 ** -11 + 2 * score + 2.0 ** -21) * spread
             + 2.0 ** -24 * (L / 4 + 256) * 30 * total + 2.0 ** -30 * 15 * most * seen)
             + (2.0 ** -25 if dtype == "f16" else 0))
    assert near.any() and not (~(np.abs(got - want) <= bound))[near].any()
    assert np.isnan(got[~near]).all()
