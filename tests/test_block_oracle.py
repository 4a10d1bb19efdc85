"""Pins of the numpy oracle of the norm, the rotary append and the 4-bit
attention (oracle/block.py) against hand-derived words and independent sums,
and planted mistakes in it that the pins have to catch.  CPU only."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block


def bits(v, dtype):
    t = torch.tensor(v, dtype=torch.float16 if dtype == "f16" else torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def values(b, dtype):
    t = torch.from_numpy(np.asarray(b).view(np.int16).copy())
    return t.view(torch.float16 if dtype == "f16" else torch.bfloat16).double().numpy()


def pin_formats():
    for dtype in ("f16", "bf16"):
        all_bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
        assert np.array_equal(block.decode(all_bits, dtype), values(all_bits, dtype), equal_nan=True)
        rng = np.random.default_rng(1)
        f = (rng.standard_normal(20000) * 10.0 ** rng.integers(-9, 5, 20000)).astype(np.float32)
        t = torch.from_numpy(f).to(torch.float16 if dtype == "f16" else torch.bfloat16)
        assert np.array_equal(block.encode(f, dtype), t.view(torch.int16).numpy().view(np.uint16))


def pin_norm_by_hand():
    # h = (3, 4): mean square 12.5, + eps 3.5 = 16, q = 1/4; y = (3/4, 2 * 4/4)
    h, y = block.rmsnorm(bits([[1.0, 5.0]], "f16"), bits([[2.0, -1.0]], "f16"), bits([1.0, 2.0], "f16"), 3.5, "f16")
    assert values(h, "f16").tolist() == [[3.0, 4.0]] and values(y, "f16").tolist() == [[0.75, 2.0]]


def pin_norm_random():
    rng = np.random.default_rng(2)
    for dtype, tol in (("f16", 2.0 ** -11), ("bf16", 2.0 ** -8)):
        x, r = bits(rng.standard_normal((3, 40)), dtype), bits(rng.standard_normal((3, 40)), dtype)
        w = bits(1 + 0.1 * rng.standard_normal(40), dtype)
        h, y = block.rmsnorm(x, r, w, 1e-5, dtype)
        hv = values(h, dtype)
        assert np.all(np.abs(hv - values(x, dtype) - values(r, dtype)) <= tol * np.abs(hv) + 1e-12)
        want = hv / np.sqrt((hv ** 2).mean(1, keepdims=True) + 1e-5) * values(w, dtype)
        # one rounding of y, and four of binary32 before it
        assert np.all(np.abs(values(y, dtype) - want) <= (tol + 5 * 2.0 ** -24) * np.abs(want) + 1e-7)


def pin_rotation():
    # a quarter turn: (x1, x2) -> (-x2, x1)
    x = bits([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]], "f16")
    cs = np.array([[0.0, 0.0, 1.0, 1.0]], dtype=np.float32)
    assert values(block.rotate(x, cs, False, "f16"), "f16").tolist() == [[[-3.0, -4.0, 1.0, 2.0, 5.0, 6.0]]]
    assert values(block.rotate(x, cs, True, "f16"), "f16").tolist() == [[[-2.0, 1.0, -4.0, 3.0, 5.0, 6.0]]]
    # any turn keeps a pair's length, and turns by p then by q as by p + q
    rng = np.random.default_rng(3)
    v = rng.standard_normal((2, 3, 32))
    ang = rng.uniform(-3, 3, (2, 16))
    for inter in (False, True):
        r = values(block.rotate(bits(v, "f16"), np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32), inter,
                                "f16"), "f16")
        a = np.arange(0, 32, 2) if inter else np.arange(16)
        b = a + (1 if inter else 16)
        want = (v[..., a] + 1j * v[..., b]) * np.exp(1j * ang)[:, None]
        assert np.abs(r[..., a] + 1j * r[..., b] - want).max() < 6e-3  # two fp16 roundings of values below 4


def pin_quantiser_by_hand():
    # range -3 .. 12: s = 1, z = 3; half-way 0.5 and 1.5 round to even (0, 2)
    x = bits([[-3.0, 12.0, 0.0, 0.5, 1.5, -0.5, 2.5, 7.0]], "f16")
    c, s, z = block.quantise(x, "f16")
    assert values(s, "f16").tolist() == [1.0] and z.tolist() == [3]
    assert c.tolist() == [[0, 15, 3, 3, 5, 3, 5, 10]]
    # nibbles 0..7 hold columns 0 2 4 6 1 3 5 7: codes 0 3 5 5 15 3 3 10
    assert block.pack(c).view(np.uint32).tolist() == [[0xA33F5530]]
    # all positive: the range starts at 0; all negative: z = 15
    c, s, z = block.quantise(bits([[15.0, 30.0]], "f16"), "f16")
    assert (values(s, "f16")[0], z[0], c[0].tolist()) == (2.0, 0, [8, 15])
    c, s, z = block.quantise(bits([[-15.0, -30.0]], "f16"), "f16")
    assert (values(s, "f16")[0], z[0], c[0].tolist()) == (2.0, 15, [7, 0])
    c, s, z = block.quantise(bits([[0.0, 0.0], [2.0 ** -24, 0.0]], "f16"), "f16")
    assert s.tolist() == [0, 0] and c.tolist() == [[0, 0], [0, 0]] and z.tolist() == [0, 0]
    c, s, z = block.quantise(bits([[float("nan"), 1.0], [float("inf"), 1.0]], "bf16"), "bf16")
    assert s.tolist() == [0x7F81, 0x7F81] and not c.any() and not z.any()


def pin_quantiser_error():
    rng = np.random.default_rng(4)
    for dtype, eps in (("f16", 2.0 ** -11), ("bf16", 2.0 ** -8)):
        x = bits(rng.standard_normal((50, 128)) * 10.0 ** rng.uniform(-3, 3, (50, 1)), dtype)
        c, s, z = block.quantise(x, dtype)
        v, sv = values(x, dtype), values(s, dtype)
        back = (c - z[:, None]) * sv[:, None]
        # half a step inside the range; its ends move by z's rounding (half a step) and s's (eps of 15 steps)
        assert np.all(np.abs(back - v) <= sv[:, None] * (1.0 + 15 * eps) + 1e-12)
        assert np.mean(np.abs(back - v) <= sv[:, None] * 0.501) > 0.97


def pin_cache_words():
    P, D = 16, 64
    assert block.head_words(D, P) == 16 * 18
    # K token 3 word 5; V token 6 word 2: block 1, column 2, place 2; metas after both
    assert block.word_at("k", P, D, 3, 5) == 29 and block.word_at("v", P, D, 6, 2) == 128 + 1 * 32 + 2 * 4 + 2
    assert block.word_at("km", P, D, 7) == 256 + 7 and block.word_at("vm", P, D, 7) == 256 + 16 + 7
    rng = np.random.default_rng(5)
    cache = np.zeros((3, 2, block.head_words(D, P)), dtype=np.int32)
    k, v = bits(rng.standard_normal((4, 2, D)), "f16"), bits(rng.standard_normal((4, 2, D)), "f16")
    slots = [2 * P + 6, 0, -1, 3 * P]
    block.store(cache, P, slots, k, v, "f16")
    assert not cache[1].any()
    for t, (page, tok) in ((0, (2, 6)), (1, (0, 0))):
        for h in range(2):
            K, V, ks, vs = block.page_values(cache, P, D, page, h, "f16")
            for got, src, s in ((K, k, ks), (V, v, vs)):
                assert np.abs(got[tok] - values(src[t, h], "f16")).max() <= 1.02 * s[tok]
                assert not got[np.arange(P) != tok].any()


def pin_attention_brute_force():
    P, D, dtype = 16, 64, "f16"
    rng = np.random.default_rng(6)
    cache = np.zeros((4, 1, block.head_words(D, P)), dtype=np.int32)
    tables = np.array([[3, 1], [2, -1]])
    lens, cu = np.array([19, 3]), np.array([0, 2, 7])  # the second has 5 new tokens but 3 in all: two see nothing
    for b in range(2):
        slots = [tables[b, t // P] * P + t % P for t in range(lens[b])]
        block.store(cache, P, slots, bits(rng.standard_normal((lens[b], 1, D)), dtype),
                    bits(rng.standard_normal((lens[b], 1, D)), dtype), dtype)
    q = bits(rng.standard_normal((7, 2, D)), dtype)
    for window in (0, 4):
        out, _, _ = block.attention(q, cache, P, tables, lens, cu, 0.25, window, dtype)
        for b in range(2):
            for i in range(cu[b + 1] - cu[b]):
                p = lens[b] - (cu[b + 1] - cu[b]) + i
                for e in range(2):
                    num, den = [0.0] * D, 0.0
                    for t in range(max(0, p - window + 1) if window else 0, p + 1):
                        K, V, _, _ = block.page_values(cache, P, D, tables[b, t // P], 0, dtype)
                        qrow = values(q[cu[b] + i, e], dtype)
                        dot = sum(Fraction(a) * Fraction(c) for a, c in zip(qrow, K[t % P]))
                        w = np.exp(0.25 * float(dot))
                        den += w
                        num = [x + w * y for x, y in zip(num, V[t % P])]
                    want = np.array(num) / den if den else np.zeros(D)
                    assert np.allclose(out[cu[b] + i, e], want, rtol=1e-10, atol=1e-12), (b, i, e)


PINS = [pin_formats, pin_norm_by_hand, pin_norm_random, pin_rotation, pin_quantiser_by_hand, pin_quantiser_error,
        pin_cache_words, pin_attention_brute_force]


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_pin(pin):
    pin()


MUTANTS = {
    "residual_dropped": ("fl32(decode(h, dtype) + decode(residual, dtype))", "fl32(decode(h, dtype))"),
    "mean_not_sum": ("/ hv.shape[1]", "/ 1.0"),
    "eps_dropped": ("mean + np.float64(np.float32(eps))", "mean"),
    "weight_dropped": ("fl32(hv * q) * decode(weight, dtype)[None, :]", "fl32(hv * q)"),
    "turn_backwards": ("fl32(fl32(a * c) - fl32(b * s))", "fl32(fl32(a * c) + fl32(b * s))"),
    "layouts_swapped": ("np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)",
                        "np.arange(rot // 2) if interleaved else np.arange(0, rot, 2)"),
    "range_without_zero": ("np.minimum(v.min(axis=-1), 0.0)", "v.min(axis=-1)"),
    "sixteen_steps": ("fl32(hi - lo) / 15.0", "fl32(hi - lo) / 16.0"),
    "zero_point_sign": ("np.rint(fl32(v / d[..., None])) + z[..., None]", "np.rint(fl32(v / d[..., None])) - z[..., None]"),
    "order": ("ORDER = (0, 2, 4, 6, 1, 3, 5, 7)", "ORDER = (0, 1, 2, 3, 4, 5, 6, 7)"),
    "value_words_like_keys": ("(token // 4) * (D // 8) * 4 + j * 4 + token % 4", "token * (D // 8) + j"),
    "metas_swapped": ('(P if kind == "vm" else 0)', '(0 if kind == "vm" else P)'),
    "causal_off_by_one": ("seen = there & (j <= p)", "seen = there & (j < p)"),
    "window_off_by_one": ("seen &= j > p - window", "seen &= j >= p - window"),
    "aligned_to_the_start": ("p = length - n + i", "p = i"),
    "scale_dropped": ("t = scale * (K[seen] @ row)", "t = K[seen] @ row"),
    "zero_point_dropped": ("(c - (u >> 16).astype(np.int64)[:, None]) * s[:, None]", "c * s[:, None]"),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_mutant_is_caught(name, monkeypatch):
    old, new = MUTANTS[name]
    src = open(block.__file__).read()
    assert src.count(old) == 1, f"mutation site for {name} not found exactly once"
    mutant = type(block)("block_mutant")
    exec(compile(src.replace(old, new), "block_mutant", "exec"), mutant.__dict__)
    monkeypatch.setitem(globals(), "block", mutant)
    for pin in PINS:
        try:
            pin()
        except Exception:
            return
    pytest.fail(f"no pin catches {name}")
