"""Rotary append into the 4-bit paged cache, against the oracle: the rotated
queries and every word of the cache bit for bit."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def b16(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def run(T, hq, hkv, D, P, rot, inter, dtype, seed=0, fused=True, spread=1.0, pages=None, slots=None, positions=None,
        edit=None):
    g = torch.Generator().manual_seed(seed)
    qkv = (spread * torch.randn(T, hq + 2 * hkv, D, generator=g)).to(DT[dtype])
    if edit:
        edit(qkv)
    pages = pages or -(-T // P) + 2
    if slots is None:
        slots = torch.randperm(pages * P, generator=g)[:T]
    if positions is None:
        positions = torch.randint(0, 5000, (T,), generator=g).to(torch.int32)
    rope = awq.rope_table(5000, rot, device="cpu") if rot else None
    start = torch.randint(-2 ** 31, 2 ** 31, (pages, hkv, block.head_words(D, P)), generator=g).to(torch.int32)
    cache = start.to(dev())
    x = qkv.to(dev())
    q, k, v = x.split((hq, hkv, hkv), 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    out = awq.kv4_append(q if hq else None, k, v, None if rope is None else rope.to(dev()), positions.to(dev()),
                         slots.to(dev()), cache, interleaved=inter)
    want = start.numpy().copy()
    hq_, hk_, hv_ = (b16(t) for t in qkv.split((hq, hkv, hkv), 1))
    qw = block.append(hq_.copy() if hq else None, hk_, hv_, None if rope is None else rope.numpy(), positions.numpy(),
                      slots.numpy(), want, P, inter, dtype)
    if hq:
        assert np.array_equal(b16(out), qw)
    else:
        assert out is None
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hkv,D,P,rot,inter", [
    (1, 1, 1, 64, 16, 64, False), (1, 32, 8, 128, 16, 128, False), (3, 32, 8, 128, 64, 128, True),
    (17, 7, 1, 128, 32, 64, False), (64, 12, 12, 64, 16, 32, True), (5, 4, 2, 128, 1024, 16, False),
    (33, 9, 3, 64, 128, 16, True), (2, 0, 5, 64, 16, 64, False), (7, 28, 4, 128, 16, 0, False),
    (130, 1, 1, 64, 256, 48, False)])
def test_append_matches_oracle(T, hq, hkv, D, P, rot, inter, dtype):
    run(T, hq, hkv, D, P, rot, inter, dtype, seed=T + D)
    run(T, hq, hkv, D, P, rot, inter, dtype, seed=T + D + 1, fused=False)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-7, 1e-4, 300.0, 2e4])
def test_append_magnitudes(dtype, size):
    """Scales from fp16's subnormal range to near its largest value."""
    run(40, 2, 2, 64, 16, 64, False, dtype, spread=size if dtype == "f16" else size ** 5, seed=4)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_special_heads(dtype):
    """Zero heads, one-sided heads, NaN and infinities of both signs, exact ties."""
    def edit(x):  # heads 0-1 queries, 2-3 keys, 4-5 values; no rotation
        x[0, 2:] = 0
        x[1, 2:] = x[1, 2:].abs()
        x[2, 2:] = -x[2, 2:].abs()
        x[3, 2, 5], x[3, 5, 0] = float("nan"), float("inf")
        x[4, 4, 63], x[4, 3, 1] = float("-inf"), -float("nan")
        x[5, 2:] = (torch.arange(64) % 31 * 0.5 - 7.5).to(x.dtype)  # range 15: s = 1, every second value a tie
        x[6, 4] = 0
        x[6, 4, 7] = 2.0 ** -24 if x.dtype == torch.float16 else 2.0 ** -133
        x[7, 2:] = x[7, 2:] * 0 + 1.5
        x[8, 2:] = -0.0
    run(9, 2, 2, 64, 16, 0, False, dtype, edit=edit, seed=5)


def test_append_skips_bad_slots_and_positions():
    slots = torch.tensor([-1, 3, 80, 2 ** 40, 17, 40, -2 ** 50, 79])
    pos = torch.tensor([0, 1, 2, 3, -1, 5000, 4, 4999], dtype=torch.int32)
    run(8, 3, 2, 64, 16, 32, False, "f16", pages=5, slots=slots, positions=pos, seed=6)
    run(8, 3, 2, 128, 16, 128, True, "bf16", pages=5, slots=slots, positions=pos, seed=7)


def test_append_in_place_and_single_token_view():
    """q_out = q, and a one-token slice of a longer tensor (whose token stride says nothing)."""
    g = torch.Generator().manual_seed(8)
    q, k, v = ((torch.randn(6, h, 128, generator=g)).half().to(dev()) for h in (8, 2, 2))
    rope = awq.rope_table(64, 128, device=dev())
    pos = torch.arange(6, dtype=torch.int32, device=dev())
    slots = torch.arange(6, device=dev())
    c1, c2 = awq.kv4_cache(1, 2, 128, 16), awq.kv4_cache(1, 2, 128, 16)
    out = awq.kv4_append(q, k, v, rope, pos, slots, c1)
    for t in range(6):
        got = awq.kv4_append(q[t:t + 1], k[t:t + 1], v[t:t + 1], rope, pos[t:t + 1], slots[t:t + 1], c2)
        assert torch.equal(got[0], out[t])
    assert torch.equal(c1, c2)
    assert awq.kv4_append(q, k, v, rope, pos, slots, c2, out=q) is q
    assert torch.equal(q, out)


def test_append_far_slots():
    """Slots past 2^31 words and bytes of the pool."""
    P, hkv, D = 1024, 8, 128
    words = hkv * block.head_words(D, P)
    pages = (5 << 30) // words  # 20 GiB
    cache = torch.empty(pages, hkv, block.head_words(D, P), dtype=torch.int32, device=dev())
    assert cache.numel() > 2 ** 32
    near = awq.kv4_cache(2, hkv, D, P)
    g = torch.Generator().manual_seed(9)
    k, v = torch.randn(4, hkv, D, generator=g).half().to(dev()), torch.randn(4, hkv, D, generator=g).half().to(dev())
    place = torch.tensor([0, 1023, 5, 514], device=dev())
    cache[pages - 1].zero_()
    cache[pages - 2].zero_()
    page = torch.tensor([0, 0, 1, 1], device=dev())
    awq.kv4_append(None, k, v, None, None, (pages - 2 + page) * P + place, cache)
    awq.kv4_append(None, k, v, None, None, page * P + place, near)
    assert torch.equal(cache[pages - 2:], near)
    # ... and read back from there
    q = torch.randn(1, 8, D, generator=g).half().to(dev())
    tab = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device=dev())
    lens = torch.tensor([2 * P - 500], dtype=torch.int32, device=dev())
    assert torch.equal(awq.kv4_attention(q, cache, tab, lens), awq.kv4_attention(q, near, tab - (pages - 2), lens))
