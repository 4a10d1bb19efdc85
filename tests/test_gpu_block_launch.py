"""More rows and tokens than one launch holds: every piece is the call's own rows."""
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev

pytestmark = pytest.mark.gpu
PIECE = 1 << 21  # rows of a launch


@pytest.mark.parametrize("K,M", [(8, 2 * PIECE + 5), (8, (1 << 25) + 3), (7, PIECE + 9)])
@pytest.mark.parametrize("fp8", [False, True])
def test_norm_of_many_rows(K, M, fp8):
    g = torch.Generator(device=dev()).manual_seed(K)
    x, r = (torch.randn(M, K, generator=g, device=dev(), dtype=torch.half) for _ in range(2))
    w = torch.randn(K, generator=g, device=dev(), dtype=torch.half)
    f = awq.rmsnorm_quant_fp8 if fp8 else awq.rmsnorm_quant
    y = torch.empty_like(x)
    whole = (*f(x, w, residual=r, y=y), y)
    torch.cuda.synchronize()
    last = (M - 1) // PIECE * PIECE
    for a, b in ((0, 40), (PIECE - 24, PIECE), (PIECE, PIECE + 8), (last, M)):  # (starts a multiple of 8: alignment)
        yp = torch.empty_like(x[a:b])
        part = (*f(x[a:b], w, residual=r[a:b], y=yp), yp)
        for s, t in zip(whole, part):
            assert torch.equal(s[a:b].view(torch.uint8), t.view(torch.uint8)), (a, b)


def test_append_of_many_tokens():
    T, hq, hkv, D, P = 2 * PIECE + 130, 1, 1, 64, 1024
    g = torch.Generator(device=dev()).manual_seed(2)
    qkv = torch.randn(T, hq + 2 * hkv, D, generator=g, device=dev(), dtype=torch.half)
    q, k, v = qkv.split((hq, hkv, hkv), 1)
    pos = (torch.arange(T, device=dev()) % 300).int()
    rope = awq.rope_table(300, D, device=dev())
    slots = torch.arange(T, device=dev())
    cache = awq.kv4_cache(-(-T // P), hkv, D, P)
    out = awq.kv4_append(q, k, v, rope, pos, slots, cache)
    for a in range(0, T, PIECE):
        b = min(a + 3000, T)
        small = awq.kv4_cache(3, hkv, D, P)
        got = awq.kv4_append(q[a:b], k[a:b], v[a:b], rope, pos[a:b], slots[a:b] - a, small)
        assert torch.equal(got, out[a:b])
        n = (b - a) // P if b < T else cache.shape[0] - a // P  # (whole pages, and the last one)
        assert n > 0 and torch.equal(small[:n], cache[a // P:a // P + n])
    assert bool((cache[:T // P, 0, -2 * P:] != 0).all()), "a token was not stored"


def test_append_past_2_to_26_tokens():
    """64 threads a token: 2^32 threads and more in all."""
    T, D, P = (1 << 26) + 70, 64, 16
    k = torch.zeros(T, 1, D, device=dev(), dtype=torch.half)
    slots = torch.full((T,), -1, dtype=torch.int64, device=dev())
    k[-20:] = torch.randn(20, 1, D, generator=torch.Generator(device=dev()).manual_seed(3), device=dev()).half()
    k[5] = k[-1]
    slots[-20:] = torch.arange(20, device=dev())
    slots[5] = 31
    cache, near = awq.kv4_cache(2, 1, D, P), awq.kv4_cache(2, 1, D, P)
    awq.kv4_append(None, k, k, None, None, slots, cache)
    keep = torch.cat((torch.arange(T - 20, T), torch.tensor([5]))).to(dev())
    awq.kv4_append(None, k[keep], k[keep], None, None, slots[keep], near)
    assert bool(near.any()) and torch.equal(cache, near)
