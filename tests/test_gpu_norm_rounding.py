"""RMS norm on rows whose mean square lies so near to the middle between two
binary32 numbers that the sum times a rounded 1 / K falls on the other side of
it from the quotient that the definition asks for, and an output shows it."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev, orc
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def row_of(K, mean, dtype):
    """K values of the type whose squares sum to K * mean exactly, times 2^-12."""
    step = 4 if dtype == "f16" else 64  # of the type's integers from 4096 to 8192 on
    base, total, tail = int(np.sqrt(mean)) // step * step, K * mean, 40
    more = min((total - K * base * base) // ((base + step) ** 2 - base * base), K)
    n = [base + step] * more + [base] * (K - tail - more)
    rest = total - sum(i * i for i in n)
    while rest:
        r = int(np.sqrt(rest))
        drop = max(0, r.bit_length() - (11 if dtype == "f16" else 8))
        n.append(r >> drop << drop)
        rest -= n[-1] ** 2
    assert len(n) <= K and sum(i * i for i in n) == total
    v = np.array(n + [0] * (K - len(n))) * 2.0 ** -12
    bits = block.encode(v, dtype)
    assert np.array_equal(block.decode(bits, dtype), v)
    return bits


def t16(bits, dtype):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(DT[dtype])


@pytest.mark.parametrize("dtype,K,mean,seed", [
    ("f16", 784, 23343267, 9), ("f16", 824, 21474855, 0), ("f16", 6272, 23342635, 16), ("f16", 13696, 24971447, 8),
    ("f16", 41209, 29244307, 13), ("bf16", 784, 23344795, 0), ("bf16", 824, 21476003, 0), ("bf16", 6272, 23344795, 0),
    ("bf16", 13696, 24973467, 0), ("bf16", 41209, 29244423, 0)])
def test_mean_square_beside_a_midpoint(dtype, K, mean, seed):
    x = row_of(K, mean, dtype)
    s = float((block.decode(x, dtype) ** 2).sum())
    assert np.float32(s / K) != np.float32(s * (1.0 / K))
    w = block.encode(1 + 0.2 * np.random.default_rng(seed).standard_normal(K), dtype)
    _, y = block.rmsnorm(x[None], None, w, 0.0, dtype)
    xd, wd = t16(x[None], dtype).to(dev()), t16(w, dtype).to(dev())
    got = torch.empty_like(xd)
    a8, s1, _ = awq.rmsnorm_quant(xd, wd, 0.0, y=got)
    assert np.array_equal(got.cpu().view(torch.int16).numpy().view(np.uint16), y)
    want = orc().quant_act(t16(y, dtype), dtype == "bf16")
    assert np.array_equal(s1.cpu().numpy(), want[1]) and np.array_equal(a8.cpu().numpy(), want[0])
