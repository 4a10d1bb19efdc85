"""Inputs and bounds of the mixture-of-experts and block-scaled E4M3 tests."""
from __future__ import annotations

import numpy as np
import torch

from gpu_helpers import dev

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # relative, of a rounding to the type


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def split_rows(counts):
    """offsets of experts with so many rows each."""
    return torch.tensor([0, *counts], dtype=torch.int64).cumsum(0).to(torch.int32)


def within(got, want, size, per_size, dtype, what=""):
    """|got - want| <= half a step of the output's type + per_size of the sum of magnitudes, elementwise.  (What
    overflows the type, or is below its normal numbers, is not among the tests' values but for zeros.)"""
    g = f64(got)
    assert g.shape == want.shape
    bound = HALF_STEP[dtype] * np.abs(want) + per_size * size * (1 + HALF_STEP[dtype]) + 2.0 ** -25
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: " \
                          f"{g[bad][0]} for {want[bad][0]}"


def rel(got, want):
    n = np.linalg.norm(want)
    return np.linalg.norm(f64(got) - want) / (n if n else 1)


def experts_weights(E, K, N, G, zeros, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def words(*shape):
        return torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, dtype=torch.int64).to(torch.int32)

    s = ((0.5 + torch.rand(E, K // G, N, generator=g)) / (4.6 * K ** 0.5)).to(DT[dtype])
    return words(E, K, N // 8), s, words(E, K // G, N // 8) if zeros else None


def e4m3_weights(E, N, K, seed):
    """Random finite codes with scales a factor of 16 apart: lead dimension E, or none for E = 0."""
    g = torch.Generator().manual_seed(seed)
    lead = (E,) if E else ()
    w = torch.randint(0, 254, (*lead, N, K), generator=g, dtype=torch.int64)
    w = (w + (w >= 127)).to(torch.uint8)  # (127 and 255 are NaN)
    s = torch.exp2(4 * torch.rand(*lead, -(-N // 128), -(-K // 128), generator=g)) / (300 * K ** 0.5)
    return w, s


def cuda(*ts):
    return [None if t is None else t.to(dev()) for t in ts]
