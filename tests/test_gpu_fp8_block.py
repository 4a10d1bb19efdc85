"""The block-scaled E4M3 quantiser, bit for bit the oracle's."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from moe_helpers import DT, f64, randn
from oracle import moe

pytestmark = pytest.mark.gpu


def check(x):
    a, s = awq.quant_act_fp8_block(x.to(dev()))
    codes, scales = moe.block_quant(f64(x))
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(moe.decode(a.cpu().numpy()), moe.decode(codes))  # (zeros of either sign)
    return a, s


@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 768, 4096, 4112])
@pytest.mark.parametrize("M", [1, 5, 67])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quant(K, M, dtype):
    check((randn(K + M, M, K) * torch.exp(3 * randn(K, M, 1))).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_value(dtype):
    """Every finite number of the type, in runs whose largest is random: every quotient that can round either way."""
    bits = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16)
    v = bits.view(DT[dtype])
    v = v[torch.isfinite(v.float())]
    g = torch.Generator().manual_seed(0)
    x = torch.stack([v[torch.randperm(len(v), generator=g)][:len(v) // 128 * 128] for _ in range(6)])
    # most runs hold a large number: divide the rest of them down by powers of two as well
    y = (x.double() * torch.exp2(-torch.randint(0, 60, (6, x.shape[1] // 128, 1), generator=g).double())
         .expand(-1, -1, 128).reshape(6, -1)).to(DT[dtype])
    check(x)
    check(y)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_small_numbers(dtype):
    """Runs of zeros, of the smallest numbers, and of those whose scale is below the normal numbers."""
    tiny = torch.tensor([1], dtype=torch.int16).view(DT[dtype])
    x = torch.zeros(64, 256, dtype=DT[dtype])
    for i in range(64):
        x[i, i] = tiny[0] * (i + 1)
        x[i, 255 - i] = -tiny[0]
        x[i, 200 - i] = float(2.0 ** -(60 + i)) if dtype == "bf16" else 0
    check(x)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_not_finite(dtype):
    """A run with a NaN or an infinity makes its row of a product NaN, and no other."""
    x = randn(0, 4, 384).to(DT[dtype])
    x[1, 130], x[2, 383] = torch.nan, -torch.inf
    a, s = awq.quant_act_fp8_block(x.to(dev()))
    ok = torch.ones(4, 3, dtype=torch.bool)
    ok[1, 1] = ok[2, 2] = False
    assert torch.equal(torch.isfinite(s.cpu()), ok)
    assert not a.cpu()[1, 128:256].any() and not a.cpu()[2, 256:].any()
    w = torch.full((64, 384), 0x38, dtype=torch.uint8, device=dev())
    y = awq.gemm_fp8_block(a, w, s, torch.ones(1, 3, device=dev()), dtype=DT[dtype]).cpu()
    assert torch.equal(torch.isnan(y).all(1), ~ok.all(1)) and torch.isfinite(y[[0, 3]]).all()


def test_many_rows():
    """More runs than one workgroup has, and rows in pieces are the rows alone."""
    x = randn(1, 3001, 272).to(torch.float16)
    a, s = check(x)
    b, t = awq.quant_act_fp8_block(x[2000:2003].to(dev()))
    assert torch.equal(a[2000:2003], b) and torch.equal(s[2000:2003], t)


def test_refusals():
    x = torch.zeros(4, 128, dtype=torch.float16, device=dev())
    for bad in (lambda: awq.quant_act_fp8_block(x.float()), lambda: awq.quant_act_fp8_block(x[:, ::2]),
                lambda: awq.quant_act_fp8_block(x[0]), lambda: awq.quant_act_fp8_block(x, a=x),
                lambda: awq.quant_act_fp8_block(x, s=torch.zeros(4, 2, device=dev()))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(awq.AWQError, match="EINVAL"):
        awq.quant_act_fp8_block(x[:, :120].contiguous())
