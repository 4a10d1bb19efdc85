"""RMS norm with the residual's addition and 8-bit output, against the oracle:
every output bit for bit (h, y, codes, scales, row sums)."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev, orc
from oracle import block

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def b16(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def inputs(M, K, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (size * torch.randn(M, K, generator=g)).to(DT[dtype])
    r = (size * torch.randn(M, K, generator=g) * (1 + 9 * (torch.rand(K, generator=g) < 0.02))).to(DT[dtype])
    return x, r, (1 + 0.2 * torch.randn(K, generator=g)).to(DT[dtype])


def check(x, r, w, eps, dtype, fp8):
    h, y = block.rmsnorm(b16(x), None if r is None else b16(r), b16(w), eps, dtype)
    d = [None if t is None else t.to(dev()) for t in (x, r, w)]
    yo = torch.empty_like(d[0])
    yt = torch.from_numpy(y.view(np.int16).copy()).view(DT[dtype])
    if fp8:
        a, s1, asum, ho = awq.rmsnorm_quant_fp8(d[0], d[2], eps, residual=d[1], y=yo)
        want = orc().quant_act_fp8(yt, dtype == "bf16")
        assert np.array_equal(asum.cpu().numpy(), want[2])
    else:
        a, s1, ho = awq.rmsnorm_quant(d[0], d[2], eps, residual=d[1], y=yo)
        want = orc().quant_act(yt, dtype == "bf16")
    if r is None:
        assert ho is None
    else:
        assert np.array_equal(b16(ho), h)
    assert np.array_equal(b16(yo), y)
    assert np.array_equal(s1.cpu().numpy(), want[1]) and np.array_equal(a.cpu().numpy(), want[0])
    # without y the codes are the same; the norm alone gives the same y
    plain = awq.rmsnorm(d[0], d[2], eps, residual=d[1])
    assert np.array_equal(b16(plain if r is None else plain[0]), y)
    again = (awq.rmsnorm_quant_fp8 if fp8 else awq.rmsnorm_quant)(d[0], d[2], eps, residual=d[1])
    assert torch.equal(again[0], a) and torch.equal(again[1], s1)


@pytest.mark.parametrize("K", [1, 7, 8, 64, 100, 768, 1024, 1032, 2040, 4096, 5120, 8192, 8200, 11008, 14336, 32768,
                               32776, 40001])
@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
def test_norm_matches_oracle(K, dtype, fp8):
    for M, res in ((1, True), (5, False)):
        x, r, w = inputs(M, K, dtype, 10 * K + M)
        check(x, r if res else None, w, 1e-6, dtype, fp8)


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", True)])
def test_norm_many_rows(dtype, fp8):
    x, r, w = inputs(1031, 512, dtype, 3)
    check(x, r, w, 1e-5, dtype, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_norm_extremes(dtype, fp8):
    """All-zero rows, tiny and large values, eps = 0 on a live row, weights of zero."""
    K = 264
    x, r, w = inputs(6, K, dtype, 5)
    x[0], r[0] = 0, 0
    x[1] = (x[1].float() * 1e-6).to(DT[dtype])
    r[1] = 0
    x[2] = (x[2].float() * (1e4 if dtype == "f16" else 1e30)).to(DT[dtype])
    r[3] = -x[3]  # cancels: h = 0
    w[:8] = 0
    check(x, r, w, 1e-6, dtype, fp8)
    check(x[4:], r[4:], w, 0.0, dtype, fp8)
    if dtype == "bf16":  # norms so small that s1 is a subnormal fp32 value
        check(x[4:], r[4:], (w.float() * 1e-37).to(DT[dtype]), 1e-6, dtype, fp8)


def test_norm_nonfinite_row_shows():
    x, r, w = inputs(3, 512, "f16", 6)
    x[1, 77] = float("nan")
    x[2, 3], r[2, 3] = 65504.0, 65504.0
    a, s1, h = awq.rmsnorm_quant(x.to(dev()), w.to(dev()), residual=r.to(dev()))
    torch.cuda.synchronize()
    assert torch.isfinite(s1[0]) and not torch.isfinite(s1[1]) and not torch.isfinite(s1[2])


@pytest.mark.parametrize("K", [640, 4096, 1001])
def test_norm_in_place(K):
    """The residual updated in place, and y over x."""
    x, r, w = inputs(9, K, "f16", 7)
    d = [t.to(dev()) for t in (x, r, w)]
    a, s1, h = awq.rmsnorm_quant(d[0], d[2], residual=d[1])
    r2 = d[1].clone()
    a2, s2, h2 = awq.rmsnorm_quant(d[0], d[2], residual=r2, residual_out=r2)
    assert h2 is r2 and torch.equal(r2, h) and torch.equal(a2, a) and torch.equal(s2, s1)
    y = awq.rmsnorm(d[0], d[2])
    x2 = d[0].clone()
    a3, s3, _ = awq.rmsnorm_quant(d[0], d[2])
    a4, s4, _ = awq.rmsnorm_quant(x2, d[2], y=x2)
    assert torch.equal(x2, y) and torch.equal(a3, a4) and torch.equal(s3, s4)


def test_norm_feeds_the_layer():
    """The codes go into the W4A8 product as the quantiser's do."""
    import synthgen
    c = synthgen.w4a8_case(33, 1024, 256, -1)
    b, s2 = c.b.to(dev()), c.s2.to(dev())
    x, r, w = inputs(33, 1024, "f16", 8)
    d = [t.to(dev()) for t in (x, r, w)]
    a8, s1, h = awq.rmsnorm_quant(d[0], d[2], residual=d[1])
    y, h2 = awq.rmsnorm(d[0], d[2], residual=d[1])
    assert torch.equal(h, h2)
    assert torch.equal(awq.w4a8_gemm(a8, b, s1, s2), awq.linear_w4a8(y, b, s2))
