"""Sizes past 32-bit offsets, past one axis of a grid and past one workgroup's tokens, against plain torch on the GPU
(rows and sums of it; whole numbers equal, the rest within the types' roundings)."""
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from moe_helpers import HALF_STEP, cuda, e4m3_weights, experts_weights
from oracle import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(300001, 16, 2), (70000, 200, 8), (40000, 1024, 16),
                                   (40000, 1024, 32),  # (more than 64 KB of LDS a workgroup)
                                   (400000, 40, 32)])
def test_route_of_many_tokens(T, E, k):
    g = torch.Generator(device=dev()).manual_seed(T)
    l = torch.randn(T, E, generator=g, device=dev()).half()
    l[torch.rand(T, generator=g, device=dev()) < 0.1] = -torch.inf  # tokens without any expert
    w, ids, offsets, rows, places = awq.moe_route(l, k)
    v, order = torch.sort(l.float(), dim=1, descending=True, stable=True)
    want = torch.where(v[:, :k] > -torch.inf, order[:, :k], -1)
    assert torch.equal(ids.long(), want)
    flat = torch.where(want < 0, E, want).flatten()
    by = torch.sort(flat, stable=True).indices
    n = int((flat < E).sum())
    assert torch.equal(offsets.long(), torch.searchsorted(flat[by], torch.arange(E + 1, device=dev())))
    assert torch.equal(rows[:n].long(), by[:n]) and torch.all(rows[n:] == -1)
    back = torch.full_like(flat, -1)
    back[by[:n]] = torch.arange(n, device=dev())
    assert torch.equal(places.long(), back)
    ref = torch.where(want >= 0, torch.softmax(l.double(), 1).gather(1, want.clamp(min=0)), 0)
    # (E + 1) sums and two exponentials of differences below 12: 12 x 2^-24, 2^-22, (E + 1) 2^-24 of the weight
    assert torch.all((w.double() - ref).abs() <= ref * ((E + 60) * 2.0 ** -24) + 1e-38)


def test_combine_of_many_tokens():
    T, k, N = 140003, 2, 8
    g = torch.Generator(device=dev()).manual_seed(0)
    y = torch.randn(T * k, N, generator=g, device=dev()).half()
    w = torch.rand(T, k, generator=g, device=dev())
    p = torch.randperm(T * k, generator=g, device=dev())
    got = awq.moe_combine(y, w, p.int()).double()
    terms = w.double()[..., None] * y[p].view(T, k, N).double()
    want = terms.sum(1)
    assert torch.all((got - want).abs() <= HALF_STEP["f16"] * want.abs() + 2 * 2.0 ** -24 * terms.abs().sum(1) + 2.0 ** -25)


def test_combine_past_32_bits():
    """y of more than 2^32 bytes."""
    R, N = (1 << 20) + 8, 2056
    y = torch.zeros(R, N, dtype=torch.float16, device=dev())
    y[-3:] = torch.arange(N, device=dev()) % 100 + torch.tensor([[1.0], [2.0], [3.0]], device=dev())
    p = torch.tensor([R - 1, R - 3, 0, R - 2], dtype=torch.int32, device=dev())
    got = awq.moe_combine(y, torch.tensor([[1.0, 2.0], [5.0, 1.0]], device=dev()), p)
    assert torch.equal(got[0].float(), y[-1].float() + 2 * y[-3].float()) and torch.equal(got[1], y[-2])


def test_quant_past_32_bits():
    """Rows in several launches, and more than 2^32 bytes of activations."""
    M, K = (1 << 27) + 77, 16
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev())
    at = torch.tensor([0, 5, (1 << 27) - 1, 1 << 27, M - 1], device=dev())
    x[at] = torch.randn(5, K, generator=torch.Generator().manual_seed(0)).bfloat16().to(dev())
    a, s = awq.quant_act_fp8_block(x)
    codes, scales = moe.block_quant(x[at].cpu().double().numpy())
    assert torch.equal(a[at].cpu(), torch.from_numpy(codes)) and torch.equal(s[at].cpu(), torch.from_numpy(scales))
    assert int((s != 0).sum()) == 5


def test_product_past_32_bits():
    """Codes of more than 2^31 bytes: every tile has a base of its own."""
    M, K, N = 600011, 4096, 64
    w, sw = cuda(*e4m3_weights(0, N, K, 0))
    a = torch.randint(0, 120, (M, K), dtype=torch.uint8, device=dev())
    sa = torch.rand(M, K // 128, device=dev()) * 2.0 ** -9
    got = awq.gemm_fp8_block(a, w, sa, sw)
    rows = torch.tensor([0, 300000, 524287, 524288, M - 1], device=dev())
    v = a[rows].view(torch.float8_e4m3fn).double() * sa[rows].double().repeat_interleave(128, 1)
    m = w.view(torch.float8_e4m3fn).double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    want = v @ m.t()
    assert ((got[rows].double() - want).norm() / want.norm()) <= HALF_STEP["bf16"]


@pytest.mark.parametrize("tokens", [300000])
def test_experts_past_32_bits(tokens):
    """Rows in the plan's order of more than 2^31 bytes; gathered ones are refused past that."""
    K, N, E = 4096, 64, 3
    q, s, z = cuda(*experts_weights(E, K, N, 128, True, "f16", 0))
    x = torch.randn(tokens, K, device=dev(), dtype=torch.float16)
    offsets = torch.tensor([0, 100000, 100001, tokens], dtype=torch.int32, device=dev())
    got = awq.moe_gemm_w4a16(x, q, s, z, offsets)
    rows = [0, 99999, 100000, 100001, 262143, 262144, tokens - 1]
    for r in rows:
        e = 0 if r < 100000 else 1 if r < 100001 else 2
        m = torch.from_numpy(moe.dequant(q[e].cpu().numpy(), s[e].double().cpu().numpy(), z[e].cpu().numpy(), 128)).to(dev())
        want = x[r].double() @ m
        assert (got[r].double() - want).norm() / want.norm() <= 3 * HALF_STEP["f16"], r
    with pytest.raises(awq.AWQError, match="EUNSUPPORTED"):
        awq.moe_gemm_w4a16(x, q, s, z, offsets, rows=torch.arange(tokens, dtype=torch.int32, device=dev()))


@pytest.mark.parametrize("N,R", [(264, 40), (288, 400)])  # the streaming kernels, and tiles through LDS
def test_offsets_that_are_no_plan_leave_the_workspace_zero(N, R):
    from bit_weight_only_awq_amd import ops
    K, E = 4096, 4
    q, s, z = cuda(*experts_weights(E, K, N, 128, True, "f16", 0))
    w, sw = cuda(*e4m3_weights(E, N, K, 0))
    x = torch.randn(R, K, device=dev(), dtype=torch.float16)
    a, sa = awq.quant_act_fp8_block(x)
    assert awq.lib().awq_moe_gemm_w4a16_workspace_bytes(R, E, N, K, 128) > 0
    assert awq.lib().awq_fp8_block_gemm_workspace_bytes(R, E, N, K) > 0
    for off in ([0, 40, 0, 0, 5], [-5, 10, 10, 2, 1 << 30], [0, 40, 0, 40, 0], [7, 7, 3, 39, -1]):
        o = torch.tensor(off, dtype=torch.int32, device=dev())
        awq.moe_gemm_w4a16(x, q, s, z, o)
        awq.moe_gemm_fp8_block(a, w, sa, sw, o)
        torch.cuda.synchronize()
        for buf in ops.WORKSPACE._bufs.values():
            assert not buf.any(), off
