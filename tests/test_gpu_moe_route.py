"""Routing and the weighted sum, against the oracle: the plan equal, the weights and sums within their roundings."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from moe_helpers import DT, f64, randn, within
from oracle import moe

pytestmark = pytest.mark.gpu


def check(logits, k, renormalize):
    l = f64(logits)
    T, E = l.shape
    got = [t.cpu() for t in awq.moe_route(logits.to(dev()), k, renormalize=renormalize)]
    ids, w = moe.choose(l, k, renormalize)
    offsets, rows, places = moe.plan(ids, E)
    assert np.array_equal(got[1].numpy(), ids)
    assert np.array_equal(got[2].numpy(), offsets)
    assert np.array_equal(got[3].numpy(), rows) and np.array_equal(got[4].numpy(), places)
    # l - m is rounded (up to |l - m| 2^-24 in the exponent: that times the weight), exp is good to two units (2^-22),
    # a sum of n such terms adds n 2^-24 of itself, the quotient half a unit; below 2^-126 values may be lost
    spread = np.minimum(np.where(np.isfinite(l), np.abs(l), 0).max(initial=0) * 2, 110)
    bound = w * (2 * spread * 2.0 ** -24 + 2 * 2.0 ** -22 + (E + 1) * 2.0 ** -24) + 2.0 ** -125
    assert np.all(np.abs(f64(got[0]) - w) <= bound), np.abs(f64(got[0]) - w).max()
    return got


@pytest.mark.parametrize("E,k", [(1, 1), (3, 2), (8, 2), (8, 8), (9, 3), (16, 4), (31, 6), (33, 8), (60, 4), (64, 8),
                                 (65, 32), (128, 8), (200, 5), (256, 8), (300, 2), (512, 10), (513, 3), (1000, 8),
                                 (1024, 32)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_route(E, k, dtype):
    for i, T in enumerate((1, 7, 16, 17, 130)):
        # (16-bit logits of this size repeat among the experts: ties)
        check((2 * randn(100 * E + T, T, E)).to(DT[dtype]), k, bool(i % 2))


@pytest.mark.parametrize("T", [0, 1, 15, 255, 256, 4095, 4097, 9000])
def test_route_tokens(T):
    got = check(randn(T, T, 16).to(torch.float16), 2, True)
    assert int(got[2][-1]) == 2 * T


@pytest.mark.parametrize("T", [3, 40, 700])
@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (130, 8), (600, 4)])
def test_route_masks(T, E, k):
    """Rows of minus infinity, of NaN, with fewer experts than choices, of the lowest number, of infinities, of equal
    logits and of zeros of both signs."""
    l = randn(E + T, T, E)
    g = torch.Generator().manual_seed(T)
    for t in range(T):
        kind = t % 9
        if kind == 1:
            l[t] = -torch.inf
        elif kind == 2:
            l[t] = torch.nan
        elif kind == 3:
            l[t, torch.rand(E, generator=g) < 0.95] = -torch.inf
        elif kind == 4:
            l[t, torch.rand(E, generator=g) < 0.9] = torch.finfo(torch.float32).min
        elif kind == 5:
            l[t, torch.rand(E, generator=g) < 0.2] = torch.inf
        elif kind == 6:
            l[t] = 1.5
        elif kind == 7:
            l[t] = torch.where(torch.rand(E, generator=g) < 0.5, -0.0, 0.0)
        elif kind == 8:
            l[t, torch.rand(E, generator=g) < 0.5] = torch.nan
    for renormalize in (False, True):
        check(l, k, renormalize)


@pytest.mark.parametrize("T", [0, 1, 2, 3])
def test_few_tokens_of_many_experts(T):
    check(randn(T, T, 700), 8, False)


def test_all_tokens_of_one_expert():
    l = torch.full((3000, 40), -torch.inf)
    l[:, 17] = 0
    got = check(l, 4, False)
    assert int(got[2][18]) == 3000 and torch.equal(got[3][:3000], 4 * torch.arange(3000, dtype=torch.int32))


def test_route_into_given_tensors():
    l = randn(5, 50, 24).to(dev())
    new = awq.moe_route(l, 3)
    out = tuple(torch.full_like(t, 77) for t in new)
    assert awq.moe_route(l, 3, out=out) is out
    for a, b in zip(new, out):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        awq.moe_route(l, 4, out=out)


@pytest.mark.parametrize("N", [8, 96, 2048, 2056, 4096])
@pytest.mark.parametrize("k", [1, 2, 3, 8, 11])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_combine(N, k, dtype):
    for T in (1, 37):
        R = T * k
        y = randn(N + k, R, N).to(DT[dtype])
        w = torch.rand(T, k, generator=torch.Generator().manual_seed(k))
        p = torch.randperm(R, generator=torch.Generator().manual_seed(N)).to(torch.int32)
        p[::5] = -1
        p[3::7] = R + 3
        if k > 1:
            p[:k] = -1  # a token without any expert: 0
        y[int(p.clamp(0, R - 1)[-1]), 0] = 0
        got = awq.moe_combine(y.to(dev()), w.to(dev()), p.to(dev()))
        want, size = moe.combine(f64(y), f64(w), p.numpy())
        within(got, want, size, k * 2.0 ** -24, dtype)
        if k > 1:
            assert not got[0].any()


def test_combine_reads_only_its_rows():
    """What stands in rows that no place names, or under a place that is none, does not reach the sum."""
    y = torch.full((6, 16), torch.nan, dtype=torch.float16)
    y[2], y[4] = 1, 2
    w = torch.tensor([[0.5, torch.nan], [0.25, 0.5]])
    got = awq.moe_combine(y.to(dev()), w.to(dev()), torch.tensor([2, -1, 4, 2], dtype=torch.int32, device=dev()))
    assert torch.equal(got.cpu(), torch.tensor([[0.5], [1.0]], dtype=torch.float16).expand(2, 16))


def test_refusals():
    l = torch.zeros(4, 8, device=dev())
    y, w = torch.zeros(8, 64, dtype=torch.float16, device=dev()), torch.zeros(4, 2, device=dev())
    p = torch.zeros(8, dtype=torch.int32, device=dev())
    for bad in (lambda: awq.moe_route(l.double(), 2), lambda: awq.moe_route(l.t(), 2), lambda: awq.moe_route(l[0], 2),
                lambda: awq.moe_combine(y.float(), w, p), lambda: awq.moe_combine(y, w.half(), p),
                lambda: awq.moe_combine(y, w, p[:7]), lambda: awq.moe_combine(y, w, p.long()),
                lambda: awq.moe_combine(y, w, p, out=y[:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(awq.AWQError, match="EINVAL"):
        awq.moe_route(l, 9)
    with pytest.raises(awq.AWQError, match="EINVAL"):
        awq.moe_combine(y[:, :60].contiguous(), w, p)
