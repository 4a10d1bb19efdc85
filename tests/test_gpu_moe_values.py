"""W4A16 products grouped by expert: what single values of x do to a row, whichever kernel the rows of an expert ask for.

The product is x . ((q - z) s) in every kernel, so an infinity in x gives the infinity of its weight's sign, NaN
where that weight is 0 or infinities of both signs meet; and large numbers give finite sums where their products are."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from moe_helpers import DT, HALF_STEP, cuda, experts_weights, f64, randn, split_rows, within
from oracle import moe

pytestmark = pytest.mark.gpu

# rows of the two experts: streaming kernel with 16 rows (one alone, and more) and 32, tiles of 64 and 128 rows
SPLITS = [[1, 1], [3, 2], [14, 17], [31, 29], [100, 100], [250, 251]]


def matrices(q, s, z, G):
    return [moe.dequant(q[e].numpy(), f64(s[e]), None if z is None else z[e].numpy(), G) for e in range(len(q))]


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("dtype,zeros,G", [("f16", True, 128), ("f16", False, 32), ("bf16", True, 64), ("bf16", False, 128)])
def test_infinities_by_their_definition(split, dtype, zeros, G):
    K, N, T = 256, 288, sum(split)
    q, s, z = experts_weights(2, K, N, G, zeros, dtype, T)
    x = randn(T, T, K).to(DT[dtype])
    x[0, 3] = torch.inf
    x[T - 1, 255] = -torch.inf
    if T > 2:
        x[1, 100], x[1, 200] = torch.inf, -torch.inf  # of both signs, in different runs
        x[2, 130] = torch.nan
    print(split, dtype, flush=True)
    xd, qd, sd, zd, od = cuda(x, q, s, z, split_rows(split))
    got = f64(awq.moe_gemm_w4a16(xd, qd, sd, zd, od, group_size=G))
    mats = matrices(q, s, z, G)
    with np.errstate(invalid="ignore"):
        for t in sorted({0, 1, min(2, T - 1), T - 1}):
            want = (f64(x[t])[:, None] * mats[0 if t < split[0] else 1]).sum(0)
            where = ~np.isfinite(want)
            assert np.array_equal(np.isnan(got[t]), np.isnan(want)), (t, "NaN")
            assert np.array_equal(got[t][where], want[where], equal_nan=True), t
            assert np.isfinite(got[t][~where]).all()


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("zeros", [True, False])
def test_large_numbers(split, zeros):
    """bf16 up to 2^116: sums of 64 products with q - z stay below 15 x 64 x 2^116 < 2^126."""
    K, N, T = 256, 288, sum(split)
    q, s, z = experts_weights(2, K, N, 128, zeros, "bf16", T)
    s = (s.double() * 2.0 ** -110).to(torch.bfloat16)
    x = ((0.5 + torch.rand(T, K, generator=torch.Generator().manual_seed(T)) / 2) * 2.0 ** 116).to(torch.bfloat16)
    mats = matrices(q, s, z, 128)
    want, size = moe.grouped(f64(x), mats, split_rows(split).tolist(), None, 1)
    xd, qd, sd, zd, od = cuda(x, q, s, z, split_rows(split))
    got = awq.moe_gemm_w4a16(xd, qd, sd, zd, od)
    want, size = (np.stack([v[t] for t in range(T)]) for v in (want, size))
    within(got, want, size, HALF_STEP["bf16"] + K * 2.0 ** -24, "bf16", f"{split}")


def to_type(v, dtype):
    return f64(torch.from_numpy(v).to(DT[dtype]))


@pytest.mark.parametrize("split", [[1, 1], [3, 2, 0, 4], [14, 17], [23, 20, 25]])
@pytest.mark.parametrize("dtype,zeros,G,N", [("f16", True, 128, 1288), ("f16", False, 32, 264), ("bf16", True, 64, 264),
                                             ("bf16", False, 128, 1288), ("bf16", True, 32, 264)])
def test_weights_are_not_rounded(split, dtype, zeros, G, N):
    """The streaming kernels' results are the exact ones rounded once, but where the sums' own error crosses a border.

    With x, s of size 1: a run of 64 products x q' (q' <= 15, or 143 in bf16) of either sign sums to about 8 q', its at most
    64 roundings of 2^-24 of that, independent, to 8 x 8 q' 2^-24; the same at worst for z' sum x.  Over the K / 64
    runs these add like the results, sqrt(K) r with r the root mean square of q - z: d = sqrt(2) 8 q' / r 2^-24 of
    the result.  A result less than d from a border (one in u / (2 d), u the type's step) moves by u: sqrt(2 d u) of
    the norm.  Weights rounded to the type give several times as much, which the oracle shows."""
    K, E, R = 512, len(split), sum(split)
    info = awq.plan_info(awq.AWQ_OP_MOE_GEMM_W4A16, R, N, K, G, experts=E)
    assert info["kernel"] == 5
    q, s, z = experts_weights(E, K, N, G, zeros, dtype, R)
    x = randn(R, R, K).to(DT[dtype])
    mats = matrices(q, s, z, G)
    want, _ = moe.grouped(f64(x), mats, split_rows(split).tolist(), None, 1)
    coarse, _ = moe.grouped(f64(x), [to_type(m, dtype) for m in mats], split_rows(split).tolist(), None, 1)
    want, coarse = (np.stack([v[t] for t in range(R)]) for v in (want, coarse))
    ref, n = to_type(want, dtype), np.linalg.norm(want)
    r = np.sqrt(np.mean([np.mean((m / np.repeat(f64(s[e]), G, 0)) ** 2) for e, m in enumerate(mats)]))
    d = np.sqrt(2) * 8 * (15 if dtype == "f16" else 143) / r * 2.0 ** -24
    bound = np.sqrt(2 * d * 2 * HALF_STEP[dtype])
    assert np.linalg.norm(to_type(coarse, dtype) - ref) / n > 2 * bound
    xd, qd, sd, zd, od = cuda(x, q, s, z, split_rows(split))
    got = f64(awq.moe_gemm_w4a16(xd, qd, sd, zd, od, group_size=G))
    assert np.linalg.norm(got - ref) / n <= bound
