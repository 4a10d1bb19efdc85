"""Products grouped by expert, W4A16 and block-scaled E4M3, and the dense E4M3 one, against the oracle.

Bounds.  W4A16: weights enter rounded to the activation type at worst (half a
step each), sums are fp32 (K products, 2^-24 each at worst).  E4M3: the matrix
cores (every fp8 instruction of gfx950 alike) line up the products of four consecutive k with the one whose
codes' exponents ea + eb add up to the most, and keep multiples of 2^(ea + eb - 13): 2^16 - 2^16 + 2^3 is 8, 2^16 -
2^16 + 2^2 is 0, where four k further 2^-7 still counts.  Each of the other three loses less than one such unit, so a
group loses less than 3 x 2^-13 of its largest max(|a|, 2^-6) max(|w|, 2^-6) (codes below 2^-6 have its exponent),
and the sum less than that part of the sum of these; the groups' sums and a block's scale are fp32.  Output: half a
step.  Against wrong operands, whose errors these bounds would partly hide, the
norm of the whole error: roundings that do not know of each other stay below their
own half step of the norm (three of them: output, weight, and the fp32 parts)."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from moe_helpers import DT, HALF_STEP, cuda, e4m3_weights, experts_weights, f64, randn, rel, split_rows, within
from oracle import moe

pytestmark = pytest.mark.gpu

# rows of each expert: single ones, none, tile edges of every kernel, far from even, the last empty
SPLITS = {
    "one": [0, 1, 0],
    "few": [1, 0, 3, 2],
    "sixteen": [16, 17, 0, 15, 1],
    "forty": [33, 64, 0, 40, 31],
    "skewed": [0, 0, 150, 1, 0, 3],
    "hundred": [100, 129, 64, 0],
    "large": [300, 0, 257, 511],
}


def check(got, R, want, size, per_size, dtype, what):
    """got [R, N] against {row: values}; rows that no expert has keep what they held (77)."""
    live = sorted(want)
    ref, mag = (np.stack([v[r] for r in live]) if live else np.zeros((0, got.shape[1])) for v in (want, size))
    rest = [r for r in range(R) if r not in want]
    assert torch.all(got.cpu()[rest] == 77), what
    if live:
        within(got[torch.tensor(live, device=got.device)], ref, mag, per_size, dtype, what)
        assert rel(got.cpu()[live], ref) <= 3 * HALF_STEP[dtype], what


def plan(split, top, seed, spare=0):
    """offsets, slots in a random order (of tokens enough for them), and their number of tokens; `spare` rows behind."""
    offsets = split_rows(split)
    n = int(offsets[-1])
    tokens = max(1, -(-n // top))
    slots = torch.randperm(tokens * top, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
    return offsets, torch.cat((slots, torch.full((spare,), -1, dtype=torch.int32))), tokens


def run_w4a16(split, K, N, G, zeros, dtype, gather, top=2, seed=0, spare=0):
    E = len(split)
    q, s, z = experts_weights(E, K, N, G, zeros, dtype, seed)
    offsets, slots, tokens = plan(split, top, seed, spare)
    R = len(slots)
    x = randn(seed + 1, tokens if gather else R, K).to(DT[dtype])
    mats = [moe.dequant(q[e].numpy(), f64(s[e]), None if z is None else z[e].numpy(), G) for e in range(E)]
    want, size = moe.grouped(f64(x), mats, offsets.tolist(), slots.tolist() if gather else None, top)
    out = torch.full((R, N), 77.0, dtype=DT[dtype], device=dev())
    xd, qd, sd, zd, od, rd = cuda(x, q, s, z, offsets, slots)
    got = awq.moe_gemm_w4a16(xd, qd, sd, zd, od, rows=rd if gather else None, top_k=top, group_size=G, out=out)
    assert got is out
    check(got, R, want, size, HALF_STEP[dtype] + K * 2.0 ** -24, dtype, f"{split} {K} {N} {G}")
    again = awq.moe_gemm_w4a16(xd, qd, sd, zd, od, rows=rd if gather else None, top_k=top, group_size=G,
                               out=torch.full_like(out, 77.0))
    assert torch.equal(got, again)


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("dtype,zeros,gather", [("f16", True, True), ("bf16", False, False), ("bf16", True, True),
                                                ("f16", False, False)])
def test_experts(split, dtype, zeros, gather):
    print(split, dtype, flush=True)
    run_w4a16(SPLITS[split], 256, 160, 128, zeros, dtype, gather)


@pytest.mark.parametrize("G,K", [(32, 96), (64, 192), (128, 128), (32, 32), (64, 1024)])
@pytest.mark.parametrize("N", [8, 136, 256, 264])
def test_experts_sizes(G, K, N):
    for split in ("few", "forty", "hundred"):
        print(split, G, K, N, flush=True)
        run_w4a16(SPLITS[split], K, N, G, True, "f16", True, top=3, seed=K + N)


@pytest.mark.parametrize("dtype,zeros,gather,K,G", [("f16", True, True, 192, 64), ("bf16", False, False, 128, 128),
                                                    ("bf16", True, True, 64, 32), ("f16", False, False, 128, 32)])
def test_experts_of_large_tiles(dtype, zeros, gather, K, G):
    """As many tiles of 256 x 256 as take them."""
    run_w4a16([700, 501, 0, 650, 599], K, 4352, G, zeros, dtype, gather, seed=K, spare=5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_experts_split_k_of_tiles(dtype):
    """The same through LDS: more than 24 rows an expert, and few tiles (of 64 rows, and of 128)."""
    for split in ([50, 40, 60, 0], [129, 1, 0, 90], [64, 64], [130, 90, 100], [30, 25]):
        K, N = 4096, 288
        assert awq.lib().awq_moe_gemm_w4a16_workspace_bytes(sum(split) + 7, len(split), N, K, 128) > 0
        print(split, flush=True)
        run_w4a16(split, K, N, 128, True, dtype, True, seed=len(split), spare=7)
        run_w4a16(split, K, N, 64, False, dtype, False, seed=len(split), spare=7)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_experts_split_k(dtype):
    """Few tiles and a long K: the workgroups along K add up their shares, row tiles of several experts at once."""
    for split in ([1, 0, 2], [5, 3, 0, 1], [20, 19], [50, 3, 0, 0]):
        K, N = 4096, 264
        assert awq.lib().awq_moe_gemm_w4a16_workspace_bytes(sum(split), len(split), N, K, 128) > 0
        print(split, flush=True)
        run_w4a16(split, K, N, 128, True, dtype, True, seed=len(split))


def test_experts_rows_behind_the_last():
    for split in ("few", "hundred"):
        for gather in (False, True):
            run_w4a16(SPLITS[split], 128, 64, 64, True, "bf16", gather, spare=37)


def test_many_experts():
    g = torch.Generator().manual_seed(0)
    for E in (64, 65, 200, 1024):
        split = (torch.randint(0, 12, (E,), generator=g) * (torch.rand(E, generator=g) < 0.4)).tolist()
        run_w4a16(split, 32, 32, 32, False, "f16", True, seed=E)


# ----------------------------------------------------------------------------- E4M3

def codes(rows, K, seed):
    x = randn(seed, rows, K) * torch.exp(randn(seed + 1, rows, 1))
    a, s = moe.block_quant(x.numpy().astype(np.float64))
    return torch.from_numpy(a), torch.from_numpy(s)


def per_size(K):
    return 3 * 2.0 ** -13 + 128 * 2.0 ** -23 + (-(-K // 128) + 2) * 2.0 ** -24


def magnitudes(codes, scales, row_block):
    """max(|code|, 2^-6) times the scales: what the matrix cores' steps are a part of."""
    least = np.where(np.abs(moe.decode(codes)) < 2.0 ** -6, 8, codes)  # code 8 is 2^-6
    return np.abs(moe.block_values(least, scales, row_block))


def run_dense(M, N, K, dtype, seed=0):
    a, sa = codes(M, K, seed)
    w, sw = e4m3_weights(0, N, K, seed)
    av, wv = moe.block_values(a.numpy(), sa.numpy(), 1), moe.block_values(w.numpy(), sw.numpy(), 128)
    ad, wd, sad, swd = cuda(a, w, sa, sw)
    got = awq.gemm_fp8_block(ad, wd, sad, swd, dtype=DT[dtype])
    assert got.dtype is DT[dtype]
    size = magnitudes(a.numpy(), sa.numpy(), 1) @ magnitudes(w.numpy(), sw.numpy(), 128).T
    within(got, av @ wv.T, size, per_size(K), dtype, f"{M} {N} {K}")
    assert rel(got, av @ wv.T) <= HALF_STEP[dtype]
    again = awq.gemm_fp8_block(ad.view(torch.float8_e4m3fn), wd.view(torch.float8_e4m3fn), sad, swd, dtype=DT[dtype])
    assert torch.equal(got, again)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 129, 255, 256, 257, 600])
@pytest.mark.parametrize("N,K", [(8, 16), (128, 128), (136, 144), (264, 640), (512, 496)])
def test_product(M, N, K):
    print(M, N, K, flush=True)
    run_dense(M, N, K, "bf16" if M % 2 else "f16", seed=M)


@pytest.mark.parametrize("M,N,K", [(1, 256, 14336), (3, 64, 4112), (40, 200, 8192), (1, 24, 131072), (70, 264, 4112),
                                   (300, 256, 2064)])
def test_product_split_k(M, N, K):
    assert awq.lib().awq_fp8_block_gemm_workspace_bytes(M, 0, N, K) > 0
    run_dense(M, N, K, "f16")


@pytest.mark.parametrize("M,N,K", [(2600, 4104, 400), (2561, 4096, 128), (3000, 3848, 2064)])
def test_product_of_large_tiles(M, N, K):
    """As many tiles of 256 x 256 as take them."""
    run_dense(M, N, K, "bf16", seed=K)


@pytest.mark.parametrize("M,N,K", [(1601, 4104, 400), (1664, 4096, 128), (1537, 3848, 16), (1600, 4096, 144), (1590, 3896, 2112)])
def test_product_of_wide_tiles(M, N, K):
    """As many tiles of 128 x 256 as take them, in one round."""
    run_dense(M, N, K, "f16", seed=K)


def run_grouped(split, K, N, dtype, gather, top=2, seed=0, spare=0):
    E = len(split)
    offsets, slots, tokens = plan(split, top, seed, spare)
    R = len(slots)
    a, sa = codes(tokens if gather else R, K, seed)
    w, sw = e4m3_weights(E, N, K, seed)
    av = moe.block_values(a.numpy(), sa.numpy(), 1)
    mats = [moe.block_values(w[e].numpy(), sw[e].numpy(), 128).T for e in range(E)]
    where = (offsets.tolist(), slots.tolist() if gather else None, top)
    want, _ = moe.grouped(av, mats, *where)
    size, _ = moe.grouped(magnitudes(a.numpy(), sa.numpy(), 1),
                          [magnitudes(w[e].numpy(), sw[e].numpy(), 128).T for e in range(E)], *where)
    out = torch.full((R, N), 77.0, dtype=DT[dtype], device=dev())
    ad, wd, sad, swd, od, rd = cuda(a, w, sa, sw, offsets, slots)
    got = awq.moe_gemm_fp8_block(ad, wd, sad, swd, od, rows=rd if gather else None, top_k=top, dtype=DT[dtype], out=out)
    check(got, R, want, size, per_size(K), dtype, f"{split} {K} {N}")


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("dtype,gather,K,N", [("f16", True, 256, 160), ("bf16", False, 256, 160), ("bf16", True, 400, 264),
                                              ("f16", False, 528, 520)])
def test_grouped_product(split, dtype, gather, K, N):
    print(split, dtype, K, N, flush=True)
    run_grouped(SPLITS[split], K, N, dtype, gather)


def test_grouped_product_of_large_tiles():
    run_grouped([900, 0, 1100, 769], 272, 4096, "f16", True, seed=5)
    run_grouped([900, 0, 1100, 769], 272, 4096, "bf16", False, seed=6, spare=3)


def test_grouped_product_of_wide_tiles():
    split = [0, 1, 130, 17, 64, 128, 129, 5, 33, 0, 90, 7, 200, 16, 15, 2]
    for K in (272, 96):
        run_grouped(split, K, 4096, "f16", True, seed=K, spare=11)
        run_grouped(split, K, 3848, "bf16", False, seed=K)


def test_grouped_product_split_k():
    for split in ([1, 0, 2], [20, 19], [50, 3, 0, 0]):
        assert awq.lib().awq_fp8_block_gemm_workspace_bytes(sum(split), len(split), 136, 8192) > 0
        run_grouped(split, 8192, 136, "bf16", True, spare=5)


def test_grouped_product_rows_behind_the_last():
    for split in ("few", "hundred", "large"):
        run_grouped(SPLITS[split], 128, 64, "bf16", True, spare=37)


@pytest.mark.parametrize("split,K,N", [([3, 1, 0, 5], 4096, 264), ([40, 33, 64, 31], 4096, 136), ([60, 33, 64, 51], 4096, 160), ([300, 150, 257, 90], 256, 160)])
def test_part_of_the_experts(split, K, N):
    """A plan's offsets from an expert on, with the matrices of some: rows of the others are left as they are."""
    q, s, z = experts_weights(len(split), K, N, 128, True, "f16", 0)
    w, sw = e4m3_weights(len(split), N, K, 0)
    offsets, slots, tokens = plan(split, 2, 0)
    x = randn(1, tokens, K).half()
    a, sa = codes(tokens, K, 0)
    xd, qd, sd, zd, wd, swd, ad, sad, od, rd = cuda(x, q, s, z, w, sw, a, sa, offsets, slots)
    for part in (slice(0, 1), slice(1, 3), slice(2, 4)):
        off = od[part.start:part.stop + 1]
        where = (off.tolist(), slots.tolist(), 2)
        print(split, part, flush=True)
        out = torch.full((len(slots), N), 77.0, dtype=torch.float16, device=dev())
        awq.moe_gemm_w4a16(xd, qd[part], sd[part], zd[part], off, rows=rd, top_k=2, out=out)
        mats = [moe.dequant(q[e].numpy(), f64(s[e]), z[e].numpy(), 128) for e in range(len(split))[part]]
        want, size = moe.grouped(f64(x), mats, *where)
        check(out, len(slots), want, size, HALF_STEP["f16"] + K * 2.0 ** -24, "f16", f"{split} {part}")
        out.fill_(77.0)
        awq.moe_gemm_fp8_block(ad, wd[part], sad, swd[part], off, rows=rd, top_k=2, out=out, dtype=torch.float16)
        mats = [moe.block_values(w[e].numpy(), sw[e].numpy(), 128).T for e in range(len(split))[part]]
        want, _ = moe.grouped(moe.block_values(a.numpy(), sa.numpy(), 1), mats, *where)
        sizes = [magnitudes(w[e].numpy(), sw[e].numpy(), 128).T for e in range(len(split))[part]]
        size, _ = moe.grouped(magnitudes(a.numpy(), sa.numpy(), 1), sizes, *where)
        check(out, len(slots), want, size, per_size(K), "f16", f"{split} {part}")


def test_no_rows_at_all():
    """Offsets of zeros: nothing is written."""
    q, s, z = cuda(*experts_weights(3, 64, 64, 64, True, "f16", 0))
    off = torch.zeros(4, dtype=torch.int32, device=dev())
    out = torch.full((5, 64), 77.0, dtype=torch.float16, device=dev())
    awq.moe_gemm_w4a16(torch.zeros(5, 64, dtype=torch.float16, device=dev()), q, s, z, off, group_size=64, out=out)
    assert torch.all(out == 77)
    w, sw = cuda(*e4m3_weights(3, 64, 64, 0))
    a, sa = torch.zeros(5, 64, dtype=torch.uint8, device=dev()), torch.ones(5, 1, device=dev())
    awq.moe_gemm_fp8_block(a, w, sa, sw, off, dtype=torch.float16, out=out)
    assert torch.all(out == 77)
    assert awq.gemm_fp8_block(a[:0], w[0], sa[:0], sw[0]).shape == (0, 64)


@pytest.mark.parametrize("T", [5, 60, 200, 500])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_infinities_stay_in_their_rows(T, dtype):
    """A row of x with an infinity or a NaN gives no number where a weight meets it, and changes no other row."""
    K, N, E = 256, 288, 2
    q, s, z = cuda(*experts_weights(E, K, N, 128, True, dtype, 0))
    x = randn(T, T, K).to(DT[dtype]).to(dev())
    off = torch.tensor([0, T // 2, T], dtype=torch.int32, device=dev())
    clean = awq.moe_gemm_w4a16(x, q, s, z, off)
    bad = torch.tensor([0, T // 2 - 1, T - 1], device=dev())
    x[bad, torch.tensor([3, 130, 255], device=dev())] = torch.tensor([torch.inf, torch.nan, -torch.inf], dtype=DT[dtype], device=dev())
    got = awq.moe_gemm_w4a16(x, q, s, z, off)
    rest = torch.ones(T, dtype=torch.bool, device=dev())
    rest[bad] = False
    assert torch.equal(got[rest], clean[rest])
    assert not torch.isfinite(got[bad]).any()


def test_offsets_that_are_no_plan():
    """Falling, negative, past the rows: whatever is computed, nothing outside the tensors is touched, and every row
    that is written is some row's product."""
    q, s, z = cuda(*experts_weights(4, 128, 64, 64, True, "f16", 0))
    x = torch.ones(40, 128, dtype=torch.float16, device=dev())
    pad = torch.full((60, 64), 77.0, dtype=torch.float16, device=dev())
    for off in ([0, 90, 3, -7, 41], [-5, 10, 10, 2, 1 << 30], [40, 30, 20, 10, 0], [-2 ** 31, 2 ** 31 - 1, 0, 5, 4]):
        o = torch.tensor(off, dtype=torch.int32, device=dev())
        rows = torch.tensor([-1, 10 ** 9, -2 ** 31, 2 ** 31 - 1, 79, 80] + [3] * 34, dtype=torch.int32, device=dev())
        awq.moe_gemm_w4a16(x, q, s, z, o, group_size=64, out=pad[10:50])
        awq.moe_gemm_w4a16(x, q, s, z, o, rows=rows, top_k=2, group_size=64, out=pad[10:50])
        assert torch.all(pad[:10] == 77) and torch.all(pad[50:] == 77)
        assert torch.isfinite(pad).all()


def test_refusals():
    x, off = torch.zeros(8, 128, dtype=torch.float16, device=dev()), torch.zeros(3, dtype=torch.int32, device=dev())
    q, s, z = cuda(*experts_weights(2, 128, 64, 64, True, "f16", 0))
    ok = dict(x=x, qweight=q, scales=s, qzeros=z, offsets=off, group_size=64)
    awq.moe_gemm_w4a16(**ok)
    rows = torch.zeros(8, dtype=torch.int32, device=dev())
    for bad in (dict(x=x.float()), dict(x=x.t()), dict(x=x[:, :64].contiguous()), dict(qweight=q[0]), dict(scales=s[:1]),
                dict(scales=s.bfloat16()), dict(qzeros=z[:, :1]), dict(offsets=off[:2]), dict(offsets=off.long()),
                dict(rows=rows.long()), dict(rows=rows.view(2, 4)), dict(out=x), dict(group_size=128),
                dict(offsets=off.cpu())):
        with pytest.raises(ValueError):
            awq.moe_gemm_w4a16(**{**ok, **bad})
    with pytest.raises(awq.AWQError, match="EINVAL"):
        awq.moe_gemm_w4a16(**ok, rows=rows, top_k=0)
    w, sw = cuda(*e4m3_weights(2, 64, 128, 0))
    a, sa = torch.zeros(8, 128, dtype=torch.uint8, device=dev()), torch.ones(8, 1, device=dev())
    ok = dict(a=a, w=w, sa=sa, sw=sw, offsets=off)
    awq.moe_gemm_fp8_block(**ok)
    for bad in (dict(a=a.float()), dict(a=a[:, ::2]), dict(w=w[0]), dict(sa=sa[:7]), dict(sw=sw[:, :, :0]),
                dict(sw=sw.double()), dict(dtype=torch.float32), dict(offsets=off[:2]), dict(out=x)):
        with pytest.raises(ValueError):
            awq.moe_gemm_fp8_block(**{**ok, **bad})
