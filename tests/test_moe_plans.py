"""The plans of grouped and block-scaled products: what awq_grouped_plan_info refuses and answers, that the shapes of
the GPU tests get the kernels that these are named after, and that plans of other devices are valid ones (no GPU)."""
import ctypes

import pytest

from bit_weight_only_awq_amd import _lib as L

W, F = L.AWQ_OP_MOE_GEMM_W4A16, L.AWQ_OP_FP8_BLOCK_GEMM


def plan(op, R, E, N, K, G=128, cus=256):
    info = L.PlanInfo()
    assert L.lib().awq_grouped_plan_info(op, R, E, N, K, G, cus, ctypes.byref(info)) == L.AWQ_OK
    return info


def tile(*args, **kw):
    p = plan(*args, **kw)
    return p.kernel, 16 * p.row_tiles, p.tile_cols


@pytest.mark.parametrize("kw,rc", [
    (dict(op=0), "EINVAL"), (dict(op=99), "EINVAL"), (dict(R=0), "EINVAL"), (dict(R=-1), "EINVAL"),
    (dict(R=(1 << 24) + 1), "EINVAL"), (dict(E=-1), "EINVAL"), (dict(op=W, E=0), "EINVAL"), (dict(E=1025), "EINVAL"),
    (dict(N=12), "EINVAL"), (dict(op=W, K=192), "EINVAL"), (dict(op=W, G=100), "EINVAL"), (dict(op=F, K=136), "EINVAL"),
    (dict(cus=-1), "EINVAL"), (dict(out=False), "EINVAL"), (dict(op=F, N=1 << 17, K=1 << 14), "EUNSUPPORTED")])
def test_refusals(kw, rc):
    a = dict(op=F, R=8, E=4, N=256, K=256, G=128, cus=256, out=True)
    a.update(kw)
    info = L.PlanInfo()
    got = L.lib().awq_grouped_plan_info(a["op"], a["R"], a["E"], a["N"], a["K"], a["G"], a["cus"],
                                        ctypes.byref(info) if a["out"] else None)
    assert got == getattr(L, "AWQ_" + rc)


def test_binding():
    import bit_weight_only_awq_amd as awq
    p = awq.plan_info(awq.AWQ_OP_MOE_GEMM_W4A16, 8192, 28672, 4096, 128, cu_count=256, experts=8)
    assert (p["kernel"], p["row_tiles"], p["tile_cols"], p["splits"]) == (3, 16, 256, 1)
    assert awq.plan_info(awq.AWQ_OP_FP8_BLOCK_GEMM, 1, 14336, 4096, 128, cu_count=256)["kernel"] == 5
    with pytest.raises(awq.AWQError, match="EINVAL"):
        awq.plan_info(awq.AWQ_OP_MOE_GEMM_W4A16, 8192, 28672, 4096, 128, cu_count=256)


def test_workspace_query_agrees():
    """(No device here: the queries plan for a whole MI355X.)"""
    for R, E, N, K in ((2, 8, 4096, 14336), (64, 8, 4096, 14336), (300, 4, 288, 4096), (1, 0, 1024, 14336),
                       (96, 0, 14336, 4096), (8192, 8, 4096, 4096)):
        assert plan(F, R, E, N, K).workspace_bytes == L.lib().awq_fp8_block_gemm_workspace_bytes(R, E, N, K)
        if E:
            assert plan(W, R, E, N, K).workspace_bytes == L.lib().awq_moe_gemm_w4a16_workspace_bytes(R, E, N, K, 128)


@pytest.mark.parametrize("args,want,splits", [
    # (op, rows, experts, N, K, G): the sizes of test_gpu_moe_gemm.py
    ((W, 2455, 5, 4352, 192, 64), (3, 256, 256), False), ((W, 2450, 5, 4352, 128, 32), (3, 256, 256), False),
    ((W, 157, 4, 288, 4096, 128), (3, 64, 128), True), ((W, 227, 4, 288, 4096, 64), (3, 64, 128), True),
    ((W, 135, 2, 288, 4096, 128), (3, 128, 128), True), ((W, 327, 3, 288, 4096, 128), (3, 128, 128), True),
    ((W, 3, 3, 264, 4096, 128), (5, 16, 256), True), ((W, 39, 2, 264, 4096, 128), (5, 32, 256), True),
    ((W, 6, 4, 160, 256, 128), (5, 16, 256), False), ((W, 168, 5, 160, 256, 128), (3, 64, 128), False),
    ((W, 293, 4, 160, 256, 128), (3, 128, 128), False), ((W, 293, 4, 136, 192, 64), (5, 32, 256), False),
    ((F, 2600, 0, 4104, 400, 0), (3, 256, 256), False), ((F, 2561, 0, 4096, 128, 0), (3, 256, 256), False),
    ((F, 3000, 0, 3848, 2064, 0), (3, 256, 256), False), ((F, 1601, 0, 4104, 400, 0), (3, 128, 256), False),
    ((F, 1664, 0, 4096, 128, 0), (3, 128, 256), False), ((F, 1537, 0, 3848, 16, 0), (3, 128, 256), False),
    ((F, 1590, 0, 3896, 2112, 0), (3, 128, 256), False), ((F, 2769, 4, 4096, 272, 0), (3, 256, 256), False),
    ((F, 2772, 4, 4096, 272, 0), (3, 256, 256), False), ((F, 853, 16, 4096, 272, 0), (3, 128, 256), False),
    ((F, 842, 16, 3848, 96, 0), (3, 128, 256), False), ((F, 8, 3, 136, 8192, 0), (5, 16, 32), True),
    ((F, 44, 2, 136, 8192, 0), (3, 128, 128), True), ((F, 1, 0, 256, 14336, 0), (5, 16, 32), True),
    ((F, 70, 0, 264, 4112, 0), (3, 128, 128), True)])
def test_kernels_of_the_gpu_tests(args, want, splits):
    op, R, E, N, K, G = args
    assert tile(op, R, E, N, K, G) == want and (plan(op, R, E, N, K, G).splits > 1) == splits


def test_weights_are_rounded_past_24_rows_only():
    """Up to 24 rows of each expert that the rows reach (23: their number is an estimate), the kernel that rounds no weight."""
    assert all(tile(W, 23 * E, E, N, K)[0] == 5 for E in (1, 8, 60) for N, K in ((4096, 14336), (28672, 4096), (768, 768)))
    assert all(tile(W, 25 * E, E, N, K)[0] == 3 for E in (1, 8) for N, K in ((4096, 14336), (28672, 4096), (768, 768)))


def test_plans_of_other_devices():
    for cus in (8, 64, 256, 304):
        for op in (W, F):
            for E in (1, 8, 64, 1024) + ((0,) if op == F else ()):
                for R in (1, 3, 17, 100, 900, 8192, 100000):
                    for N, K in ((8, 128), (768, 768), (4096, 14336), (28672, 4096), (1000, 4096)):
                        p = plan(op, R, E, N, K, cus=cus)
                        assert p.cu_count == cus and p.kernel in (3, 5) and 1 <= p.splits <= max(1, K // 128)
                        assert p.tiles_n == -(-N // p.tile_cols)
                        rows = 16 * p.row_tiles
                        assert p.tiles_m == (min(E, R) + R // rows if E else -(-R // rows))
                        assert (p.workspace_bytes > 0) == (p.splits > 1)
                        assert p.splits == 1 or p.workspace_bytes >= 4 * p.splits * R * N
