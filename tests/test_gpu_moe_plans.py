"""Each kernel of the grouped and block-scaled products at sizes well inside those that it is chosen for, the plan
asserted; bounds as in test_gpu_moe_gemm.py."""
import pytest

import bit_weight_only_awq_amd as awq
from test_gpu_moe_gemm import run_dense, run_grouped, run_w4a16

pytestmark = pytest.mark.gpu


def planned(op, R, E, N, K, G, want, split):
    p = awq.plan_info(op, R, N, K, G, experts=E)
    assert (p["kernel"], 16 * p["row_tiles"], p["tile_cols"]) == want and (p["splits"] > 1) == split, p


@pytest.mark.parametrize("dtype,zeros,gather", [("f16", True, True), ("bf16", False, False), ("bf16", True, True)])
@pytest.mark.parametrize("split,K,N,G,want,k_split", [
    ([4, 1, 0, 7, 3], 512, 4360, 64, (5, 16, 256), False),
    ([4, 1, 0, 7, 3], 4096, 520, 128, (5, 16, 256), True),
    ([20, 16, 33, 1, 18], 512, 4360, 64, (5, 32, 256), False),
    ([20, 16, 33, 1, 18], 4096, 520, 128, (5, 32, 256), True),
    ([40, 65, 0, 30, 64, 41], 512, 2080, 64, (3, 64, 128), False),
    ([40, 65, 0, 30, 64, 41], 4096, 544, 128, (3, 64, 128), True),
    ([120, 129, 90, 0, 128, 127], 512, 2080, 32, (3, 128, 128), False),
    ([120, 129, 90, 0, 128, 127], 4096, 544, 128, (3, 128, 128), True),
    ([760, 700, 0, 650, 769], 256, 4384, 32, (3, 256, 256), False)])
def test_w4a16(split, K, N, G, want, k_split, dtype, zeros, gather):
    planned(awq.AWQ_OP_MOE_GEMM_W4A16, sum(split), len(split), N, K, G, want, k_split)
    print(split, want, dtype, flush=True)
    run_w4a16(split, K, N, G, zeros, dtype, gather, seed=len(split))


@pytest.mark.parametrize("K,N,G", [(96, 256, 32), (160, 136, 32), (256, 1000, 128)])
def test_w4a16_many_rows_of_shapes_without_tiles(K, N, G):
    """K % 64 or N % 32: the streaming kernel takes any number of rows."""
    split = [700, 0, 33, 1025, 1]
    planned(awq.AWQ_OP_MOE_GEMM_W4A16, sum(split), len(split), N, K, G, (5, 32, 256), False)
    run_w4a16(split, K, N, G, True, "f16", True, seed=K)
    run_w4a16(split, K, N, G, False, "bf16", False, seed=N, spare=9)


@pytest.mark.parametrize("dtype,gather", [("f16", True), ("bf16", False)])
@pytest.mark.parametrize("split,K,N,want,k_split", [
    ([2, 1, 0, 3], 512, 4104, (5, 16, 32), False),
    ([2, 1, 0, 3], 8192, 136, (5, 16, 32), True),
    ([40, 33, 0, 17, 60], 528, 2056, (3, 128, 128), False),
    ([40, 33, 0, 17, 60], 4112, 264, (3, 128, 128), True),
    ([120, 40, 0, 129, 90, 60, 256, 31], 400, 6152, (3, 128, 256), False),
    ([900, 850, 0, 1000, 1025, 777], 272, 4104, (3, 256, 256), False)])
def test_grouped_e4m3(split, K, N, want, k_split, dtype, gather):
    planned(awq.AWQ_OP_FP8_BLOCK_GEMM, sum(split), len(split), N, K, 128, want, k_split)
    print(split, want, dtype, flush=True)
    run_grouped(split, K, N, dtype, gather, seed=K)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N,want,k_split", [
    (3, 528, 8200, (5, 16, 32), False), (9, 8192, 264, (5, 16, 32), True), (100, 1040, 14344, (3, 128, 128), False),
    (100, 8208, 520, (3, 128, 128), True), (500, 272, 14344, (3, 128, 256), False), (3300, 272, 3848, (3, 256, 256), False)])
def test_dense_e4m3(M, K, N, want, k_split, dtype):
    planned(awq.AWQ_OP_FP8_BLOCK_GEMM, M, 0, N, K, 128, want, k_split)
    run_dense(M, N, K, dtype, seed=M)
