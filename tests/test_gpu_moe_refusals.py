"""Numbers and plans that the binding of the mixture-of-experts calls uses before the library sees them: refused as the
library and the binding refuse others."""
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from moe_helpers import cuda, e4m3_weights, experts_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top_k", [0, -1, -7, 9, 1 << 40])
def test_top_k(top_k):
    with pytest.raises(awq.AWQError, match="EINVAL"):
        awq.moe_route(torch.zeros(4, 8, device=dev()), top_k)


@pytest.mark.parametrize("group", [0, -1, -128])
def test_group_size(group):
    q, s, z = cuda(*experts_weights(2, 128, 64, 128, True, "f16", 0))
    x, off = torch.zeros(4, 128, dtype=torch.float16, device=dev()), torch.zeros(3, dtype=torch.int32, device=dev())
    with pytest.raises(awq.AWQError, match="EINVAL"):
        awq.moe_gemm_w4a16(x, q, s, z, off, group_size=group)


@pytest.mark.parametrize("shape", [(), (4, 1), (1, 4)])
def test_rows_of_other_dimensions(shape):
    q, s, z = cuda(*experts_weights(2, 128, 64, 128, True, "f16", 0))
    w, sw = cuda(*e4m3_weights(2, 64, 128, 0))
    x, off = torch.zeros(4, 128, dtype=torch.float16, device=dev()), torch.zeros(3, dtype=torch.int32, device=dev())
    a, sa = awq.quant_act_fp8_block(x)
    rows = torch.zeros(shape, dtype=torch.int32, device=dev())
    with pytest.raises(ValueError):
        awq.moe_gemm_w4a16(x, q, s, z, off, rows=rows)
    with pytest.raises(ValueError):
        awq.moe_gemm_fp8_block(a, w, sa, sw, off, rows=rows)
