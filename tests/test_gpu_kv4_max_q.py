"""The attention's binding where cu_q is given and max_q is not: every row is written."""
import numpy as np
import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from test_gpu_kv4_attention import Case, t16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new", [([300, 90, 200], [70, 20, 1]), ([40, 9], [3, 2]), ([17, 5], [1, 1])])
def test_every_row_is_written_without_max_q(lens, new):
    c = Case(lens, new, 4, 2, 64, 16, "f16", seed=sum(new))
    q, cache, tables, lens_, cu = (t.to(dev()) for t in (t16(c.q, "f16"), *map(torch.from_numpy, (
        c.cache, c.tables, c.lens, c.cu))))
    out = torch.full_like(q, 7.0)
    awq.kv4_attention(q, cache, tables, lens_, cu_q=cu, out=out)
    # (another max_q may be another kernel: equal but for the numerators' and the output's rounding)
    want = awq.kv4_attention(q, cache, tables, lens_, cu_q=cu, max_q=int(np.max(new)))
    assert not bool((out == 7.0).all(-1).any())
    assert float((out.double() - want.double()).norm() / want.double().norm()) < 2.0 ** -10
