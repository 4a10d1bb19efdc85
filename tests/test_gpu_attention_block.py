"""The example of an attention block: norm, products, append and attention together, prompts and a graph of steps.

Bound on its error: the dense layer has the same weights, so what differs is
the 8-bit codes of the two products' inputs (steps of max / 127: below 2 % of
random data's norm each) and the 4-bit keys and values.  A value's step is
about 6 standard deviations / 15, an error of 0.4 / sqrt(12) = 0.115 of its
norm; the keys' moves a score by 0.115 |q| sqrt(D) D^-1/2, with scores near 1
a weight by about that share again.  Independent: below 0.115 sqrt(2) + 0.04
= 0.2; a wrong page, head, position or rotation gives 1."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(), dict(prompts=(1, 33, 64), heads=4, kv_heads=4, head_dim=64, page=32, hidden=512)])
def test_attention_block(kw, dtype):
    import attention_block
    errors = attention_block.run(steps=5, dtype=dtype, **kw)
    assert len(errors) == 6 and max(errors) < 0.2, errors
