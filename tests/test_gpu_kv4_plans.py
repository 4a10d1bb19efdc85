"""Attention over the 4-bit paged cache through each way of launching it.

Which kernel a call takes depends on its rows and on how much work the call's
bounds stand for; a high max_kv stands for much.  Bounds on the errors: those
of test_gpu_kv4_attention.py, whose cases these are."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev
from oracle import block
from test_gpu_kv4_attention import Case, b16

pytestmark = pytest.mark.gpu
LONG = 131072  # with more than 128 rows: the prompts' kernel, whatever the batch


@pytest.mark.parametrize("hq,hkv,D,P,window,dtype", [
    (4, 1, 128, 16, 0, "f16"), (2, 2, 64, 32, 0, "bf16"), (8, 2, 128, 64, 50, "bf16"), (4, 4, 64, 16, 130, "f16"),
    (7, 1, 128, 128, 0, "bf16"), (3, 1, 64, 1024, 1, "f16")])
def test_prompts(hq, hkv, D, P, window, dtype):
    """Whole prompts and chunks over earlier context, of lengths around the tiles'; more new tokens than context."""
    lens, new = [140, 300, 128, 65, 513, 0, 50], [140, 77, 128, 65, 33, 3, 60]
    Case(lens, new, hq, hkv, D, P, dtype, seed=hq * D).check(window=window, max_kv=LONG)


@pytest.mark.parametrize("D,dtype,window", [(64, "f16", 0), (128, "bf16", 0), (128, "f16", 700)])
def test_prompts_split(D, dtype, window):
    """Sequences over several workgroups: many splits, or a few, and some that need one only."""
    c = Case([2900, 150], [200, 150], 2, 1, D, 32, dtype, seed=D)
    y = c.check(max_kv=32768, window=window)
    for _ in range(3):
        assert torch.equal(c.gpu(max_kv=32768, window=window), y)
    Case([1500, 200, 0, 700], [200, 7, 0, 170], 8, 8, D, 16, dtype, seed=D + 1).check(max_kv=4096, window=window)


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
def test_few_splits(D, dtype):
    for new in (1, 6):
        Case([1500, 700, 0, 130, 1], [new] * 5, 4, 1, D, 32, dtype, seed=new).check(max_kv=1536)


@pytest.mark.parametrize("D,dtype,window", [(64, "f16", 0), (128, "bf16", 0), (64, "bf16", 40)])
def test_many_tiles(D, dtype, window):
    """Tiles of 32 rows, where there are enough of them; the same rows of one sequence only, in tiles of 16."""
    c = Case([200, 90, 97, 130], [100, 90, 97, 3], 32, 32, D, 16, dtype, seed=D)
    c.check(window=window)
    Case([200], [100], 4, 2, D, 16, dtype, seed=D).check(window=window)


def test_rows_past_max_q_are_left():
    c = Case([240, 240], [200, 150], 2, 1, 64, 16, "f16", seed=1)
    full = c.check(max_kv=LONG)
    out = torch.full_like(full, 7.0)
    c.gpu(max_q=130, max_kv=LONG, out=out)
    assert torch.equal(out[:130], full[:130]) and torch.equal(out[200:330], full[200:330])
    assert bool((out[130:200] == 7).all()) and bool((out[330:] == 7).all())


def test_missing_pages_hide_their_tokens():
    c = Case([400, 190], [150, 150], 4, 2, 64, 16, "f16", seed=2)
    c.tables[0, 3] = -1
    c.tables[0, 17] = c.cache.shape[0]
    c.tables[1, :] = np.int32(2 ** 31 - 1)
    y = c.check(max_kv=LONG)
    assert not y[150:].any()


@pytest.mark.parametrize("kw", [dict(max_kv=LONG), dict()])
@pytest.mark.parametrize("new", [3, 50, 150])
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("meta", ["km", "vm"])
def test_scale_that_is_not_finite(meta, what, new, kw):
    """Of a token that the rows from one on see: those before it are as they were with any other value there."""
    c = Case([320, 160], [new, new], 2, 1, 64, 16, "f16", seed=4)
    tok = 320 - new // 2 - 1
    at = c.tables[0, tok // 16], 0, block.word_at(meta, 16, 64, tok % 16)
    first = tok - (320 - new)
    c.cache[at] = 0x3C00
    ref = block.decode(b16(c.gpu(**kw)), "f16")
    c.cache[at] = 0x7E00 if what == "nan" else 0x7C00
    got = block.decode(b16(c.gpu(**kw)), "f16")
    assert not np.isfinite(got[first:new]).any(-1).all(), "the token is seen"
    # (the reference may follow the hidden token's scale: the numerators' rounding differs)
    assert np.isfinite(got[:first]).all() and np.abs(got[:first] - ref[:first]).max(initial=0.0) < 2e-2
    assert np.array_equal(got[new:], ref[new:])


def test_nan_in_a_query_stays_in_its_row():
    c = Case([220, 160], [150, 150], 2, 1, 64, 16, "f16", seed=5)
    ref = c.check(max_kv=LONG)
    c.q[3, 1, 9] = 0x7E00
    got = c.gpu(max_kv=LONG)
    keep = torch.ones_like(ref, dtype=torch.bool)
    keep[3, 1] = False
    assert torch.equal(got[keep], ref[keep]) and bool(got[3, 1].isnan().all())


@pytest.mark.parametrize("dtype,k_size,v_size", [("f16", 1e-5, 1e-5), ("f16", 300.0, 300.0), ("bf16", 1e-25, 1e-25),
                                                 ("bf16", 1e25, 1e25), ("f16", 40.0, 1.0)])
def test_magnitudes(dtype, k_size, v_size):
    scale = 0.125 / max(k_size, 1.0) if k_size != 40.0 else None
    Case([190, 161], [150, 140], 4, 2, 64, 16, dtype, seed=6, k_size=k_size, v_size=v_size).check(scale=scale,
                                                                                                   max_kv=LONG)


def test_workspace_left_zero():
    import bit_weight_only_awq_amd as awq
    s = torch.cuda.Stream()
    for c, max_kv in ((Case([2900, 150], [200, 150], 2, 1, 64, 32, "f16", seed=9), 32768),
                      (Case([1500, 700, 0, 130, 1], [6] * 5, 4, 1, 64, 32, "f16", seed=3), 1536)):
        with torch.cuda.stream(s):
            c.gpu(max_kv=max_kv)
        s.synchronize()
        with torch.cuda.stream(s):
            buf = awq.ops.WORKSPACE.get(dev(), 1)
        torch.cuda.synchronize()
        assert not buf.any()
