"""The torch binding's own parts, without a GPU: workspaces and strides; launches past the runtime's limit."""
import gc
import weakref

import pytest
import torch

from bit_weight_only_awq_amd import _lib as L
from bit_weight_only_awq_amd import ops


@pytest.fixture
def space(monkeypatch):
    """A Workspace whose memory is the host's, and the number of the capture under way (0: none)."""
    capture = [0]
    monkeypatch.setattr(ops, "_zeros", lambda index, nbytes: torch.zeros(nbytes, dtype=torch.uint8))
    monkeypatch.setattr(ops, "_capture_id", lambda stream: capture[0])
    return ops.Workspace(), capture


MB = 1 << 20


def test_workspace_is_shared_by_a_streams_calls(space):
    ws, _ = space
    a = ws.of_stream(0, 7, 100)
    assert a == ws.of_stream(0, 7, MB) and a[1] == MB
    assert ws.of_stream(0, 8, 100)[0] != a[0] and ws.of_stream(1, 7, 100)[0] != a[0]


def test_replaced_workspace_stays_alive(space):
    """A graph that was captured with it still writes there."""
    ws, _ = space
    first = ws._buffer(0, 7, 100)
    ref, at = weakref.ref(first), first.data_ptr()
    del first
    sizes = [ws.of_stream(0, 7, n)[1] for n in (MB + 1, 2 * MB + 1, 30 * MB, 30 * MB + 1)]
    assert sizes == [2 * MB, 4 * MB, 30 * MB, 60 * MB]
    gc.collect()
    assert ref() is not None and ref().data_ptr() == at
    assert sum(t.numel() for t in ws._kept) < sizes[-1]


def test_capture_takes_the_streams_workspace(space):
    ws, capture = space
    a = ws.of_stream(0, 7, 100)
    capture[0] = 5
    assert ws.of_stream(0, 7, MB) == a


@pytest.mark.parametrize("eager_first", [False, True])
def test_memory_zeroed_in_a_capture_stays_in_it(space, eager_first):
    """Its zero-fill runs when the graph does, so nothing else may rely on it."""
    ws, capture = space
    get = lambda n: ws._buffer(0, 7, n)  # noqa: E731
    eager = get(100) if eager_first else None
    capture[0] = 5
    recorded = get(3 * MB)
    assert recorded is not eager and get(2 * MB) is recorded  # one fill a capture
    grown = get(4 * MB)
    assert grown.numel() == 6 * MB and get(3 * MB) is grown
    capture[0] = 6
    other = get(3 * MB)
    assert other is not grown
    capture[0] = 0
    after = get(100)
    assert after is eager if eager_first else not any(after is t for t in (recorded, grown, other))
    assert not any(get(3 * MB) is t for t in (recorded, grown, other))


def test_capture_id_refuses():
    assert L.lib().awq_stream_capture_id(None, None) == L.AWQ_EINVAL
    assert ops._capture_id(0) == 0


def test_stride_of_a_single_token_says_nothing():
    """One token out of rows whose length is odd, or far apart: the append takes it as dense."""
    wide = torch.zeros(3, 2 * 64 + 1, dtype=torch.float16)
    for t in (wide[:1, :128].view(1, 2, 64), torch.zeros(1, 2, 64, dtype=torch.float16).expand(1, 2, 64),
              torch.as_strided(torch.zeros(128, dtype=torch.float16), (1, 2, 64), (1 << 40, 64, 1))):
        assert ops._heads(t, torch.Size((1, 2, 64)), torch.float16, -1, "k") == 128
    assert ops._heads(torch.zeros(0, 2, 64, dtype=torch.float16), torch.Size((0, 2, 64)), torch.float16, -1, "k") == 128
    rows = torch.zeros(3, 200, dtype=torch.float16)
    assert ops._heads(rows[:, :128].view(3, 2, 64), torch.Size((3, 2, 64)), torch.float16, -1, "k") == 200


def test_attention_past_the_launch_limit():
    """A grid holds less than 2^32 threads along an axis: said before anything is enqueued."""
    def call(B, heads, max_q=1):
        return L.lib().awq_kv4_attention(0x10000, 0x10000, 0x10000, 0x10000, 0x10000, 0x10000, B, B, max_q, 100, heads,
                                         heads, 64, 16, 9, 7, 0.125, 0, 0, 0x10000, 1 << 40, None)
    assert call(1 << 20, 16) == L.AWQ_EUNSUPPORTED
    assert call(1 << 20, 4096) == L.AWQ_EUNSUPPORTED
    assert call(1 << 20, 8, 200) == L.AWQ_EUNSUPPORTED  # (the prompts' kernel has twice the threads)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_refuses_y_over_the_residual_stream(fp8):
    """Both would be written to one place, and one of them lost."""
    a, o = 0x10000, 0x20000
    fn = L.lib().w4a8_fp8_rmsnorm_quant if fp8 else L.lib().w4a8_rmsnorm_quant
    assert fn(a, a, a, o, o, a, a, *([a] if fp8 else []), 4, 64, 1e-6, 0, None) == L.AWQ_EINVAL
