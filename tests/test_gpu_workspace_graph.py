"""Workspaces of captured graphs: a graph keeps the memory it was captured with
when later calls need more, and memory that is zeroed inside a graph serves
that graph alone."""
import pytest
import torch

import bit_weight_only_awq_amd as awq
import synthgen
from gpu_helpers import dev, to_dev
from test_gpu_kv4_attention import Case, t16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fresh(monkeypatch):
    """Workspaces of its own for each test (a stream's handle may come back from an earlier one)."""
    monkeypatch.setattr(awq.ops, "WORKSPACE", awq.ops.Workspace())
    yield
    torch.cuda.synchronize()


def attention(c, max_kv):
    q, cache, tables, lens, cu = (t.to(dev()) for t in (t16(c.q, c.dtype), *map(torch.from_numpy, (
        c.cache, c.tables, c.lens, c.cu))))
    out = torch.empty_like(q)
    most = int(c.new.max())

    def run():
        awq.kv4_attention(q, cache, tables, lens, cu_q=None if most == 1 else cu, max_q=most, max_kv=max_kv, out=out)
    return run, out


def buffer(stream):
    return awq.ops.WORKSPACE._bufs.get((dev().index or 0, stream.cuda_stream))


def test_graph_keeps_its_workspace():
    s = torch.cuda.Stream()
    step, out = attention(Case([2000, 700], [1, 1], 4, 2, 128, 16, "f16", seed=1), 2048)
    chunk, _ = attention(Case([2900, 150], [200, 150], 2, 1, 128, 32, "f16", seed=2), 32768)
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    want = out.clone()
    first = buffer(s)
    at, size = first.data_ptr(), first.numel()
    del first
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        chunk()
        assert buffer(s).numel() > size and buffer(s).data_ptr() != at
        # whatever the allocator has to give goes to others now
        others = [torch.full((size,), 0x5A, dtype=torch.uint8, device=dev()) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(t.data_ptr() != at for t in others)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(bool((t == 0x5A).all()) for t in others)
        with torch.cuda.stream(s):
            chunk()
        torch.cuda.synchronize()


def test_captures_without_a_call_before():
    """Two graphs captured on a stream that has no workspace, the second replayed first, eager split calls between."""
    s = torch.cuda.Stream()
    c = synthgen.w4a16_case(1, 4096, 4096, 128)      # counting accumulators
    m = synthgen.w4a16_case(32, 4096, 4096, 128)     # partial quads, the last workgroup to arrive
    a, b = to_dev(c.x, c.qweight, c.scales, c.qzeros), to_dev(m.x, m.qweight, m.scales, m.qzeros)
    step, out = attention(Case([2000, 700], [1, 1], 4, 2, 128, 16, "f16", seed=3), 2048)
    ya, yb = (torch.empty(t[0].shape[0], 4096, dtype=torch.float16, device=dev()) for t in (a, b))

    def work():
        awq.gemv_w4a16(*a, 128, out=ya)
        awq.gemm_w4a16(*b, 128, out=yb)
        step()

    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in (ya, yb, out)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g, stream=s):
            work()
    assert buffer(s) is None

    def same():
        torch.cuda.synchronize()
        ok = [torch.equal(t, w) for t, w in zip((ya, yb, out), want)]
        for t in (ya, yb, out):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        return all(ok)

    assert same()
    for rep in range(3):
        for g in graphs[::-1]:
            g.replay()
            assert same(), rep
            with torch.cuda.stream(s):
                work()
            assert same(), rep
            assert not bool(buffer(s).any())
