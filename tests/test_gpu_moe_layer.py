"""Routing, grouped products and the weighted sum together, as a layer runs them.

Bound on the example's error.  W4A16: what differs from fp64 is the rounding of
activations and outputs to 16 bits (half a step 2^-11 or 2^-8 of each value, five
times on the way: two products, silu, its product with up, the sum; and the
weights' where a kernel rounds them): below 7 half steps of the norm.  E4M3: two
quantisations of activations to codes of 4 significant bits, half a step 2^-4 at
worst, evenly spread over it on average 2^-4 / sqrt(3) / 1.4 = 0.026 of the value each;
independent in a sum of many: below 0.026 sqrt(2) sqrt(1 + 1) = 0.052 (the first passes
through gate and up, two factors).  A wrong expert, row or weight gives errors near 1."""
import os
import sys
import threading

import pytest
import torch

import bit_weight_only_awq_amd as awq
from gpu_helpers import dev
from moe_helpers import DT, HALF_STEP, cuda, e4m3_weights, experts_weights, randn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["w4a16", "fp8"])
@pytest.mark.parametrize("kw", [dict(), dict(prompt=300, experts=4, top_k=2, batch=1), dict(prompt=40, experts=70, top_k=8,
                                                                                            hidden=256, inner=128)])
def test_moe_block(fmt, dtype, kw):
    import moe_block
    errors = moe_block.run(fmt, steps=3, dtype=DT[dtype], **kw)
    assert len(errors) == 4 and max(errors) < (7 * HALF_STEP[dtype] if fmt == "w4a16" else 0.052 + 7 * HALF_STEP[dtype])


class Layer:
    """Both formats' products over one routing, few rows an expert or many; every output of a step."""

    def __init__(self, T, E=5, k=2, K=1024, N=264, seed=0):
        self.k = k
        self.q, self.s, self.z = cuda(*experts_weights(E, K, N, 128, True, "f16", seed))
        self.w, self.sw = cuda(*e4m3_weights(E, N, K, seed))
        self.logits, self.x = randn(seed, T, E).to(dev()), randn(seed + 1, T, K).to(torch.float16).to(dev())

    def step(self):
        weights, experts, offsets, rows, places = awq.moe_route(self.logits, self.k)
        y = awq.moe_gemm_w4a16(self.x, self.q, self.s, self.z, offsets, rows=rows, top_k=self.k)
        a, sa = awq.quant_act_fp8_block(self.x)
        v = awq.moe_gemm_fp8_block(a, self.w, sa, self.sw, offsets, rows=rows, top_k=self.k, dtype=torch.float16)
        d = awq.gemm_fp8_block(a, self.w[0], sa, self.sw[0], dtype=torch.float16)
        return (weights, experts, offsets, rows, places, y, a, sa, v, d, awq.moe_combine(y, weights, places),
                awq.moe_combine(v, weights, places))


def same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b, strict=True))


@pytest.mark.parametrize("T,N,K", [(1, 264, 1024), (6, 264, 1024), (40, 264, 1024), (400, 264, 1024), (90, 288, 4096),
                                   (400, 288, 4096)])
def test_graph_replays(T, N, K):
    """One captured step, replayed on other inputs between eager steps: every replay gives the eager step's bits."""
    layer = Layer(T, N=N, K=K)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = layer.step()
    for i in range(4):
        layer.logits.copy_(randn(50 + i, *layer.logits.shape))
        layer.x.copy_(randn(60 + i, *layer.x.shape))
        torch.cuda.synchronize()
        eager = [t.clone() for t in layer.step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(eager, out), i
        assert same(eager, layer.step()), i


def test_two_graphs_and_an_eager_stream():
    """Graphs captured on two streams, and eager steps on a third, in flight together: workspaces of their own."""
    layers = [Layer(3, seed=1), Layer(9, seed=2), Layer(70, seed=3)]
    want = [[t.clone() for t in m.step()] for m in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    graphs, outs = [], []
    for m, s in zip(layers[:2], streams):
        with torch.cuda.stream(s):
            m.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(m.step())
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [layers[2].step() for _ in range(2)]
        torch.cuda.synchronize()
        assert same(want[0], outs[0]) and same(want[1], outs[1]) and all(same(want[2], e) for e in eager)


def test_host_threads():
    """Two threads, each on a stream of its own."""
    layers = [Layer(5, seed=1), Layer(33, seed=2)]
    want = [[t.clone() for t in m.step()] for m in layers]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                out = layers[i].step()
                torch.cuda.current_stream().synchronize()
                if not same(out, want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("call", ["experts", "product", "grouped"])
def test_workspace_is_zero_after(call):
    from bit_weight_only_awq_amd import ops
    for T, N in ((1, 264), (20, 264), (90, 264), (90, 288)):
        m = Layer(T, K=4096, N=N)
        _, _, offsets, rows, _ = awq.moe_route(m.logits, m.k)
        a, sa = awq.quant_act_fp8_block(m.x)
        R, (E, N, K) = T * m.k, m.w.shape
        if call == "experts":
            need = awq.lib().awq_moe_gemm_w4a16_workspace_bytes(R, E, N, K, 128)
            awq.moe_gemm_w4a16(m.x, m.q, m.s, m.z, offsets, rows=rows, top_k=m.k)
        elif call == "product":
            need = awq.lib().awq_fp8_block_gemm_workspace_bytes(T, 0, N, K)
            awq.gemm_fp8_block(a, m.w[0], sa, m.sw[0])
        else:
            need = awq.lib().awq_fp8_block_gemm_workspace_bytes(R, E, N, K)
            awq.moe_gemm_fp8_block(a, m.w, sa, m.sw, offsets, rows=rows, top_k=m.k)
        assert need > 0 or (T, N) == (90, 264)
        torch.cuda.synchronize()
        for buf in ops.WORKSPACE._bufs.values():
            assert not buf.any()
