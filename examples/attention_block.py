"""The attention half of a decoder layer, served in 4 bits: weights W4A8, keys
and values in the paged 4-bit cache.

    hidden state --norm, int8 codes--> QKV product --rotary append--> cache
    rotated queries --attention over the cache--> output product
    output + residual --norm, int8 codes--> (the MLP half would follow)

Two ragged prompts are taken in one step, then tokens one at a time from a HIP
graph; every step is compared with the same layer computed densely in fp64
from the unquantised keys and values, and the relative error printed (4-bit
keys and values of random data: about 0.16).

    python examples/attention_block.py [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_awq_amd as awq  # noqa: E402


class AttentionBlock:
    """Weights and cache of one layer; sequences own rows of the page table."""

    def __init__(self, hidden, heads, kv_heads, head_dim, page, sequences, max_len, dtype=torch.float16, seed=0,
                 device="cuda"):
        self.heads, self.kv_heads, self.dim, self.page, self.max_len = heads, kv_heads, head_dim, page, max_len
        self.width = (heads + 2 * kv_heads) * head_dim
        g = torch.Generator().manual_seed(seed)

        def weights(k, n):  # (packed, scales, the matrix they stand for)
            w = torch.randint(-8, 8, (k, n), generator=g, dtype=torch.int8)
            s = (0.5 + torch.rand(n, generator=g)) / (4.6 * k ** 0.5)
            return awq.pack(w.to(device), "k8"), s.to(dtype).to(device), w.double() * s.to(dtype).double()

        self.qkv, self.qkv_scale, self.qkv_dense = weights(hidden, self.width)
        self.out, self.out_scale, self.out_dense = weights(heads * head_dim, hidden)
        self.norm_in = (1 + 0.1 * torch.randn(hidden, generator=g)).to(dtype).to(device)
        self.norm_post = (1 + 0.1 * torch.randn(hidden, generator=g)).to(dtype).to(device)
        self.rope = awq.rope_table(max_len, head_dim, device=device)
        pages = -(-max_len // page)
        self.cache = awq.kv4_cache(sequences * pages, kv_heads, head_dim, page, device=device)
        self.tables = torch.randperm(sequences * pages, generator=g).view(sequences, pages).to(torch.int32).to(device)

    def slots(self, seq, pos):
        """Where token `pos` of sequence `seq` is kept (int64 tensors, elementwise)."""
        page = self.tables[seq, pos // self.page].long()
        return page * self.page + pos % self.page

    def step(self, x, residual, positions, slots, lens, cu_q=None, max_q=1, max_kv=None):
        """x [tokens, hidden]: what the layer before adds to the residual
        stream.  Returns the int8 codes and scales for the MLP half, and the
        residual stream."""
        a8, s1, residual = awq.rmsnorm_quant(x, self.norm_in, residual=residual)
        qkv = awq.w4a8_gemm(a8, self.qkv, s1, self.qkv_scale).view(-1, self.width // self.dim, self.dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        q = awq.kv4_append(q, k, v, self.rope, positions, slots, self.cache)
        o = awq.kv4_attention(q, self.cache, self.tables, lens, cu_q=cu_q, max_q=max_q,
                              max_kv=max_kv or self.max_len)
        y = awq.linear_w4a8(o.view(o.shape[0], -1), self.out, self.out_scale)
        return awq.rmsnorm_quant(y, self.norm_post, residual=residual)

    def dense(self, h):
        """The residual stream after the block for one sequence's h [tokens, hidden], in fp64, nothing quantised
        but the weights."""
        h = h.double().cpu()
        n, D, G = h.shape[0], self.dim, self.heads // self.kv_heads
        x = h * (h.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * self.norm_in.double().cpu()
        q, k, v = (x @ self.qkv_dense).view(n, -1, D).split((self.heads, self.kv_heads, self.kv_heads), 1)
        cos, sin = self.rope[:n].double().cpu()[:, None].chunk(2, -1)

        def turn(t):
            a, b = t.chunk(2, -1)
            return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

        q, k = turn(q).transpose(0, 1), turn(k).transpose(0, 1).repeat_interleave(G, 0)
        v = v.transpose(0, 1).repeat_interleave(G, 0)
        scores = (q @ k.transpose(1, 2)) * D ** -0.5
        scores = scores.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf"))
        o = (scores.softmax(-1) @ v).transpose(0, 1).reshape(n, -1)
        return h + o @ self.out_dense


def run(steps=8, prompts=(37, 150), hidden=1024, heads=8, kv_heads=2, head_dim=128, page=16, dtype=torch.float16,
        device="cuda"):
    """Serves the prompts and `steps` more tokens; returns the relative error of each step."""
    B = len(prompts)
    block = AttentionBlock(hidden, heads, kv_heads, head_dim, page, B, max(prompts) + steps, dtype, device=device)
    g = torch.Generator().manual_seed(1)
    streams = [torch.randn(n + steps, hidden, generator=g).to(dtype).to(device) for n in prompts]
    zeros = torch.zeros(sum(prompts), hidden, dtype=dtype, device=device)

    def error(got, step):
        worst = 0.0
        for b, n in enumerate(prompts):
            want = block.dense(streams[b][:n + step])[-1] - streams[b][n + step - 1].double().cpu()
            have = got[b].double().cpu() - streams[b][n + step - 1].double().cpu()
            worst = max(worst, float((have - want).norm() / want.norm()))
        return worst

    # the prompts, both in one step
    pos = torch.cat([torch.arange(n) for n in prompts]).to(device)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(prompts)]).to(device)
    lens = torch.tensor(prompts, dtype=torch.int32, device=device)
    cu_q = torch.tensor([0, *prompts], dtype=torch.int32, device=device).cumsum(0, dtype=torch.int32)
    x = torch.cat([s[:n] for s, n in zip(streams, prompts)])
    _, _, h = block.step(x, zeros, pos.int(), block.slots(seq, pos), lens, cu_q, max(prompts))
    errors = [error(h[(cu_q[1:] - 1).long()], 0)]

    # then a token of each at a time: one graph, its inputs filled in place
    x, zero = torch.empty(B, hidden, dtype=dtype, device=device), torch.zeros(B, hidden, dtype=dtype, device=device)
    seq, pos = torch.arange(B, device=device), torch.zeros(B, dtype=torch.int32, device=device)
    slots = torch.full((B,), -1, dtype=torch.int64, device=device)  # (nothing is stored while warming up)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    x.zero_()
    with torch.cuda.stream(stream):
        block.step(x, zero, pos, slots, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        _, _, h = block.step(x, zero, pos, slots, lens)
    for i in range(steps):
        x.copy_(torch.stack([s[n + i] for s, n in zip(streams, prompts)]))
        pos.copy_(lens)
        slots.copy_(block.slots(seq, lens.long()))
        lens += 1
        graph.replay()
        torch.cuda.synchronize()
        errors.append(error(h, i + 1))
    return errors


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=8)
    for i, e in enumerate(run(p.parse_args().steps)):
        print("prompts" if i == 0 else f"token {i}", f"relative error {e:.3f}")
