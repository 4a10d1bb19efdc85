"""The MLP half of a mixture-of-experts decoder layer, served quantised: experts
in AWQ 4 bits (W4A16) or in block-scaled E4M3.

    hidden state --norm--> router --> each token's experts and the plan
    tokens --gate and up products, grouped by expert, rows gathered by the plan-->
    silu(gate) up --down products, grouped by expert--> weighted sum over a token's experts

A prompt is taken first, then batches of single tokens from a HIP graph; every
step is compared with the same layer computed densely in fp64 from the
experts' values, and the relative error printed (W4A16: activations in 16 bits;
E4M3: activations in 8, about 0.04).

    python examples/moe_block.py [--format w4a16|fp8] [--steps 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_awq_amd as awq  # noqa: E402


class Experts:
    """Matrices [K, N] of E experts in one of the two formats, and the values they stand for."""

    def __init__(self, E, K, N, fmt, dtype, group=128, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.group, self.dtype = fmt, group, dtype
        if fmt == "w4a16":
            q = torch.randint(0, 16, (E, K, N), generator=g, dtype=torch.uint8)
            z = torch.randint(4, 12, (E, K // group, N), generator=g, dtype=torch.uint8)
            s = ((0.5 + torch.rand(E, K // group, N, generator=g)) / (4.6 * K ** 0.5)).to(dtype)
            self.q = torch.stack([awq.pack(e.to(device)) for e in q])
            self.z = torch.stack([awq.pack(e.to(device)) for e in z])
            self.s = s.to(device)
            self.dense = (q.double() - z.double().repeat_interleave(group, 1)) * s.double().repeat_interleave(group, 1)
            return
        # blocks of 128 x 128, each scaled to the largest E4M3 number
        w = torch.randn(E, N, K, generator=g) * K ** -0.5
        nb, kb = -(-N // 128), -(-K // 128)
        pad = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).view(E, nb, 128, kb, 128)
        s = pad.abs().amax((2, 4)) / 448
        codes = (pad / s[:, :, None, :, None]).clamp(-448, 448).reshape(E, nb * 128, kb * 128)[:, :N, :K]
        codes = codes.to(torch.float8_e4m3fn)
        self.q, self.s = codes.contiguous().to(device), s.to(device)
        self.dense = (codes.double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :N, :K])
        self.dense = self.dense.transpose(1, 2)

    def __call__(self, x, offsets, rows=None, top_k=1):
        """x's rows through their experts (rows, top_k: gathered by a plan)."""
        if self.fmt == "w4a16":
            return awq.moe_gemm_w4a16(x, self.q, self.s, self.z, offsets, rows=rows, top_k=top_k, group_size=self.group)
        a, sa = awq.quant_act_fp8_block(x)
        return awq.moe_gemm_fp8_block(a, self.q, sa, self.s, offsets, rows=rows, top_k=top_k, dtype=self.dtype)


class MoEBlock:
    def __init__(self, hidden, inner, experts, top_k, fmt, dtype=torch.float16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.top_k = top_k
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=g)).to(dtype).to(device)
        self.router = (torch.randn(hidden, experts, generator=g) * 2 * hidden ** -0.5).to(dtype).to(device)
        self.gate_up = Experts(experts, hidden, 2 * inner, fmt, dtype, seed=seed + 1, device=device)
        self.down = Experts(experts, inner, hidden, fmt, dtype, seed=seed + 2, device=device)

    def step(self, h, keep=None):
        """h [tokens, hidden], the residual stream; keep: tokens that are not padding (bool).  Returns what the block
        adds to it (0 for padding), the normed state and the plan."""
        x = awq.rmsnorm(h, self.norm)
        logits = (x @ self.router).float()
        if keep is not None:
            logits = logits.masked_fill(~keep[:, None], float("-inf"))  # no expert, no rows
        plan = awq.moe_route(logits, self.top_k, renormalize=True)
        weights, _, offsets, rows, places = plan
        y = self.gate_up(x, offsets, rows, self.top_k)
        gate, up = y.chunk(2, 1)
        y = self.down((torch.nn.functional.silu(gate) * up), offsets)
        return awq.moe_combine(y, weights, places), x, plan

    def dense(self, x, plan):
        """The same from the experts' values in fp64, with the plan's choice and weights."""
        weights, experts = plan[0].double().cpu(), plan[1].cpu()
        x = x.double().cpu()
        out = torch.zeros_like(x)
        for t in range(x.shape[0]):
            for j in range(self.top_k):
                e = int(experts[t, j])
                if e >= 0:
                    gate, up = (x[t] @ self.gate_up.dense[e]).chunk(2)
                    out[t] += weights[t, j] * ((torch.nn.functional.silu(gate) * up) @ self.down.dense[e])
        return out


def run(fmt="w4a16", steps=4, prompt=75, batch=6, hidden=512, inner=384, experts=12, top_k=3, dtype=torch.float16,
        device="cuda"):
    """A prompt (its last fifth padding) and `steps` batches; returns the relative error of each."""
    block = MoEBlock(hidden, inner, experts, top_k, fmt, dtype, device=device)
    g = torch.Generator().manual_seed(1)

    def error(got, x, plan):
        want = block.dense(x, plan)
        return float((got.double().cpu() - want).norm() / want.norm())

    h = torch.randn(prompt, hidden, generator=g).to(dtype).to(device)
    keep = torch.arange(prompt, device=device) < prompt - prompt // 5
    y, x, plan = block.step(h, keep)
    assert not y[~keep].any()
    errors = [error(y, x, plan)]

    # batches of single tokens: one graph, its input filled in place
    h = torch.randn(batch, hidden, generator=g).to(dtype).to(device)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        block.step(h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y, x, plan = block.step(h)
    for _ in range(steps):
        h.copy_(torch.randn(batch, hidden, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        errors.append(error(y, x, plan))
    return errors


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--format", choices=("w4a16", "fp8"), default="w4a16")
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    for i, e in enumerate(run(a.format, a.steps)):
        print("prompt" if i == 0 else f"batch {i}", f"relative error {e:.4f}")
