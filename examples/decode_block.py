"""The attention block of a decoder layer, prompt and decode steps, on one GPU:

    qkv = x W_qkv^T                             skinny_gemm_residual
    q   = norm, rotation; k, v to the cache     sgr_kv_append
    o   = attention over the cache              sgr_kv_attention
    y   = o W_out^T + x                         skinny_gemm_residual

Prompts of different lengths go through together, in chunks of at most
--chunk tokens a sequence; then each step adds one token a sequence, and one
CUDA graph of the block serves every step: the lengths are device data, the
block table names all the pages from the start.

    python examples/decode_block.py [--batch 32] [--prompt 2000] [--steps 64]

Weights and inputs are random.  The last step's output is compared with the
same block in 32 bits without a cache, and the time of a step is printed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import skinny_bf16_gemm_residual_gb300 as sgr  # noqa: E402


def rotation_table(positions: int, dim: int, base: float = 10000.0):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** -(torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([angle.cos(), angle.sin()], -1).float().cuda()


class Block:
    """Weights, cache and batch of one layer."""

    def __init__(self, batch, max_len, heads, kv_heads, dim, page, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.heads, self.kv_heads, self.dim, self.width = heads, kv_heads, dim, heads * dim
        self.w_qkv = (randn((heads + 2 * kv_heads) * dim, self.width) / self.width ** 0.5).bfloat16()
        self.w_out = (randn(self.width, self.width) / self.width ** 0.5).bfloat16()
        self.rope = sgr.RopeNorm(rotation_table(max_len, dim), q_weight=(1 + 0.1 * randn(dim)).bfloat16(),
                                 k_weight=(1 + 0.1 * randn(dim)).bfloat16())
        pages = -(-max_len // page)
        self.cache = sgr.KvCache.empty(batch * pages, kv_heads, page, dim)
        self.table = torch.randperm(batch * pages, device="cuda", generator=g).int().view(batch, pages)
        self.seq_len = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def step(self, x, batch, workspace=None):
        """x [tokens, heads * dim] -> y, the batch's new tokens appended."""
        tokens = x.shape[0]
        none = torch.zeros(tokens, self.w_qkv.shape[0], dtype=torch.bfloat16, device=x.device)
        qkv = sgr.skinny_gemm_residual(x, self.w_qkv, none).view(tokens, -1, self.dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)  # slices, not copies
        q = sgr.sgr_kv_append(self.cache, batch, k, v, self.rope, q=q, q_out=q)
        o = sgr.sgr_kv_attention(self.cache, batch, q, workspace=workspace)
        return sgr.skinny_gemm_residual(o.view(tokens, self.width), self.w_out, x)


def plain(block: Block, x):
    """The block over one whole sequence x [tokens, width] in 32 bits: the last token's output."""
    x = x.float()
    qkv = (x @ block.w_qkv.float().t()).view(x.shape[0], -1, block.dim)
    q, k, v = qkv.split((block.heads, block.kv_heads, block.kv_heads), 1)
    table = block.rope.table[:x.shape[0], None]
    cos, sin = table.chunk(2, -1)

    def rotate(t, w):
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = t.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k = rotate(q, block.rope.q_weight)[-1], rotate(k, block.rope.k_weight)
    group = block.heads // block.kv_heads
    k, v = (t.repeat_interleave(group, 1) for t in (k, v))
    p = (torch.einsum("hd,thd->ht", q, k) * block.dim ** -0.5).softmax(-1)
    return torch.einsum("ht,thd->hd", p, v).reshape(1, -1) @ block.w_out.float().t() + x[-1:]


def run(batch=32, prompt=2000, chunk=512, steps=64, heads=28, kv_heads=4, dim=128, page=64, seed=0):
    """Returns (largest error, largest magnitude, microseconds a step)."""
    lens = [max(1, prompt - 37 * (i % 8)) for i in range(batch)]  # ragged prompts
    max_len = max(lens) + steps
    block = Block(batch, max_len, heads, kv_heads, dim, page, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    xs = [torch.randn(n + steps, block.width, device="cuda", generator=g).bfloat16() for n in lens]

    # Prompts, a chunk of every unfinished one at a time.
    done = [0] * batch
    while any(d < n for d, n in zip(done, lens)):
        new = [min(chunk, n - d) for d, n in zip(done, lens)]
        x = torch.cat([t[d:d + n] for t, d, n in zip(xs, done, new)])
        done = [d + n for d, n in zip(done, new)]
        block.seq_len.copy_(torch.tensor(done, dtype=torch.int32))
        start = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        block.step(x, sgr.KvBatch(block.table, block.seq_len, start, tokens=sum(new), max_new=max(new)))

    # Decode steps: one graph, whose lengths grow by one a replay.
    rows = sgr.KvBatch(block.table, block.seq_len)  # one row a sequence
    workspace = sgr.kv_attention_workspace(block.cache, rows, heads)
    x = torch.empty(batch, block.width, dtype=torch.bfloat16, device="cuda")
    new_x = torch.stack([t[n:] for t, n in zip(xs, lens)], 1)  # [steps, batch, width]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.seq_len.add_(1)
        y = block.step(x, rows, workspace)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for i in range(steps):
        x.copy_(new_x[i])
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    code = sgr.sgr_device_error(0)
    if code:
        raise RuntimeError(f"device error word {code}")
    want = torch.cat([plain(block, t) for t in xs])
    return (y.float() - want).abs().max().item(), want.abs().max().item(), begin.elapsed_time(end) * 1e3 / steps


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 32), ("prompt", 2000), ("chunk", 512), ("steps", 64), ("heads", 28), ("kv-heads", 4),
                        ("dim", 128), ("page", 64)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    torch.backends.cuda.matmul.allow_tf32 = False
    error, largest, us = run(a.batch, a.prompt, a.chunk, a.steps, a.heads, a.kv_heads, a.dim, a.page)
    print(f"{a.batch} sequences, prompts of up to {a.prompt} tokens, {a.steps} steps: {us:.1f} us a step, "
          f"largest error {error:.4f} of {largest:.2f}")


if __name__ == "__main__":
    main()
