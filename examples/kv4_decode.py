"""One attention layer of a decoder on 4-bit weights and a 4-bit key/value cache.

    python examples/kv4_decode.py [--steps 24] [--budget 256]

Random weights of a Qwen2.5-1.5B-shaped layer (1536 wide, 12 query heads on 2 key/value heads of
128). Three prompts of mixed lengths enter the paged cache together (w4a16_matmul, kv4_append,
kv4_attention with the weight every cached token receives), kv4_evict keeps the budget's heaviest
tokens a head, and decoding goes on from there, a token a sequence and step. One step is captured
in a CUDA graph and replayed: lengths, page table and weights live on the device. A model would
rotate q and k between the projection and the append.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_w4a16_group_gb300 as w4  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM = 1536, 12, 2, 128
GROUP, PAGE = 64, 64


def projection(n: int, k: int, gen) -> tuple:
    """W4A16 weights (packed, scales, minimums) of an n x k layer."""
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    codes, scales, mins = w4.w4a16_quantize(w)
    return w4.w4a16_pack(codes), scales, mins


def starts_of(counts) -> torch.Tensor:
    return torch.tensor([0, *counts], device="cuda").cumsum(0).to(torch.int32)


class Layer:
    """Projections, cache and page tables of one layer for a batch of sequences."""

    def __init__(self, batch: int, longest: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.qkv = projection((HEADS + 2 * KV_HEADS) * DIM, HIDDEN, gen)
        self.out = projection(HIDDEN, HEADS * DIM, gen)
        width = (longest + PAGE - 1) // PAGE
        self.cache = w4.kv4_cache(batch * width * 2, KV_HEADS, DIM, PAGE, GROUP)
        # a serving system hands pages out as sequences grow; here each has its own from the start,
        # and a second set for the tokens that an eviction keeps
        pages = torch.randperm(batch * width * 2, generator=gen, device="cuda").to(torch.int32)
        self.table, self.spare = pages.view(2, batch, width).unbind(0)
        self.table, self.spare = self.table.contiguous(), self.spare.contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.weights = torch.zeros(batch, KV_HEADS, width * PAGE, device="cuda")
        self.longest = width * PAGE

    def __call__(self, x, starts, max_new: int, workspace=None):
        """x bf16 [tokens, 1536], the sequences' new tokens one after the other -> the same."""
        self.lens.add_(starts[1:] - starts[:-1])
        qkv = w4.w4a16_matmul(x, *self.qkv).view(x.shape[0], -1, DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        w4.kv4_append(self.cache, self.table, self.lens, starts, k, v, group=GROUP,
                      weights=self.weights)
        y = w4.kv4_attention(q, self.cache, self.table, self.lens, starts, self.longest, max_new,
                             group=GROUP, weights=self.weights, weights_out=self.weights,
                             workspace=workspace)
        self.q, self.y = q, y
        return x + w4.w4a16_matmul(y.view(x.shape[0], -1), *self.out)

    def evict(self, budget: int, first: int = 4, recent: int = 32):
        kept, lens, weights = w4.kv4_evict(
            self.cache, self.table, self.lens, self.weights, self.spare, budget, self.longest, DIM,
            first=first, recent=recent, group=GROUP)
        self.table, self.spare = self.spare, self.table
        self.lens.copy_(lens)
        self.weights[..., :budget] = weights
        return kept


def main(steps: int = 24, budget: int = 256, lengths=(700, 300, 90)) -> dict:
    batch = len(lengths)
    layer = Layer(batch, max(lengths) + steps + 1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randn(sum(lengths), HIDDEN, generator=gen, device="cuda").bfloat16()
    hidden = layer(prompt, starts_of(lengths), max(lengths))
    ends = starts_of(lengths)[1:].long() - 1
    kept = layer.evict(budget)

    one = starts_of([1] * batch)
    workspace = torch.zeros(w4.kv4_attention_workspace_bytes(
        batch, batch, 1, layer.longest, HEADS, KV_HEADS, DIM, GROUP, True), dtype=torch.uint8,
        device="cuda")
    x = hidden[ends].contiguous()
    x.copy_(layer(x, one, 1, workspace))       # warm-up, and the first step
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(layer(x, one, 1, workspace))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()

    # the last step against the values that the cache holds
    lens = layer.lens.tolist()
    k, v = w4.kv4_read(layer.cache, layer.table, layer.lens, starts_of(lens), sum(lens), DIM,
                       group=GROUP)
    worst = 0.0
    for b, (n, lo) in enumerate(zip(lens, starts_of(lens).tolist())):
        for h in range(HEADS):
            kv = h // (HEADS // KV_HEADS)
            s = k[lo:lo + n, kv].double() @ layer.q[b, h].double() * DIM ** -0.5
            want = torch.softmax(s, 0) @ v[lo:lo + n, kv].double()
            worst = max(worst, ((layer.y[b, h].double() - want).norm() / want.norm()).item())
    bf16 = 2 * KV_HEADS * DIM * 2
    here = KV_HEADS * (DIM + 8 * DIM // GROUP)
    return {"lengths": list(lengths), "kept a head": [int((r >= 0).sum()) for r in kept[:, 0]],
            "lengths now": lens, "us a step (graph)": begin.elapsed_time(end) * 1e3 / steps,
            "bytes a cached token": here, "in BF16": bf16, "status": w4.w4a16_device_status(),
            "largest relative error of a head": worst}


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=24)
    p.add_argument("--budget", type=int, default=256)
    args = p.parse_args()
    for key, value in main(args.steps, args.budget).items():
        print(f"{key}: {value}")
