#!/usr/bin/env python3
"""One attention layer decoding on operands held in few bits.

The layer's two weight matrices (queries, keys and values together, and the
output) are kept in 4 bits, its keys and values in a paged 8-bit cache.  Ragged
prompts are taken in first -- their many rows go through the weights' bfloat16
values and the ordinary product --, then every step sends one row of each
sequence through

    gemm_w4 -> kv_append -> kv_attention -> gemm_w4

recorded once as a CUDA graph.  At the end the last step is computed again in
float32 from the weights' values and the cache's, read back.

    python examples/decode_step.py [--batch 8] [--steps 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from accelerator_gb300 import binding, lowbit  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, PAGE = 1024, 16, 4, 64, 32


class Layer:
    def __init__(self, generator):
        def weight(rows, columns):
            return torch.randn(rows, columns, generator=generator, device="cuda") * rows ** -0.5
        self.qkv = lowbit.w4_quantize(weight(HIDDEN, (Q_HEADS + 2 * KV_HEADS) * DIM), group=64)
        self.out = lowbit.w4_quantize(weight(Q_HEADS * DIM, HIDDEN), group=64)

    @staticmethod
    def heads(joint):
        """Queries, keys and values: three slices of one array, rows x heads x dim."""
        joint = joint.view(joint.shape[0], -1, DIM)
        return joint.split((Q_HEADS, KV_HEADS, KV_HEADS), 1)

    def prompt(self, x, cache, table, starts, first, lengths):
        joint = binding.gemm(x, lowbit.w4_dequantize(self.qkv), mode="bf16").to(torch.bfloat16)
        q, k, v = self.heads(joint)
        lowbit.kv_append(cache, k, v, table, starts, first)
        o = lowbit.kv_attention(q, cache, table, starts, lengths)
        return binding.gemm(o.flatten(1), lowbit.w4_dequantize(self.out), mode="bf16").to(torch.bfloat16)

    def step(self, x, cache, table, starts, first, lengths):
        q, k, v = self.heads(lowbit.gemm_w4(x, self.qkv))
        lowbit.kv_append(cache, k, v, table, starts, first)
        o = lowbit.kv_attention(q, cache, table, starts, lengths)
        return lowbit.gemm_w4(o.flatten(1), self.out)

    def plain_step(self, x, cache, table, lengths):
        """The step in float32, over the tokens that the cache holds."""
        q, _, _ = self.heads((x.float() @ lowbit.w4_dequantize(self.qkv, dtype=torch.float32)).to(torch.bfloat16))
        starts = torch.zeros(len(lengths) + 1, dtype=torch.int32, device="cuda")
        starts[1:] = lengths.cumsum(0)
        k, v = lowbit.kv_read(cache, table, starts, torch.zeros_like(lengths), int(starts[-1]), dtype=torch.float32)
        rows = []
        for b, (lo, hi) in enumerate(zip(starts[:-1].tolist(), starts[1:].tolist())):
            keys, values = (t[lo:hi].repeat_interleave(Q_HEADS // KV_HEADS, 1) for t in (k, v))
            a = torch.einsum("hd,nhd->hn", q[b].float(), keys) * DIM ** -0.5
            rows.append(torch.einsum("hn,nhd->hd", a.softmax(-1), values).flatten())
        o = torch.stack(rows).to(torch.bfloat16).float()
        return o @ lowbit.w4_dequantize(self.out, dtype=torch.float32)


def main(batch=8, steps=64, report=print):
    g = torch.Generator(device="cuda").manual_seed(0)
    layer = Layer(g)
    prompts = [5 + 37 * b % 200 for b in range(batch)]
    width = -(-(max(prompts) + steps) // PAGE)
    cache = lowbit.KvCache.empty(batch * width, KV_HEADS, DIM, PAGE)
    table = torch.randperm(batch * width, generator=g, device="cuda").to(torch.int32).view(batch, width)
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    first = torch.zeros_like(lengths)
    starts = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    starts[1:] = lengths.cumsum(0)
    x = torch.randn(sum(prompts), HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
    y = layer.prompt(x, cache, table, starts, first, lengths)
    x = y[starts[1:].long() - 1].clone()

    one = torch.arange(batch + 1, dtype=torch.int32, device="cuda")

    def step():
        first.copy_(lengths)
        lengths.add_(1)
        return layer.step(x, cache, table, one, first, lengths)

    x.copy_(torch.nn.functional.normalize(step().float(), dim=1) * HIDDEN ** 0.5)      # the first step outside of the graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps - 2):
        graph.replay()
        x.copy_(torch.nn.functional.normalize(y.float(), dim=1) * HIDDEN ** 0.5)
    end.record()
    graph.replay()
    torch.cuda.synchronize()
    status = binding.debug_status()
    if status != binding.OK:
        raise RuntimeError(binding.status_string(status))
    want = layer.plain_step(x, cache, table, lengths)
    error = ((y.float() - want).norm() / want.norm()).item()
    report(f"{batch} sequences of {int(lengths.min())} to {int(lengths.max())} tokens: "
           f"{begin.elapsed_time(end) / max(steps - 2, 1) * 1e3:.1f} us a step, {error:.1e} off float32")
    return error


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    main(a.batch, max(a.steps, 3))
