"""One attention layer over a paged 8-bit cache: prompts in, then steps of one
or several tokens per request.

    python examples/paged_attention.py

A step is q, k, v projections (4-bit weights), a plan (which blocks the new
tokens take, which rows they are), the append, the attention and the output
projection.  Nothing is read back to the host between the steps, so a step of
a fixed shape is captured once as a CUDA graph and replayed: its lengths, block
tables and free list live on the device.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from skinny_gemm_gb300 import ops, synth  # noqa: E402


class Layer:
    """Grouped-query attention with W4A16 projections and its part of the cache."""

    def __init__(self, hidden, q_heads, kv_heads, dim, blocks, block, seed=0, window=0):
        self.q_heads, self.kv_heads, self.dim, self.window = q_heads, kv_heads, dim, window
        shapes = [(q_heads * dim, hidden), (kv_heads * dim, hidden), (kv_heads * dim, hidden), (hidden, q_heads * dim)]
        self.wq, self.wk, self.wv, self.wo = (
            ops.W4Matrix.from_host(synth.make_weights(seed + i, n, k)) for i, (n, k) in enumerate(shapes))
        self.cache = ops.KVCache.empty(blocks, kv_heads, block, dim)

    def __call__(self, x, plan, table, max_new, max_len):
        T = x.shape[0]
        ws = [self.wq, self.wk, self.wv]
        q, k, v = ops.mm_group([x] * 3, ws) if T <= 8 else [ops.mm(x, w) for w in ws]
        ops.kv_append(k.view(T, self.kv_heads, self.dim), v.view(T, self.kv_heads, self.dim), self.cache, plan.slots)
        y = ops.kv_attention(q.view(T, self.q_heads, self.dim), self.cache, table, plan.cu, plan.lens, max_new, max_len,
                             window=self.window)
        return ops.mm(y.view(T, -1), self.wo)


class Requests:
    """Lengths, block tables and the free list of a batch, on the device."""

    def __init__(self, B, max_len, blocks, block):
        self.B, self.block, self.max_len = B, block, max_len
        self.cached = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.table = torch.full((B, max_len // block), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(blocks, device="cuda").to(torch.int32)  # any order will do
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, layer, x, new, max_new):
        """One step: new (int32 [B] on the device, at most max_new each) tokens of each request, the rows of x."""
        plan = ops.kv_plan(self.cached, new, self.table, self.free, x.shape[0], self.block, head=self.head)
        y = layer(x, plan, self.table, max_new, self.max_len)
        self.cached.copy_(plan.lens)
        self.head.copy_(plan.head)
        return y


def run(hidden=2560, q_heads=8, kv_heads=2, dim=256, block=64, prompts=(700, 64, 5), steps=32, draft=4, max_len=4096,
        report=print):
    """Prompts, `steps` one-token steps by graph replay, one step of `draft` tokens per request; the last step's output."""
    torch.manual_seed(0)
    B = len(prompts)
    blocks = B * (max_len // block)
    layer, reqs = Layer(hidden, q_heads, kv_heads, dim, blocks, block), Requests(B, max_len, blocks, block)

    def rows(n):
        return torch.randn(n, hidden, device="cuda").to(torch.bfloat16)

    reqs.step(layer, rows(sum(prompts)), torch.tensor(prompts, dtype=torch.int32, device="cuda"), max(prompts))
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    reqs.step(layer, rows(B), one, 1)  # (the first call of this shape, outside capture: workspaces are made)
    torch.cuda.synchronize()
    x, graph = rows(B), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = reqs.step(layer, x, one, 1)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(steps):
        if i == steps // 2:
            start.record()
        graph.replay()
        x.copy_(out / out.float().abs().amax(-1, keepdim=True).clamp_min(1e-6))  # stands in for the rest of a model
    end.record()
    y = reqs.step(layer, rows(B * draft), one * draft, draft)
    lens = [n + 1 + steps + draft for n in prompts]
    assert reqs.cached.tolist() == lens and ops.device_status() == 0
    assert int(reqs.head) == sum(-(-n // block) for n in lens)
    report(f"{B} requests of {lens} tokens, cache {layer.cache.nbytes / 1e6:.0f} MB; "
           f"one-token step {start.elapsed_time(end) / (steps - steps // 2) * 1e3:.1f} us")
    return layer, reqs, y


if __name__ == "__main__":
    run()
