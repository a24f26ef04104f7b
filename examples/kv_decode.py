"""Serving one attention layer from a paged NVFP4 key/value cache.

Prompts of several requests are planned, appended and attended, then tokens
are decoded one per request: page plan, norm + rotation + quantizing append
and attention captured once in a HIP graph and replayed per token.  A request
that ends gives its pages back, and a new one takes them.  Weights and inputs
are random; the last step is checked against plain attention over the values
that the cache holds.

  python examples/kv_decode.py [--requests 8] [--tokens 32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_02_amd as nv  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 32, 8, 128, 16


class Layer:
    """One attention layer's weights, its cache and its requests."""

    def __init__(self, requests, width, hidden=1024, device="cuda"):
        g = torch.Generator(device=device).manual_seed(0)
        rand = lambda *n: torch.randn(*n, device=device, generator=g)  # noqa: E731
        rows = (HEADS + 2 * KV_HEADS) * DIM
        self.qkv = (rand(hidden, rows) * hidden ** -0.5).bfloat16()
        self.q_weight, self.k_weight = (1 + 0.1 * rand(2, DIM)).bfloat16().unbind(0)
        self.cos, self.sin = nv.rope_table(width * PAGE, DIM, device=device)
        # amaxes as a calibration run gives them: a normed key's largest value
        # is about sqrt(DIM), a value's a few deviations
        full = lambda v: torch.full((KV_HEADS,), v, device=device)  # noqa: E731
        self.pages = requests * width
        self.cache = nv.kv_cache(self.pages, KV_HEADS, PAGE, DIM, full(12.0), full(6.0))
        ints = lambda *n: torch.zeros(*n, dtype=torch.int32, device=device)  # noqa: E731
        self.ctx, self.table = ints(requests), ints(requests, width)
        self.free = torch.arange(self.pages, dtype=torch.int32, device=device)
        self.count = torch.full((1,), self.pages, dtype=torch.int32, device=device)
        # the layer's own, as its steps are captured: long sequences are joined in one launch
        self.counters = torch.zeros(nv.KV_COUNTER_BYTES, dtype=torch.uint8, device=device)

    def step(self, x, new, one_each):
        """x [tokens, hidden] bf16: the requests' new tokens one after another
        (new [requests] of them); returns (attention output, plan)."""
        p = nv.kv_plan(self.ctx, new, self.table, self.free, self.count, page_size=PAGE,
                       num_pages=self.pages, tokens=x.shape[0])
        y = (x @ self.qkv).view(x.shape[0], -1, DIM)
        q, k, v = y.split((HEADS, KV_HEADS, KV_HEADS), 1)  # views: nothing is copied
        q = nv.kv_append(self.cache, k, v, p.slots, q=q, positions=p.positions, cos=self.cos,
                         sin=self.sin, q_weight=self.q_weight, k_weight=self.k_weight)
        out = nv.kv_attention(q, self.cache, self.table, p.seq_lens, None if one_each else p.cu_new,
                              counters=self.counters)
        self.ctx.copy_(p.seq_lens)
        self.count.copy_(p.free_count)
        self.q = q
        return out, p

    def release(self, request):
        """Gives a request's pages back: their numbers go on top of the stack."""
        n = -(-int(self.ctx[request]) // PAGE)
        top = int(self.count)
        self.free[top:top + n] = self.table[request, :n]
        self.count += n
        self.ctx[request] = 0


def plain(layer, request):
    """Attention of a request's last query over what the cache holds for it, in 32 bits."""
    n = int(layer.ctx[request])
    j = torch.arange(n, device="cuda")
    k, v = nv.kv_read(layer.cache, layer.table[request].long()[j // PAGE] * PAGE + j % PAGE)
    q = layer.q[request].float().view(KV_HEADS, -1, DIM)
    w = torch.softmax(q @ k.float().permute(1, 2, 0).contiguous() * DIM ** -0.5, -1)
    return (w @ v.float().transpose(0, 1).contiguous()).view(HEADS, DIM)


def main(requests=8, tokens=32, prompt=200):
    width = -(-(prompt + 2 * tokens + PAGE) // PAGE) + 1
    layer = Layer(requests, width)
    g = torch.Generator(device="cuda").manual_seed(1)
    # prompts of different lengths in one call
    lens = [max(1, prompt - 17 * b % prompt) for b in range(requests)]
    new = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), layer.qkv.shape[0], device="cuda", generator=g).bfloat16()
    _, p = layer.step(x, new, False)
    assert int(p.refused) == 0 and layer.ctx.tolist() == lens
    # decoding: one token each, captured once
    x = torch.randn(requests, layer.qkv.shape[0], device="cuda", generator=g).bfloat16()
    new = torch.ones(requests, dtype=torch.int32, device="cuda")
    layer.step(x, new, True)  # allocates what the capture needs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = layer.step(x, new, True)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(tokens):
        x.normal_(generator=g)
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - began) / tokens * 1e6
    # one request ends and another takes its place in the running batch
    layer.release(0)
    x.normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    assert layer.ctx.tolist() == [1] + [n + tokens + 2 for n in lens[1:]]
    worst = 0.0
    for b in range(requests):
        want = plain(layer, b)
        worst = max(worst, float((out[b].float() - want).norm() / want.norm()))
    print(f"{requests} requests, {tokens} tokens each: {us:.1f} us a decode step; "
          f"last step against plain attention over the cache: {worst:.2e} relative")
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args()
    sys.exit(0 if main(a.requests, a.tokens) < 1e-2 else 1)
