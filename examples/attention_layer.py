"""The attention half of a decoder layer, served: quantised projections, a paged
cache in Q8_0 or Q4_0, and the attention over it.

A layer's q/k/v and output weights stay resident in Q4_K.  A batch of prompts of
different lengths is answered: one step over the whole prompts, then one token a
step, each step being

    rg_mul_mat   x -> q | k | v       (one fused projection)
    rg_kv_write  k, v -> the cache
    rg_kv_attend q over the cache
    rg_mul_mat   -> the layer's output

The steps of a single token are captured once in a CUDA graph and replayed: the
batch's lengths live in device memory.  Every step is compared with the same
layer computed in 64 bits without a cache.

    python examples/attention_layer.py [--type q8_0|q4_0|f16|bf16] [--steps N]
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_weight_out_gb300 import binding as rg  # noqa: E402
from quantized_weight_out_gb300 import build as rgbuild  # noqa: E402
from quantized_weight_out_gb300 import inputs  # noqa: E402


class Layer:
    """Weights in Q4_K, a cache of the given type, its page table and the step's buffers."""

    def __init__(self, hidden, heads, kv_heads, dim, ctype, seqs, longest, page=64, seed=0):
        self.hidden, self.heads, self.kv, self.dim, self.seqs = hidden, heads, kv_heads, dim, seqs
        self.dev = torch.device("cuda:0")
        rows = (heads + 2 * kv_heads) * dim
        self.rows = rows
        self.w_qkv, self.w_o = (torch.from_numpy(inputs.gen_weight(inputs.Q4_K, n, k, seed=seed, stream=s)).to(self.dev)
                                for n, k, s in ((rows, hidden, 1), (hidden, heads * dim, 2)))
        self.per = -(-longest // page)
        pool = torch.empty(seqs * self.per * rg.rg_kv_page_bytes(ctype, dim, kv_heads, page), dtype=torch.uint8,
                           device=self.dev)
        order = torch.randperm(seqs * self.per, device=self.dev).to(torch.int32)
        self.table = order.view(seqs, self.per).contiguous()
        self.pool = pool
        self.cache = rg.kv_cache(ctype, dim, kv_heads, page, seqs * self.per, pool)
        self.kv_len = torch.zeros(seqs, dtype=torch.int32, device=self.dev)

    def step(self, x, new_start, max_new, stream, out):
        """x [tokens, hidden] F32, the sequences' newest tokens packed; kv_len already counts them."""
        tokens, D = x.shape[0], self.dim
        qkv = torch.empty(tokens, self.rows, device=self.dev)
        att = torch.empty(tokens, self.heads * D, device=self.dev)
        batch = rg.kv_batch(new_start, self.kv_len, self.table, tokens, max_new)
        rg.check(rg.rg_mul_mat(inputs.Q4_K, self.w_qkv, self.rows, self.hidden, x, tokens, qkv, 0.0, stream), "rg_mul_mat")
        k, v = qkv[:, self.heads * D:], qkv[:, (self.heads + self.kv) * D:]
        rg.check(rg.rg_kv_write(self.cache, batch, inputs.F32, k, self.rows, D, v, self.rows, D, stream), "rg_kv_write")
        rg.check(rg.rg_kv_attend(self.cache, batch, inputs.F32, qkv, self.rows, D, self.heads, att, self.heads * D, D,
                                 1 / math.sqrt(D), 0, stream), "rg_kv_attend")
        rg.check(rg.rg_mul_mat(inputs.Q4_K, self.w_o, self.hidden, self.heads * D, att, tokens, out, 0.0, stream),
                 "rg_mul_mat")
        return out

    def plain(self, xs):
        """The layer in 64 bits over one sequence's whole inputs [n, hidden]."""
        def dense(w, n, k):
            out = torch.empty(n, k, device=self.dev)
            rg.check(rg.rg_dequant_async(inputs.Q4_K, w, n, k, out, torch.cuda.current_stream()), "rg_dequant")
            return out.double()
        D, G = self.dim, self.heads // self.kv
        qkv = (xs.double() @ dense(self.w_qkv, self.rows, self.hidden).T).view(len(xs), -1, D)
        q, k, v = qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv], qkv[:, self.heads + self.kv:]
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(D)
        s = s.masked_fill(torch.ones_like(s[0], dtype=torch.bool).triu(1), -math.inf)
        o = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v).reshape(len(xs), -1)
        return o @ dense(self.w_o, self.hidden, self.heads * D).T


def run(ctype=inputs.Q8_0, prompts=(93, 17, 300, 64), steps=8, hidden=1024, heads=8, kv_heads=2, dim=128, seed=0,
        verbose=True):
    """Answers the prompts; returns the largest relative error (2-norm) of a step."""
    rgbuild.build()
    S = len(prompts)
    L = Layer(hidden, heads, kv_heads, dim, ctype, S, max(prompts) + steps, seed=seed)
    g = torch.Generator(device=L.dev).manual_seed(seed)
    xs = [torch.randn(n + steps, hidden, generator=g, device=L.dev) for n in prompts]
    want = [L.plain(x) for x in xs]
    worst = 0.0

    def compare(got, ref):
        nonlocal worst
        worst = max(worst, float((got.double() - ref).norm() / ref.norm()))

    # the prompts, packed
    start = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device=L.dev)
    L.kv_len += torch.tensor(prompts, dtype=torch.int32, device=L.dev)
    x = torch.cat([xs[s][:n] for s, n in enumerate(prompts)])
    out = L.step(x, start, max(prompts), torch.cuda.current_stream(), torch.empty_like(x))
    compare(out, torch.cat([want[s][:n] for s, n in enumerate(prompts)]))
    # one token a sequence and step, replayed
    one = torch.arange(S + 1, dtype=torch.int32, device=L.dev)
    x, out = torch.empty(S, hidden, device=L.dev), torch.empty(S, hidden, device=L.dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # every allocation and lookup once before the capture (kv_len still
        L.step(x.zero_(), one, 1, side, out)  # names prompt tokens: the prompts are stored again below)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.kv_len += 1
        L.step(x, one, 1, torch.cuda.current_stream(), out)
    xp = torch.cat([xs[s][:n] for s, n in enumerate(prompts)])
    L.step(xp, start, max(prompts), torch.cuda.current_stream(), torch.empty_like(xp))
    spent = 0.0
    for i in range(steps):
        x.copy_(torch.stack([xs[s][n + i] for s, n in enumerate(prompts)]))
        torch.cuda.synchronize()
        t = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        spent += time.perf_counter() - t
        compare(out, torch.stack([want[s][n + i] for s, n in enumerate(prompts)]))
    rg.check(rg.rg_check(torch.cuda.current_stream()), "rg_check")
    if verbose:
        print(f"{inputs.TYPE_NAMES[ctype]} cache, prompts of {list(prompts)} tokens, {steps} steps: largest relative "
              f"error of a step {worst:.2e}, {spent / steps * 1e6:.0f} us a step")
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--type", default="q8_0", choices=["q8_0", "q4_0", "f16", "bf16"])
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    run(inputs.NAME_TO_TYPE[a.type], steps=a.steps)
