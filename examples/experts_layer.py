"""A layer of experts on a resident table, trained and served.

The table (Q6_K or any type) and the experts' weights stay resident in their
block types.  A step over a batch of tokens is

    rg_get_rows    token numbers -> x                      (the table's rows, scaled)
    rg_mul_mat     x -> the router's logits
    rg_route       logits -> experts, weights, slots by expert
    rg_mul_mat_id  x -> gate, up                           (a row per slot)
    rg_mul_mat_id  silu(gate) * up -> y                    (summed by the weights)

and back from the gradient of y

    rg_out_prod_id dy -> the slots' dh, their dot products with h the weights' gradient
    rg_out_prod_id dgate, dup -> dx                        (summed by token)
    rg_route_back  the weights' gradient -> dlogits;  rg_out_prod dlogits -> dx
    rg_get_rows_back dx -> the gradient of an adapter on the table, by token.

The forward is also captured in a CUDA graph for single decoding steps.  Both
directions are compared with the same layer in 64 bits.

    python examples/experts_layer.py [--type q4_k|q8_0|mxfp4|...] [--tokens N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_weight_out_gb300 import binding as rg  # noqa: E402
from quantized_weight_out_gb300 import build as rgbuild  # noqa: E402
from quantized_weight_out_gb300 import inputs  # noqa: E402

BF16, F32 = inputs.BF16, inputs.F32
SLOT, TOKEN = rg.RG_ROWS_SLOT, rg.RG_ROWS_TOKEN


class Layer:
    def __init__(self, wtype, vocab, hidden, inner, experts, top, rank=16, seed=0):
        self.wtype, self.vocab, self.hidden, self.inner = wtype, vocab, hidden, inner
        self.experts, self.top, self.rank, self.scale = experts, top, rank, 0.5
        self.dev = torch.device("cuda:0")

        def weight(t, rows, k, stream):
            return torch.from_numpy(inputs.gen_weight(t, rows, k, seed=seed, stream=stream)).to(self.dev)

        self.table = weight(inputs.Q6_K, vocab, hidden, 1)
        self.router = weight(inputs.F16, experts, hidden, 2)
        self.gate, self.up = (weight(wtype, experts * inner, hidden, s) for s in (3, 4))
        self.down = weight(wtype, experts * hidden, inner, 5)
        g = torch.Generator(device=self.dev).manual_seed(seed)
        # an adapter on the table: x += a[token] . b
        self.a = torch.randn(vocab, rank, generator=g, device=self.dev) * 0.1
        self.b = torch.randn(rank, hidden, generator=g, device=self.dev) * 0.1

    def forward(self, tokens, stream):
        """tokens: device int32 [T].  y [T, hidden] bf16, and what the way back needs."""
        T, H, I, E, k = len(tokens), self.hidden, self.inner, self.experts, self.top
        dev = self.dev
        x = torch.empty(T, H, device=dev)
        rg.check(rg.rg_get_rows(inputs.Q6_K, self.table, self.vocab, H, tokens, T, self.scale, F32, x, H, stream))
        low = torch.empty(T, self.rank, device=dev)
        rg.check(rg.rg_get_rows(F32, self.a, self.vocab, self.rank, tokens, T, 1.0, F32, low, self.rank, stream))
        x += low @ self.b
        logits = torch.empty(T, E, device=dev)
        rg.check(rg.rg_mul_mat(inputs.F16, self.router, E, H, x, T, logits, 0.0, stream))
        ids = torch.empty(T, k, dtype=torch.int32, device=dev)
        w = torch.empty(T, k, device=dev)
        start = torch.empty(E + 1, dtype=torch.int32, device=dev)
        order = torch.empty(T * k, dtype=torch.int32, device=dev)
        rg.check(rg.rg_route(logits, E, T, E, k, rg.RG_ROUTE_TOP, 1.0, ids, w, start, order, stream))
        batch = rg.id_batch(E, k, start, order)
        xb = x.to(torch.bfloat16)
        gate, up = (torch.empty(T * k, I, dtype=torch.bfloat16, device=dev) for _ in range(2))
        for weight, y in ((self.gate, gate), (self.up, up)):
            rg.check(rg.rg_mul_mat_id(self.wtype, weight, I, H, batch, BF16, xb, H, TOKEN, y, I, SLOT, None, 0.0, stream))
        h = (torch.nn.functional.silu(gate.float()) * up.float()).to(torch.bfloat16)
        y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        rg.check(rg.rg_mul_mat_id(self.wtype, self.down, H, I, batch, BF16, h, I, SLOT, y, H, TOKEN, w, 0.0, stream))
        return y, dict(tokens=tokens, x=x, logits=logits, ids=ids, w=w, start=start, order=order, batch=batch, gate=gate,
                       up=up, h=h)

    def backward(self, dy, s, stream):
        """dy [T, hidden] bf16.  (dx, the gradient of the adapter's a), from what forward kept."""
        T, H, I, E, k = len(dy), self.hidden, self.inner, self.experts, self.top
        dev = self.dev
        dh = torch.empty(T * k, I, dtype=torch.bfloat16, device=dev)
        rg.check(rg.rg_out_prod_id(self.wtype, self.down, H, I, s["batch"], BF16, dy, H, TOKEN, dh, I, SLOT, None, 0.0,
                                   stream))
        dh = dh.float()
        dw = (dh * s["h"].float()).sum(1).view(T, k).contiguous()
        dh = dh * s["w"].view(-1, 1)
        gate, up = s["gate"].float(), s["up"].float()
        sig = torch.sigmoid(gate)
        dgate, dup = (dh * up * sig * (1 + gate * (1 - sig))).to(torch.bfloat16), (dh * gate * sig).to(torch.bfloat16)
        dx = torch.empty(T, H, device=dev)
        rg.check(rg.rg_out_prod_id(self.wtype, self.gate, I, H, s["batch"], F32, dgate.float(), I, SLOT, dx, H, TOKEN, None,
                                   0.0, stream))
        rg.check(rg.rg_out_prod_id(self.wtype, self.up, I, H, s["batch"], F32, dup.float(), I, SLOT, dx, H, TOKEN, None,
                                   1.0, stream))
        dl = torch.empty(T, E, device=dev)
        rg.check(rg.rg_route_back(s["logits"], E, T, E, k, rg.RG_ROUTE_TOP, 1.0, s["ids"], dw, dl, E, stream))
        rg.check(rg.rg_out_prod(inputs.F16, self.router, E, H, dl, T, dx, 1.0, stream))
        da = torch.empty(self.vocab, self.rank, device=dev)
        low = dx @ self.b.T
        rg.check(rg.rg_get_rows_back(F32, low, self.rank, s["tokens"], T, 1.0, da, self.rank, self.vocab, self.rank, 0.0,
                                     stream))
        return dx, da

    def plain(self, tokens, ids, dy):
        """The layer in 64 bits with the same choices: y, dx, da, by autograd."""
        def dense(t, w, n, k):
            out = torch.empty(n, k, device=self.dev)
            rg.check(rg.rg_dequant_async(t, w, n, k, out, torch.cuda.current_stream()), "rg_dequant")
            return out.double()
        H, I, E, k = self.hidden, self.inner, self.experts, self.top
        a = self.a.double().requires_grad_()
        x = dense(inputs.Q6_K, self.table, self.vocab, H)[tokens.long()] * self.scale + a[tokens.long()] @ self.b.double()
        x.retain_grad()
        logits = x @ dense(inputs.F16, self.router, E, H).T
        w = torch.softmax(logits.gather(1, ids.long()), -1).view(-1)
        gate, up = (dense(self.wtype, v, E * I, H).view(E, I, H) for v in (self.gate, self.up))
        down = dense(self.wtype, self.down, E * H, I).view(E, H, I)
        flat = ids.long().view(-1)
        rows = torch.zeros(len(flat), H, dtype=torch.float64, device=self.dev)
        for e in range(E):
            at = torch.nonzero(flat == e).view(-1)
            v = x[at // k]
            rows = rows.index_add(0, at, (torch.nn.functional.silu(v @ gate[e].T) * (v @ up[e].T)) @ down[e].T)
        y = (rows * w[:, None]).view(-1, k, H).sum(1)
        y.backward(dy.double())
        return y.detach(), x.grad, a.grad


def run(wtype=inputs.Q4_K, tokens=300, vocab=1000, hidden=2048, inner=768, experts=16, top=3, seed=0, verbose=True):
    """A training step and replayed decoding steps; the largest relative errors (2-norm) of y, dx, da and a decoded y."""
    rgbuild.build()
    L = Layer(wtype, vocab, hidden, inner, experts, top, seed=seed)
    g = torch.Generator(device=L.dev).manual_seed(seed + 1)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device=L.dev).to(torch.int32)
    stream = torch.cuda.current_stream()
    y, s = L.forward(ids, stream)
    dy = (torch.randn(tokens, hidden, generator=g, device=L.dev) * 1e-3).to(torch.bfloat16)
    dx, da = L.backward(dy, s, stream)
    rg.check(rg.rg_check(stream), "rg_check")
    far = [float((got.double() - ref).norm() / ref.norm()) for got, ref in zip((y, dx, da), L.plain(ids, s["ids"], dy))]
    # decoding: one captured step of two tokens, replayed with other tokens
    step = ids[:2].clone()
    side = torch.cuda.Stream()
    side.wait_stream(stream)
    with torch.cuda.stream(side):
        L.forward(step, side)
    stream.wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, kept = L.forward(step, torch.cuda.current_stream())
    worst = 0.0
    for i in range(0, 8, 2):
        step.copy_(ids[i:i + 2])
        graph.replay()
        ref = L.plain(step, kept["ids"], dy[:2])[0]
        worst = max(worst, float((out.double() - ref).norm() / ref.norm()))
    rg.check(rg.rg_check(torch.cuda.current_stream()), "rg_check")
    if verbose:
        print(f"{inputs.TYPE_NAMES[wtype]} experts, {tokens} tokens: relative errors of y {far[0]:.2e}, dx {far[1]:.2e}, "
              f"the adapter's gradient {far[2]:.2e}; of decoded tokens {worst:.2e}")
    return (*far, worst)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--type", default="q4_k", choices=sorted(inputs.NAME_TO_TYPE))
    ap.add_argument("--tokens", type=int, default=300)
    a = ap.parse_args()
    run(inputs.NAME_TO_TYPE[a.type], tokens=a.tokens)
