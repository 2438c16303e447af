"""Indexed work on resident weights, as it is measured: rows of a table by token, experts' products by slot, and the
router that says which expert a slot goes to.

Five operators (include/rg.h): ``rg_get_rows`` looks rows of a resident table up and scales them, ``rg_get_rows_back``
adds a gradient's rows to the rows of a trained table by token; ``rg_route`` picks each token's experts and sorts the
slots by expert, ``rg_route_back`` is its gradient; ``rg_mul_mat_id`` and ``rg_out_prod_id`` are the forward and the
activation gradient through the experts' resident weights, each expert with the slots that were sorted to it.

``run`` computes a case with elementary torch operations in 32 bits, or, with ``own`` set, through the library.  A
token has ``k`` slots, slot ``s`` belongs to token ``s // k``; ``order`` lists the slots sorted by expert, expert ``e``'s
at ``start[e] .. start[e + 1] - 1``, those of no expert (padding) behind them.
"""
import math
import random

import torch

own = False

ACT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"f16": 1, "bf16": 2, "q8_0": 3, "q4_k": 5, "q6_k": 10, "f32": 11, "mxfp4": 14}  # rg_wtype
BLOCK = {"f16": (1, 2), "bf16": (1, 2), "q8_0": (32, 34), "q4_k": (256, 144), "q6_k": (256, 210), "mxfp4": (32, 17)}
SLOT, TOKEN = 0, 1    # whose rows an array of a product holds
TOP, ALL = 0, 1       # softmax over the chosen experts, or over all


# ---------------------------------------------------------------------------
# the cases

def _case(name, op, **kw):
    base = {"rows": dict(type="q4_k", act="bf16", vocab=32000, k=4096, n=1, scale=1.0, pad=0.0),
            "rows_back": dict(act="bf16", vocab=32000, k=4096, n=1, scale=1.0, pad=0.0),
            "route": dict(tokens=1, experts=8, top=2, mode=TOP, back=False),
            "mul": dict(type="q4_k", act="bf16", tokens=1, experts=8, top=2, n=14336, k=4096, into=TOKEN, out=SLOT,
                        weigh=False, pad=0.0),
            "out_prod": dict(type="q4_k", act="bf16", tokens=1, experts=8, top=2, n=14336, k=4096, into=SLOT,
                             out=TOKEN, weigh=False, pad=0.0)}[op]
    return dict(name=name, op=op, **{**base, **kw})


def listed():
    return [
        # one decoding step of seven users: their tokens' rows of the table
        _case("rows 7 q4_k", "rows", n=7),
        # a packed batch of prompts through a large vocabulary, scaled by sqrt(k) as some models do, padding among it
        _case("rows 8191 q6_k", "rows", type="q6_k", vocab=128256, n=8191, scale=64.0, pad=0.02),
        # an adapter on the table (rows as long as its rank) trained on one short sequence
        _case("rows back 509 rank 64", "rows_back", k=64, n=509, scale=2.0),
        # a trained table's gradient from a batch of sequences; a few tokens make up most of them
        _case("rows back 16381", "rows_back", n=16381, pad=0.02),
        # one decoding token's choice among few experts
        _case("route 1 of 8", "route"),
        # a training batch's choice among many, and what flows back through the weights
        _case("route 8192 of 128 back", "route", tokens=8192, experts=128, top=8, mode=ALL, back=True),
        # a decoding token's projection into two large experts: latency counts
        _case("mul 1 q4_k 2of8", "mul"),
        # a decoding batch of many users into small experts, back to the model's width and summed by the
        # router's weights: few slots an expert, every expert read
        _case("mul 40 q8_0 8of64 down", "mul", type="q8_0", tokens=40, experts=64, top=8, n=2048, k=1024, into=SLOT,
              out=TOKEN, weigh=True),
        # a prompt through small four-bit experts, some very popular, padding among the tokens
        _case("mul 4096 mxfp4 8of128", "mul", type="mxfp4", tokens=4096, experts=128, top=8, n=768, k=2048, pad=0.03),
        # a prompt through large experts
        _case("mul 4093 q4_k 2of8", "mul", tokens=4093),
        # a training batch's gradient through small 16-bit experts, a row for each slot
        _case("out_prod 2039 bf16 8of64", "out_prod", type="bf16", tokens=2039, experts=64, top=8, n=1024, k=2048,
              into=TOKEN, out=SLOT),
        # a training batch's gradient through large experts, summed by token
        _case("out_prod 4093 q4_k 2of8", "out_prod", tokens=4093),
    ]


def _cost(c):
    w = work(c)
    plain = 0.0  # what the plain form holds at once: decoded weights, the padded groups
    if c["op"] in ("mul", "out_prod"):
        m = 2.5 * c["tokens"] * c["top"] / c["experts"] + 4
        plain = 4.0 * c["experts"] * (c["n"] * c["k"] + m * (c["n"] + c["k"]))
    return w["bytes"], w["flops"], plain


def draw(rng):
    """One more case: the listed ones' ranges, sizes spread over their logarithm."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    top = [_cost(c) for c in listed()]
    top = tuple(max(t[i] for t in top) for i in range(3))
    while True:
        op = rng.choice(["rows", "rows_back", "route", "mul", "mul", "mul", "out_prod", "out_prod"])
        pad = rng.choice([0.0, 0.0, 0.01, 0.1])
        if op == "rows":
            kind = rng.choice(["q4_k", "q6_k", "q8_0", "mxfp4", "bf16", "f16"])
            c = _case("", op, type=kind, act=rng.choice(["bf16", "bf16", "f16", "f32"]), vocab=log(1000, 128256),
                      k=256 * log(2, 16), n=log(7, 8191), scale=rng.choice([1.0, 0.125, 64.0]), pad=pad)
        elif op == "rows_back":
            c = _case("", op, act=rng.choice(["bf16", "bf16", "f16", "f32"]), vocab=log(1000, 32000),
                      k=8 * log(2, 512), n=log(100, 16381), scale=rng.choice([1.0, 2.0, 0.125]), pad=pad)
        elif op == "route":
            experts = rng.choice([4, 8, 16, 32, 60, 64, 128, 160, 256])
            c = _case("", op, tokens=log(1, 8192), experts=experts, top=rng.randint(1, min(8, experts)),
                      mode=rng.choice([TOP, ALL]), back=rng.random() < 0.5)
        else:
            kind = rng.choice(["q4_k", "q4_k", "q8_0", "mxfp4", "bf16", "f16"])
            experts = rng.choice([4, 8, 16, 32, 60, 64, 128])
            # f16 activations where the weights' operands are exact
            act = {"bf16": "bf16", "f16": "f16"}.get(kind, "bf16")
            tokens = log(1, 4093) if op == "mul" else log(100, 4093)
            c = _case("", op, type=kind, act=act, tokens=tokens, experts=experts, top=rng.randint(1, min(8, experts)),
                      n=8 * log(64, 1792), k=256 * log(2, 16) if kind != "mxfp4" else 512 * log(1, 8),
                      into=rng.choice([SLOT, TOKEN]), out=rng.choice([SLOT, TOKEN]), weigh=rng.random() < 0.5, pad=pad)
        del c["name"]
        cost = _cost(c)
        if all(x <= t for x, t in zip(cost, top)):
            return c


def _row_bytes(kind, k):
    v, b = BLOCK[kind]
    return k // v * b


def work(case):
    c = case
    if c["op"] == "rows":
        size = 4 if c["act"] == "f32" else 2
        return {"bytes": c["n"] * (_row_bytes(c["type"], c["k"]) + c["k"] * size + 4), "flops": 2 * c["n"] * c["k"]}
    if c["op"] == "rows_back":
        size = 4 if c["act"] == "f32" else 2
        return {"bytes": c["n"] * (c["k"] * size + 4) + c["vocab"] * c["k"] * 4, "flops": 2 * c["n"] * c["k"]}
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top"]
        passes = 1 + 2 * c["back"]                                   # logits, dlogits (and logits again)
        return {"bytes": 4 * (t * e * passes + t * k * (3 + 2 * c["back"]) + e), "flops": (4 + 4 * c["back"]) * t * e}
    slots = c["tokens"] * c["top"]
    wide, out = (c["k"], c["n"]) if c["op"] == "mul" else (c["n"], c["k"])
    rows = {SLOT: slots, TOKEN: c["tokens"]}
    return {"bytes": min(c["experts"], slots) * c["n"] * _row_bytes(c["type"], c["k"])
            + 2 * (rows[c["into"]] * wide + rows[c["out"]] * out) + 4 * (slots * (1 + c["weigh"]) + c["experts"]),
            "flops": 2 * slots * c["n"] * c["k"]}


# ---------------------------------------------------------------------------
# inputs

def _weights(kind, rows, k, g):
    """`rows` stored rows of k values of a type: uint8 [rows, bytes], values of about 1 / sqrt(k)."""
    dev, s = "cuda", 1 / math.sqrt(k)
    if kind in ("f16", "bf16"):
        w = torch.empty(rows, k, dtype=ACT[kind], device=dev)
        step = max(1, (1 << 26) // k)
        for i in range(0, rows, step):
            w[i:i + step] = (torch.randn(min(step, rows - i), k, generator=g, device=dev) * s).to(ACT[kind])
        return w.view(torch.uint8)
    v, b = BLOCK[kind]
    n = rows * (k // v)
    x = torch.randint(0, 256, (n, b), generator=g, dtype=torch.uint8, device=dev)
    d = (0.5 + torch.rand(n, 1, generator=g, device=dev)) * s

    def half(t):
        return t.to(torch.float16).view(torch.uint8)

    if kind == "q8_0":
        x[:, 2:] = (torch.randn(n, 32, generator=g, device=dev) * 40).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        x[:, :2] = half(d / 40)
    elif kind == "q4_k":
        # eight sub-blocks' scale and minimum alike, so that the values lie around zero
        x[:, 4:8] = x[:, 4:8] & 0x3F | 0x10
        x[:, 8:12] = x[:, 4:8]
        x[:, 12:16] = (x[:, 12:16] & 15) * 17
        x[:, :2] = half(d / 150)
        x[:, 2:4] = half(7.5 * d / 150)
    elif kind == "q6_k":
        x[:, 192:208] = torch.randint(-100, 100, (n, 16), generator=g, device=dev).to(torch.int8).view(torch.uint8)
        x[:, 208:] = half(d / 1000)
    else:
        x[:, :1] = (126 + torch.log2(d / 2)).round().to(torch.uint8)
    return x.view(rows, -1)


def _tokens(c, g):
    """Token numbers of a text: the lower, the more frequent; -1 where a batch is padded."""
    u = torch.rand(c["n"], generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(c["vocab"])) - 1).long().clamp(0, c["vocab"] - 1)
    return torch.where(torch.rand(c["n"], generator=g, device="cuda") < c["pad"], -1, ids).to(torch.int32)


def _sorted_slots(ids, experts):
    """order and start of slots' experts (below 0: none)."""
    key = torch.where(ids < 0, experts, ids.long())
    order = torch.sort(key, stable=True).indices
    start = torch.searchsorted(key[order].contiguous(), torch.arange(experts + 1, device=ids.device))
    return order.to(torch.int32), start.to(torch.int32)


def prepare(case, seed):
    """The weights, the call's inputs, and the buffers that a program keeps for its results."""
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    if c["op"] == "rows":
        act = ACT[c["act"]]
        return dict(case=c, w=_weights(c["type"], c["vocab"], c["k"], g), ids=_tokens(c, g),
                    out=torch.zeros(c["n"], c["k"], dtype=act, device=dev))
    if c["op"] == "rows_back":
        dy = torch.randn(c["n"], c["k"], generator=g, device=dev) * 1e-3
        return dict(case=c, dy=dy.to(ACT[c["act"]]), ids=_tokens(c, g),
                    grad=torch.zeros(c["vocab"], c["k"], device=dev))
    t, e, k = c["tokens"], c["experts"], c["top"]
    # a token's logits: some experts are popular
    logits = torch.randn(t, e, generator=g, device=dev) * 1.5 + torch.randn(e, generator=g, device=dev) * 0.7
    if c["op"] == "route":
        return dict(case=c, logits=logits, dweights=torch.randn(t, k, generator=g, device=dev) * 1e-2,
                    ids=torch.zeros(t, k, dtype=torch.int32, device=dev), weights=torch.zeros(t, k, device=dev),
                    start=torch.zeros(e + 1, dtype=torch.int32, device=dev),
                    order=torch.zeros(t * k, dtype=torch.int32, device=dev), dlogits=torch.zeros(t, e, device=dev))
    best = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids, weights = best.indices[:, :k], torch.softmax(best.values[:, :k], -1)
    ids = torch.where(torch.rand(t, 1, generator=g, device=dev) < c["pad"], -1, ids).reshape(-1)
    order, start = _sorted_slots(ids, e)
    wide, out = (c["k"], c["n"]) if c["op"] == "mul" else (c["n"], c["k"])
    rows = {SLOT: t * k, TOKEN: t}
    # activations with a few strong channels; gradients are small
    x = torch.randn(rows[c["into"]], wide, generator=g, device=dev)
    x *= 1 + 4 * (torch.rand(wide, generator=g, device=dev) < 0.01).float() if c["op"] == "mul" else 1e-3
    # the experts in use, and where each sorted slot's row goes in their groups, padded to the longest
    count = start.diff()
    used, longest = torch.nonzero(count > 0).view(-1), max(1, int(count.max()))
    live = order.long()[:int(start[-1])]
    expert = ids[live].long()
    place = torch.searchsorted(used, expert) * longest + torch.arange(len(live), device=dev) - start.long()[expert]
    return dict(case=c, w=_weights(c["type"], e * c["n"], c["k"], g), x=x.to(ACT[c["act"]]), ids=ids, order=order,
                start=start, weights=weights.reshape(-1).contiguous() if c["weigh"] else None, longest=longest, live=live,
                used=used, place=place, out=torch.zeros(rows[c["out"]], out, dtype=ACT[c["act"]], device=dev))


# ---------------------------------------------------------------------------
# the plain form

def _f16(x):
    return x.contiguous().view(torch.float16).float()


def _values(kind, w):
    """The 32-bit values [rows, k] of stored rows [rows, bytes]."""
    if kind in ("f16", "bf16"):
        return w.view(ACT[kind]).float()
    v, b = BLOCK[kind]
    x = w.unflatten(-1, (-1, b))
    if kind == "q8_0":
        y = _f16(x[..., :2]) * x[..., 2:].view(torch.int8).float()
    elif kind == "mxfp4":
        q = torch.cat((x[..., 1:] & 15, x[..., 1:] >> 4), -1).int()
        m = (q & 7).float()
        size = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
        y = torch.where(q > 7, -size, size) * torch.exp2(x[..., :1].float() - 127)
    elif kind == "q4_k":
        s = x[..., 4:16].int()
        a, m, z = s[..., :4], s[..., 4:8], s[..., 8:]
        scale = torch.cat((a & 63, (z & 15) | ((a >> 6) << 4)), -1).float()
        least = torch.cat((m & 63, (z >> 4) | ((m >> 6) << 4)), -1).float()
        q = x[..., 16:].unflatten(-1, (4, 32))
        q = torch.stack((q & 15, q >> 4), -2).flatten(-3, -2).float()
        y = q * (_f16(x[..., :2]) * scale)[..., None] - (_f16(x[..., 2:4]) * least)[..., None]
        y = y.flatten(-2)
    else:
        low = x[..., :128].unflatten(-1, (2, 2, 32)).int()
        low = torch.cat((low & 15, low >> 4), -2)                                       # half, quarter, value
        high = x[..., 128:192].unflatten(-1, (2, 1, 32)).int()
        high = torch.cat((high & 3, high >> 2 & 3, high >> 4 & 3, high >> 6), -2)
        scale = _f16(x[..., 208:]) * x[..., 192:208].view(torch.int8).float()
        y = (low + 16 * high - 32).flatten(-3).unflatten(-1, (16, 16)).float() * scale[..., None]
        y = y.flatten(-2)
    return y.flatten(-2)


def _plain_rows(s):
    c = s["case"]
    ids = s["ids"].long()
    x = _values(c["type"], s["w"][ids.clamp(min=0)]) * c["scale"]
    return torch.where(ids[:, None] < 0, 0, x).to(ACT[c["act"]])


def _plain_rows_back(s):
    c = s["case"]
    ids = s["ids"].long()
    x = torch.where(ids[:, None] < 0, 0, s["dy"].float())
    grad = torch.zeros(c["vocab"], c["k"], device=x.device)
    return grad.index_add_(0, ids.clamp(min=0), x * c["scale"])


def _plain_route(s):
    c = s["case"]
    logits, k = s["logits"], c["top"]
    best = torch.sort(logits, dim=-1, descending=True, stable=True)  # of equals the lowest number first
    ids, top = best.indices[:, :k], best.values[:, :k]
    part = torch.exp(top - top[:, :1])
    whole = torch.exp(logits - top[:, :1])
    total = (part if c["mode"] == TOP else whole).sum(-1, keepdim=True)
    weights = part / total
    order, start = _sorted_slots(ids.reshape(-1), c["experts"])
    got = {"ids": ids.to(torch.int32), "weights": weights, "start": start, "order": order}
    if c["back"]:
        dw = s["dweights"]
        mean = (weights * dw).sum(-1, keepdim=True)
        if c["mode"] == TOP:
            got["dlogits"] = torch.zeros_like(logits).scatter_(1, ids, weights * (dw - mean))
        else:
            p = whole / total
            got["dlogits"] = (-p * mean).scatter_add_(1, ids, weights * dw)
    return got


def _plain_product(s):
    c = s["case"]
    k, e = c["top"], len(s["used"])
    stored = s["w"].view(c["experts"], c["n"], -1)
    w = _values(c["type"], (stored if e == c["experts"] else stored[s["used"]]).flatten(0, 1)).view(e, c["n"], c["k"])
    live = s["live"]
    x = s["x"].float()[live // k if c["into"] == TOKEN else live]
    groups = x.new_zeros(e * s["longest"], x.shape[1])
    groups[s["place"]] = x
    groups = groups.view(e, s["longest"], -1)
    y = torch.bmm(groups, w.transpose(1, 2) if c["op"] == "mul" else w).flatten(0, 1)[s["place"]]
    rows = y.new_zeros(c["tokens"] * k, y.shape[1])
    rows[live] = y if s["weights"] is None else y * s["weights"][live, None]
    if c["out"] == TOKEN:
        rows = rows.view(c["tokens"], k, -1).sum(1)
    return rows.to(ACT[c["act"]])


# ---------------------------------------------------------------------------
# the library

def _handles(s):
    """The batch's description, which a user's program keeps."""
    if "rg" not in s:
        from quantized_weight_out_gb300 import binding as rg
        c = s["case"]
        s["rg"] = rg
        if c["op"] in ("mul", "out_prod"):
            s["batch"] = rg.id_batch(c["experts"], c["top"], s["start"], s["order"])
    return s["rg"], torch.cuda.current_stream()


def _own(s):
    rg, stream = _handles(s)
    c = s["case"]
    if c["op"] == "rows":
        rg.check(rg.rg_get_rows(CODE[c["type"]], s["w"], c["vocab"], c["k"], s["ids"], c["n"], c["scale"],
                                CODE[c["act"]], s["out"], c["k"], stream), "rg_get_rows")
        return s["out"]
    if c["op"] == "rows_back":
        rg.check(rg.rg_get_rows_back(CODE[c["act"]], s["dy"], c["k"], s["ids"], c["n"], c["scale"], s["grad"], c["k"],
                                     c["vocab"], c["k"], 0.0, stream), "rg_get_rows_back")
        return s["grad"]
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top"]
        rg.check(rg.rg_route(s["logits"], e, t, e, k, c["mode"], 1.0, s["ids"], s["weights"], s["start"], s["order"],
                             stream), "rg_route")
        got = {n: s[n] for n in ("ids", "weights", "start", "order")}
        if c["back"]:
            rg.check(rg.rg_route_back(s["logits"], e, t, e, k, c["mode"], 1.0, s["ids"], s["dweights"], s["dlogits"],
                                      e, stream), "rg_route_back")
            got["dlogits"] = s["dlogits"]
        return got
    wide, out = (c["k"], c["n"]) if c["op"] == "mul" else (c["n"], c["k"])
    call = rg.rg_mul_mat_id if c["op"] == "mul" else rg.rg_out_prod_id
    rg.check(call(CODE[c["type"]], s["w"], c["n"], c["k"], s["batch"], CODE[c["act"]], s["x"], wide, c["into"],
                  s["out"], out, c["out"], s["weights"], 0.0, stream), "rg_%s_id" % c["op"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"rows": _plain_rows, "rows_back": _plain_rows_back, "route": _plain_route, "mul": _plain_product,
            "out_prod": _plain_product}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions

def _fields(kind):
    """Of each value of a block: the byte that holds its code (or the low part), how far up, and the type's others."""
    v = torch.arange(BLOCK[kind][0], device="cuda")
    if kind == "q4_k":
        return 16 + 32 * (v // 64) + v % 32, 4 * (v // 32 % 2), v // 32
    if kind == "q6_k":
        h, i, at = v // 128, v // 32 % 4, v % 32
        return 64 * h + 32 * (i % 2) + at, 4 * (i // 2), 128 + 32 * h + at, 2 * i, 192 + v // 16
    return 1 + v % 16, 4 * (v // 16)


def _number16(x, at):
    """The fp16 number at byte `at` of blocks, from its bits."""
    u = x[..., at].long() + 256 * x[..., at + 1].long()
    e, m = (u >> 10) & 31, (u & 1023).double()
    size = torch.where(e == 0, m * 2.0 ** -24, (1024 + m) * torch.exp2(e.double() - 25))
    return torch.where(u >= 32768, -size, size)[..., None]


def _exact_values(kind, w):
    """Stored rows in 64 bits, each value's code found by its place."""
    if kind in ("f16", "bf16"):
        return w.view(ACT[kind]).double()
    x = w.reshape(w.shape[0], -1, BLOCK[kind][1])
    if kind == "q8_0":
        y = x[..., 2:].double()
        y = torch.where(y > 127, y - 256, y) * _number16(x, 0)
    elif kind == "mxfp4":
        at, up = _fields(kind)
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=w.device)
        y = table[((x[..., at] >> up.to(torch.uint8)) & 15).long()] * torch.exp2(x[..., :1].double() - 127)
    elif kind == "q4_k":
        at, up, j = _fields(kind)
        q = ((x[..., at] >> up.to(torch.uint8)) & 15).double()
        b = x.long()
        late = j >= 4
        lo, hi, mix = b[..., 4 + j % 4], b[..., 8 + j % 4], b[..., 12 + j % 4]
        scale = torch.where(late, mix % 16 + lo // 64 * 16, lo % 64)
        least = torch.where(late, mix // 16 + hi // 64 * 16, hi % 64)
        y = _number16(x, 0) * scale * q - _number16(x, 2) * least
    else:
        at, up, at2, up2, sc = _fields(kind)
        q = ((x[..., at] >> up.to(torch.uint8)) & 15).double() + 16 * ((x[..., at2] >> up2.to(torch.uint8)) & 3).double()
        scale = x[..., sc].double()
        y = _number16(x, 208) * torch.where(scale > 127, scale - 256, scale) * (q - 32)
    return y.reshape(w.shape[0], -1)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rows":
        got = torch.zeros(c["n"], c["k"], dtype=torch.float64, device="cuda")
        real = s["ids"] >= 0
        got[real] = _exact_values(c["type"], s["w"][s["ids"][real].long()]) * c["scale"]
        return got
    if c["op"] == "rows_back":
        got = torch.zeros(c["vocab"], c["k"], dtype=torch.float64, device="cuda")
        real = s["ids"] >= 0
        got.index_put_((s["ids"][real].long(),), s["dy"][real].double() * c["scale"], accumulate=True)
        return got
    if c["op"] == "route":
        logits, k = s["logits"].double(), c["top"]
        chosen = torch.zeros_like(logits, dtype=torch.bool)
        ids = torch.empty(c["tokens"], k, dtype=torch.long, device="cuda")
        for j in range(k):
            left = logits.masked_fill(chosen, -math.inf)
            lane = torch.arange(c["experts"], device="cuda")
            ids[:, j] = torch.where(left == left.max(-1, keepdim=True).values, lane, c["experts"]).min(-1).values
            chosen.scatter_(1, ids[:, j:j + 1], True)
        p = torch.softmax(logits if c["mode"] == ALL else logits.masked_fill(~chosen, -math.inf), -1)
        got = {"ids": None, "weights": p.gather(1, ids), "start": None, "order": None}
        if c["back"]:
            up = torch.zeros_like(p).scatter_(1, ids, s["dweights"].double())
            got["dlogits"] = p * (up - (p * up).sum(-1, keepdim=True))
        return got
    t, k = c["tokens"], c["top"]
    x = s["x"].double()
    if c["into"] == TOKEN:
        x = x.repeat_interleave(k, 0)
    got = torch.zeros(t * k, c["n"] if c["op"] == "mul" else c["k"], dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        at = torch.nonzero(s["ids"] == e).view(-1)
        if len(at):
            w = _exact_values(c["type"], s["w"][e * c["n"]:(e + 1) * c["n"]])
            got[at] = x[at] @ (w.T if c["op"] == "mul" else w)
    if s["weights"] is not None:
        got *= s["weights"].double()[:, None]
    return got.view(t, k, -1).sum(1) if c["out"] == TOKEN else got
