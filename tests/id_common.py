"""A stack of experts, its slots and activations for the tests, on both sides."""
import numpy as np

import oracle
from kv_common import to_act
from quantized_weight_out_gb300 import inputs

F32, F16, BF16 = inputs.F32, inputs.F16, inputs.BF16
SLOT, TOKEN = 0, 1
HALF_STEP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
SMALLEST = {F32: 0.0, F16: 2.0 ** -25, BF16: 0.0}  # half of the smallest step of a type's small values


def torch_act(torch, atype):
    return {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}[atype]


def weight_error(wtype, K):
    """How far a decoded operand may be from the weight, relative to the weight: half a step for each rounding of a
    product to fp16 (the scale's own, then the value's); the types with a minimum lose more where scale * q and the
    minimum cancel, and have the bound that the header gives for them all."""
    if wtype in (inputs.F16, inputs.BF16, inputs.NVFP4, inputs.MXFP4, inputs.F32):
        return 0.0
    if wtype in (inputs.Q8_0, inputs.Q4_0, inputs.Q5_0):
        return 2.0 ** -11
    if wtype in (inputs.Q6_K, inputs.Q3_K):
        return 2 * 2.0 ** -11
    return 4e-3


def product_tolerance(wtype, K, wide, atype, mag, ref, beta=0.0, old=0.0):
    """The error that a product's result may have: the input row's rounding to the operands' kind (nothing where the
    activations' type is within it; fp16 copies keep 11 bits down to 2^-28 of a row's largest value), the weights',
    the F32 sums' (one half step a term, twice for the tensor cores' truncated additions) and the result's own."""
    kind = BF16 if wtype == BF16 else F16
    simt = wtype == F32
    into = 0.0 if simt or atype == kind or (kind == F16 and atype == BF16) else HALF_STEP[kind]
    each = into + (0.0 if simt else weight_error(wtype, K)) + 2 * (wide + 8) * 2.0 ** -24
    return each * mag * 1.01 + HALF_STEP[atype] * (np.abs(ref) + each * mag + np.abs(beta * old)) * 1.01 + \
        SMALLEST[atype] + 1e-30


class Stack:
    def __init__(self, torch, rg, wtype, experts, N, K, ids, per_token, seed=0, W=None):
        self.torch, self.rg, self.dev = torch, rg, torch.device("cuda:0")
        self.wtype, self.experts, self.N, self.K, self.per_token = wtype, experts, N, K, per_token
        self.ids = np.asarray(ids, np.int32).reshape(-1)
        self.slots, self.tokens = len(self.ids), len(self.ids) // per_token
        self.rng = np.random.default_rng(seed)
        self.W = inputs.gen_weight(wtype, experts * N, K, seed=seed, stream=1) if W is None else W
        self.W_d = torch.from_numpy(np.ascontiguousarray(self.W).view(np.uint8).reshape(-1)).to(self.dev)
        self.start, self.order = oracle.group(self.ids, experts)
        self.start_d, self.order_d = (torch.from_numpy(x).to(self.dev) for x in (self.start, self.order))
        self.batch = rg.id_batch(experts, per_token, self.start_d, self.order_d)

    def act(self, rows, width, atype, scale=1.0):
        return to_act((self.rng.standard_normal((rows, width)) * scale).astype(np.float32), atype)

    def put(self, x, atype, pad=0, fill=7.0):
        """x in device memory, rows `pad` values longer."""
        t = self.torch
        d = t.full((x.shape[0], x.shape[1] + pad), fill, dtype=torch_act(t, atype), device=self.dev)
        d[:, :x.shape[1]] = t.from_numpy(x.astype(np.float32)).to(self.dev).to(torch_act(t, atype))
        return d

    def run(self, fwd, atype, x, x_of, out_of, weights=None, beta=0.0, old=None, pad=0, stream=None, ws=False):
        """The result [rows, width] and its padding, after the call's status and the device's were checked."""
        t, rg = self.torch, self.rg
        wide, width = (self.K, self.N) if fwd else (self.N, self.K)
        x_d = self.put(x, atype, pad)
        rows = self.tokens if out_of == TOKEN else self.slots
        out = self.put(np.full((rows, width), np.nan) if old is None else old, atype, pad)
        w_d = None if weights is None else t.from_numpy(weights.astype(np.float32)).to(self.dev)
        args = (self.wtype, self.W_d, self.N, self.K, self.batch, atype, x_d, wide + pad, x_of, out, width + pad, out_of,
                w_d, beta)
        s = stream or t.cuda.current_stream()
        s.wait_stream(t.cuda.current_stream())
        if ws:
            size = (rg.rg_mul_mat_id_workspace_bytes if fwd else rg.rg_out_prod_id_workspace_bytes)(
                self.wtype, self.N, self.K, self.batch, out_of)
            work = t.full((size + 256,), 0xFF, dtype=t.uint8, device=self.dev)
            st = (rg.rg_mul_mat_id_ws if fwd else rg.rg_out_prod_id_ws)(*args, work, size, s)
            rg.check(st)
            assert rg.rg_check(s) == 0
            assert bool((work[size:] == 0xFF).all())
        else:
            rg.check((rg.rg_mul_mat_id if fwd else rg.rg_out_prod_id)(*args, s))
            assert rg.rg_check(s) == 0
        got = out.float().cpu().numpy()
        if pad:
            assert (got[:, width:] == 7.0).all()
        return got[:, :width]

    def check(self, fwd, atype, x_of, out_of, weigh=False, beta=0.0, pad=0, scale=1.0, ws=False, x=None):
        wide, width = (self.K, self.N) if fwd else (self.N, self.K)
        if x is None:
            x = self.act(self.tokens if x_of == TOKEN else self.slots, wide, atype, scale)
        weights = self.rng.random(self.slots).astype(np.float32) if weigh else None
        rows = self.tokens if out_of == TOKEN else self.slots
        old = self.act(rows, width, atype, scale) if beta else None
        got = self.run(fwd, atype, x, x_of, out_of, weights, beta, old, pad, ws=ws)
        ref, mag = oracle.product_id(fwd, self.wtype, self.W, self.experts, self.N, self.K, self.ids, self.per_token, x,
                                     x_of == TOKEN, weights)
        live = (self.ids >= 0) & (self.ids < self.experts)
        if out_of == TOKEN:
            ref, mag = (a.reshape(rows, self.per_token, width).sum(1) for a in (ref, mag))
            live = np.ones(rows, bool)
        else:
            left = got[~live]
            assert np.isnan(left).all() if old is None else np.array_equal(left, old[~live])
        o = 0.0 if old is None else old[live].astype(np.float64)
        ref = ref[live] + beta * o
        tol = product_tolerance(self.wtype, self.K, wide, atype, mag[live], ref, beta, o)
        err = np.abs(got[live] - ref)
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
