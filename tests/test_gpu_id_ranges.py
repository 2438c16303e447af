"""Experts' products whose ranges of slots are not a partition of the sorted order, on a GB300: sums over tokens and
rows by slot take in the slots of accepted ranges, and nothing that no kernel wrote."""
import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from id_common import BF16, F32, SLOT, TOKEN, Stack, product_tolerance  # noqa: E402

E, TOP = 4, 2


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


# the streaming form, tiles of one CTA and of pairs; a copy of W's rows; plain threads
ROUTES = [(inputs.Q8_0, 5, 512), (inputs.Q8_0, 60, 512), (inputs.Q8_0, 301, 512), (inputs.Q6_K, 6, 768),
          (F32, 40, 64)]


def _stack(rg, wtype, tokens, K):
    rng = np.random.default_rng(tokens)
    ids = np.stack([rng.permutation(E)[:TOP] for _ in range(tokens)])
    ids[::7, 1] = -1
    return Stack(torch, rg, wtype, E, 72, K, ids.reshape(-1), TOP, seed=tokens)


def _check(rg, s, fwd, x_of, out_of, start, status, first=0, weigh=False, beta=0.0):
    """The product with `start` in place of the stack's own, over a workspace of 0xFF, against the definition with the
    slots of accepted ranges only.  first: experts from this one on alone, their part of W and of start."""
    experts = s.experts - first
    start = np.asarray(start, np.int64)[first:]
    ids = np.full(s.slots, -1, np.int64)
    for e in range(experts):
        lo, hi = start[e], start[e + 1]
        if 0 <= lo <= hi <= s.slots:
            ids[s.order[lo:hi]] = e
    W = s.W.reshape(s.experts, -1)[first:]
    W_d = torch.from_numpy(np.ascontiguousarray(W).view(np.uint8).reshape(-1)).cuda()
    start_d = torch.from_numpy(start.astype(np.int32)).cuda()
    batch = rg.id_batch(experts, s.per_token, start_d, s.order_d)
    wide, width = (s.K, s.N) if fwd else (s.N, s.K)
    x = s.act(s.tokens if x_of == TOKEN else s.slots, wide, BF16)
    weights = s.rng.random(s.slots).astype(np.float32) if weigh else None
    rows = s.tokens if out_of == TOKEN else s.slots
    old = s.act(rows, width, BF16)
    x_d, out = s.put(x, BF16), s.put(old, BF16)
    w_d = torch.from_numpy(weights).cuda() if weigh else None
    query, call = ((rg.rg_mul_mat_id_workspace_bytes, rg.rg_mul_mat_id_ws) if fwd else
                   (rg.rg_out_prod_id_workspace_bytes, rg.rg_out_prod_id_ws))
    size = query(s.wtype, s.N, s.K, batch, out_of)
    work = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda:0")
    st = torch.cuda.current_stream()
    rg.check(call(s.wtype, W_d, s.N, s.K, batch, BF16, x_d, wide, x_of, out, width, out_of, w_d, beta, work, size, st))
    assert rg.rg_check(st) == status
    got = out.float().cpu().numpy()
    ref, mag = oracle.product_id(fwd, s.wtype, W, experts, s.N, s.K, ids, s.per_token, x, x_of == TOKEN, weights)
    live = ids >= 0
    if out_of == TOKEN:
        ref, mag = (a.reshape(rows, s.per_token, width).sum(1) for a in (ref, mag))
        live = np.ones(rows, bool)
    assert np.array_equal(got[~live], old[~live])
    o = old[live].astype(np.float64)
    ref = ref[live] + beta * o
    tol = product_tolerance(s.wtype, s.K, wide, BF16, mag[live], ref, beta, o)
    assert (np.abs(got[live] - ref) <= tol).all()


@pytest.mark.parametrize("wtype,tokens,K", ROUTES)
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("x_of", [SLOT, TOKEN])
def test_some_of_the_experts(rg, wtype, tokens, K, fwd, x_of):
    """A caller that holds the experts from the second on passes their part of W and start + 1: the slots before
    start[0] have no expert here."""
    s = _stack(rg, wtype, tokens, K)
    for out_of in (SLOT, TOKEN):
        _check(rg, s, fwd, x_of, out_of, s.start, rg.RG_OK, first=1, weigh=True, beta=0.5)
    _check(rg, s, fwd, x_of, TOKEN, s.start, rg.RG_OK, first=E - 1)


@pytest.mark.parametrize("wtype,tokens,K", ROUTES)
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("at,value", [(1, -7), (2, 1 << 30), (0, -1), (4, 1 << 30)])
def test_a_range_that_is_none(rg, wtype, tokens, K, fwd, at, value):
    """One entry of start spoiled: the ranges that it ends or begins are none where they are no range, reported; the
    slots of those add nothing to their tokens."""
    s = _stack(rg, wtype, tokens, K)
    start = s.start.copy()
    start[at] = value
    assert any(not 0 <= lo <= hi <= s.slots for lo, hi in zip(start[:-1].astype(np.int64), start[1:].astype(np.int64)))
    for out_of in (SLOT, TOKEN):
        _check(rg, s, fwd, TOKEN, out_of, start, rg.RG_ERR_INDEX, beta=-1.0)


@pytest.mark.parametrize("tokens", [27, 60, 301, 800])
@pytest.mark.parametrize("fwd", [True, False])
def test_ranges_that_overlap(rg, tokens, fwd):
    """More tiles than slots could have: those past the table are dropped, reported, and no sum takes in their rows (each
    is one of the experts' or nothing, never what the workspace held)."""
    experts = 11
    s = Stack(torch, rg, inputs.Q8_0, experts, 72, 512, np.arange(tokens * TOP) % experts, TOP)
    start = torch.tensor([0 if e % 2 == 0 else s.slots for e in range(experts + 1)], dtype=torch.int32, device="cuda:0")
    batch = rg.id_batch(experts, TOP, start, s.order_d)
    wide, width = (512, 72) if fwd else (72, 512)
    x_d = s.put(s.act(tokens, wide, BF16), BF16)
    out = s.put(np.full((tokens, width), np.nan), BF16)
    query, call = ((rg.rg_mul_mat_id_workspace_bytes, rg.rg_mul_mat_id_ws) if fwd else
                   (rg.rg_out_prod_id_workspace_bytes, rg.rg_out_prod_id_ws))
    size = query(s.wtype, s.N, s.K, batch, TOKEN)
    work = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda:0")
    st = torch.cuda.current_stream()
    rg.check(call(s.wtype, s.W_d, s.N, s.K, batch, BF16, x_d, wide, TOKEN, out, width, TOKEN, None, 0.0, work, size, st))
    assert rg.rg_check(st) == rg.RG_ERR_INDEX
    assert bool(torch.isfinite(out.float()).all())


# The input's copy, tile routes: which rows it holds.
@pytest.mark.parametrize("wtype,tokens,K", ROUTES)
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("last", ["negative", "too small"])
def test_a_last_entry_below_the_ranges(rg, wtype, tokens, K, fwd, last):
    """Only the last expert's range is spoiled by it; the others' rows are right."""
    s = _stack(rg, wtype, tokens, K)
    start = s.start.copy()
    start[E] = -1 if last == "negative" else 1
    for x_of in (SLOT, TOKEN):
        for out_of in (SLOT, TOKEN):
            _check(rg, s, fwd, x_of, out_of, start, rg.RG_ERR_INDEX, weigh=True)
