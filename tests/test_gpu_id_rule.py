"""Experts' products of 16-bit weights on both sides of the rule that picks their form, on a GB300: experts of 64 MB
stream up to a slot each, whoever has them."""
import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from id_common import BF16, F32, SLOT, TOKEN, product_tolerance, torch_act  # noqa: E402


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("wtype", [inputs.F16, inputs.BF16])
@pytest.mark.parametrize("atype", [F32, BF16])
@pytest.mark.parametrize("ids,per", [([5] * 8, 1), ([0, 2, 2, 0, 5, -1, 5, 5], 2), ([2] * 9, 1), ([7, 5, 0, 5], 1)])
def test_large_experts(rg, wtype, atype, ids, per):
    E, N, K = 8, 8192, 4096
    rng = np.random.default_rng(len(ids))
    rows = np.ascontiguousarray(inputs.gen_weight(wtype, 64, K, seed=3, stream=1)).view(np.uint8).reshape(64, -1)
    pick = rng.integers(0, 64, E * N)
    W = torch.from_numpy(rows).cuda()[torch.from_numpy(pick).cuda()].reshape(-1)
    dense = oracle.dequant(wtype, rows.reshape(-1), 64, K).astype(np.float64)
    ids = np.asarray(ids)
    tokens = len(ids) // per
    start, order = oracle.group(ids, E)
    start_d, order_d = torch.from_numpy(start).cuda(), torch.from_numpy(order).cuda()
    batch = rg.id_batch(E, per, start_d, order_d)
    assert (rg.rg_mul_mat_id_workspace_bytes(wtype, N, K, batch, SLOT) == 0) == (len(ids) <= E)
    x = torch.randn(tokens, K, device="cuda:0").to(torch_act(torch, atype))
    a = x.double().cpu().numpy()
    y = torch.full((tokens, N), float("nan"), dtype=torch_act(torch, atype), device="cuda:0")
    w = rng.random(len(ids)).astype(np.float32)
    s = torch.cuda.current_stream()
    rg.check(rg.rg_mul_mat_id(wtype, W, N, K, batch, atype, x, K, TOKEN, y, N, TOKEN, torch.from_numpy(w).cuda(), 0.0, s))
    assert rg.rg_check(s) == 0
    each, size = a @ dense.T, np.abs(a) @ np.abs(dense).T   # every token with every generated row
    ref, mag = np.zeros((tokens, N)), np.zeros((tokens, N))
    for i, e in enumerate(ids):
        if e >= 0:
            of = pick[e * N:(e + 1) * N]
            ref[i // per] += w[i].astype(np.float64) * each[i // per][of]
            mag[i // per] += w[i].astype(np.float64) * size[i // per][of]
    assert (np.abs(y.double().cpu().numpy() - ref) <= product_tolerance(wtype, K, K, atype, mag, ref)).all()
