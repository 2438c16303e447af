"""Seeded random batches with infinities and NaN among the values near sequences' ends, where
some rows see them and others do not: every output is the definition's, finite or not."""
import numpy as np
import pytest

from quantized_weight_out_gb300 import inputs

from kv_common import RG_BF16, RG_F16, RG_F32, Setup, to_act
from test_gpu_kv_attend import _attend, _contexts, _reference, rg  # noqa: F401  (rg: the fixture)
from test_gpu_kv_random import _sequence

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
              pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.mark.parametrize("seed", range(40))
def test_random_batches_with_infinities(rg, seed):  # noqa: F811
    r = np.random.default_rng(5000 + seed)
    wtype = int(r.choice([inputs.F16, inputs.BF16, inputs.Q8_0, inputs.Q4_0]))
    atype = int(r.choice([RG_F32, RG_F16, RG_BF16]))
    D, H = int(r.choice([64, 128, 256])), int(r.choice([1, 2, 3]))
    G, P = int(r.choice([1, 2, 4, 8, 16, 40])), int(r.choice([16, 48, 64, 256]))
    seqs = [_sequence(r) for _ in range(int(r.integers(1, 8)))]
    if sum(n for n, _ in seqs) == 0:
        seqs.append((1, 5))
    while sum(n for n, _ in seqs) * H * G > 6000 and len(seqs) > 1:
        seqs.remove(max(seqs))
    if seed % 5 == 0:
        seqs.append((int(r.integers(1, 40)), int(r.integers(3000, 9000))))
    window, scale = int(r.choice([0, 0, 1, 17, 130, 1000])), float(r.choice([1.0, -1.0])) * D ** -0.5
    su = Setup(torch, rg, wtype, D, H, P, seqs, seed=seed, atype=atype, fill=None if seed % 2 else "random")
    k, v = _contexts(su, 1.0)
    finite, ends = v.copy(), np.cumsum(np.maximum(su.len, 0))
    for _ in range(int(r.integers(1, 6)) if len(v) else 0):
        t = min(len(v) - 1, max(0, int(r.choice(ends)) - 1 - int(r.integers(0, 200))))
        v[t, int(r.integers(0, H)), int(r.integers(0, D))] = r.choice([np.inf, -np.inf, np.nan])
    su.fill(k, v)
    q = to_act(r.standard_normal((su.tokens, H * G, D)).astype(np.float32), atype)
    got = _attend(rg, su, q, H * G, scale, window)
    ref = _reference(su, q, k, v, scale, window)[0]
    bound = _reference(su, q, k, finite, scale, window)[1]
    there = np.isfinite(ref)
    assert (np.abs(got - ref) <= bound)[there].all()
    assert np.array_equal(got[~there], ref[~there], equal_nan=True)
