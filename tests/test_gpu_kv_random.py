"""Seeded random batches through rg_kv_attend against the oracle: types, head sizes
and layouts, pages, windows, scales, and sequences of every kind side by side."""
import numpy as np
import pytest

from quantized_weight_out_gb300 import inputs

from kv_common import RG_BF16, RG_F16, RG_F32
from test_gpu_kv_attend import _case, rg  # noqa: F401  (rg: the fixture)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _sequence(r):
    """(new tokens, length with them) of one kind or another."""
    kind = r.integers(0, 7)
    if kind == 0:
        return 1, int(r.integers(1, 2000))
    if kind == 1:
        n = int(r.integers(2, 12))
        return n, n + int(r.integers(0, 1500))
    if kind == 2:
        n = int(r.integers(12, 200))
        return n, n + int(r.integers(0, 900))
    if kind == 3:
        n = int(r.integers(1, 400))
        return n, n
    if kind == 4:
        return 0, int(r.integers(0, 100))
    if kind == 5:
        n = int(r.integers(1, 90))
        return n, int(r.integers(0, n + 1))  # some tokens before the cache's start
    return 1, 16 * int(r.integers(1, 40)) + int(r.integers(0, 2))


@pytest.mark.parametrize("seed", range(48))
def test_random_batches(rg, seed):  # noqa: F811
    r = np.random.default_rng(1000 + seed)
    wtype = int(r.choice([inputs.F16, inputs.BF16, inputs.Q8_0, inputs.Q4_0]))
    atype = int(r.choice([RG_F32, RG_F16, RG_BF16]))
    D, H = int(r.choice([64, 128, 256])), int(r.choice([1, 2, 3, 5]))
    G = int(r.choice([1, 2, 3, 4, 7, 8, 16]))
    P = int(r.choice([16, 32, 48, 64, 112, 256]))
    seqs = [_sequence(r) for _ in range(int(r.integers(1, 9 if seed % 6 else 40)))]
    if sum(n for n, _ in seqs) == 0:
        seqs.append((1, 5))
    # the oracle walks rows x heads in Python: keep that to some thousands
    while sum(n for n, _ in seqs) * H * G > 9000 and len(seqs) > 1:
        seqs.remove(max(seqs))
    window = int(r.choice([0, 0, 0, 1, 17, 130, 1000]))
    scale = float(r.choice([1.0, -1.0, 2.0])) * D ** -0.5
    _case(rg, wtype, atype, D, H, G, P, seqs, window=window, seed=seed, scale=scale,
          fill="random" if seed % 3 == 0 else None)
