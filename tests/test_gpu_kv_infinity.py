"""An infinity among the values: what the definition gives, in every dimension, where a
sequence is shared by many CTAs and its parts are joined."""
import numpy as np
import pytest

from quantized_weight_out_gb300 import inputs

from kv_common import RG_F32, Setup
from test_gpu_kv_attend import _attend, _contexts, _reference, rg  # noqa: F401  (rg: the fixture)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("wtype", [inputs.F16, inputs.BF16])
@pytest.mark.parametrize("n", [1, 7, 150])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("back", [0.0, 0.3, 1.0])
def test_an_infinity_stays_one(rg, wtype, n, sign, back):  # noqa: F811
    """One infinite value at a token that every row sees, near the newest one or far
    behind it: that infinity in its dimension, every other dimension as without it."""
    D, G, L = 128, 4, 9011
    su = Setup(torch, rg, wtype, D, 1, 64, [(n, L)], seed=5, atype=RG_F32)
    k, v = _contexts(su, 0.0)
    q = su.rng.standard_normal((n, G, D)).astype(np.float32)
    clean = v.copy()
    v[int((L - n) * (1 - back)), 0, 9] = sign * np.inf
    su.fill(k, v)
    got = _attend(rg, su, q, G, D ** -0.5)
    ref, bound = _reference(su, q, k, clean, D ** -0.5)
    rest = np.arange(D) != 9
    assert (np.abs(got - ref) <= bound)[..., rest].all()
    assert (got[..., 9] == sign * np.inf).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_in_many_short_items(rg, D):  # noqa: F811
    """Items of more than 256 rows among shorter ones, several a CTA pair, each with an infinity
    that only its last rows see: every item's own, time after time."""
    G, H = 4, 2
    lens = [(128, 128) if s % 4 == 0 else (17 + s % 40, 17 + s % 40) for s in range(240)]
    su = Setup(torch, rg, inputs.BF16, D, H, 16, lens, seed=6, atype=RG_F32)
    k, v = _contexts(su, 0.0)
    at = np.cumsum([n for n, _ in lens]) - 2  # each sequence's last token but one
    v[at, np.arange(len(lens)) % H, np.arange(len(lens)) % D] = np.inf
    su.fill(k, v)
    q = su.rng.standard_normal((su.tokens, H * G, D)).astype(np.float32)
    want = np.zeros((su.tokens, H, D), bool)
    for s, t in enumerate(at):
        want[t:t + 2, s % H, s % D] = True
    want = np.repeat(want, G, 1)
    first = _attend(rg, su, q, H * G, D ** -0.5)
    assert (first[want] == np.inf).all() and np.isfinite(first[~want]).all()
    for _ in range(20):
        assert np.array_equal(first, _attend(rg, su, q, H * G, D ** -0.5))
