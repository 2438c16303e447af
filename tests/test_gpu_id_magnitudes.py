"""Experts' products on a GB300 at the ends of the activations' range: no factor of a row overflows or vanishes where
the result does not."""
import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from id_common import F32, SLOT, TOKEN, Stack, product_tolerance  # noqa: E402


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


def _stack(rg, wtype, tokens, N=72, K=512, W=None):
    rng = np.random.default_rng(tokens)
    ids = np.stack([rng.permutation(4)[:2] for _ in range(tokens)]).reshape(-1)
    return Stack(torch, rg, wtype, 4, N, K, ids, 2, seed=tokens, W=W)


@pytest.mark.parametrize("wtype", inputs.ALL_TYPES)
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("scale", [1e-30, 2.0 ** 115, 4e35])
def test_magnitudes_of_every_type(rg, wtype, fwd, scale):
    """Rows whose largest magnitudes lie on both sides of 2^118, and tiny ones, in the streaming form and the tiles; the
    results are finite.  Rows of W that are zeros give zeros."""
    for tokens in (2, 9, 150):
        s = _stack(rg, wtype, tokens)
        W = s.W.view(np.uint8).reshape(4 * 72, -1).copy()
        W[:3] = 0
        s.W = W.reshape(-1)
        s.W_d = torch.from_numpy(s.W).cuda()
        x = s.act(tokens, 512 if fwd else 72, F32, scale)
        ref, mag = oracle.product_id(fwd, wtype, s.W, 4, 72, 512, s.ids, 2, x, True, None)
        assert mag.max() < 3e38
        got = s.run(fwd, F32, x, TOKEN, SLOT)
        assert (np.abs(got - ref) <= product_tolerance(wtype, 512, x.shape[1], F32, mag, ref)).all()
