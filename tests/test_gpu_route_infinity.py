"""The router's gradient on a GB300 where logits or the weights' gradient are not finite."""
import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("E,top", [(8, 2), (40, 4), (300, 8)])
@pytest.mark.parametrize("mode", [0, 1])
def test_back(rg, E, top, mode):
    """Rows with one or two logits of +inf, all of -inf, an infinite or NaN gradient, and logits whose exponentials
    vanish: NaN exactly where the definition has NaN, zeros where an expert takes no part."""
    rng = np.random.default_rng(E)
    T = 8
    logits = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, top)).astype(np.float32)
    logits[1, 3] = np.inf
    logits[2, [0, E - 1]] = np.inf
    logits[3] = -np.inf
    logits[4, 5:] = -np.inf
    logits[4, 1] = np.inf
    logits[5, :E // 2] = -300.0   # (their exponentials are 0 in F32)
    dw[6, 1] = np.inf
    dw[7, 0] = np.nan
    ids, weights = oracle.route(logits, top, mode, 1.5)
    dl = torch.full((T, E), 7.0, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_route_back(torch.from_numpy(logits).cuda(), E, T, E, top, mode, 1.5, torch.from_numpy(ids).cuda(),
                              torch.from_numpy(dw).cuda(), dl, E, s))
    assert rg.rg_check(s) == 0
    got = dl.cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        ref = oracle.route_back(logits, ids, mode, 1.5, dw)
    finite = [0, 3, 5]
    most = np.abs(dw[finite]).max()
    assert (np.abs(got[finite] - ref[finite]) <= (E + 64) * 2.0 ** -24 * 1.5 * 2 * most).all()
    for t in (1, 2, 4, 6, 7):
        assert np.array_equal(np.isfinite(got[t]), np.isfinite(ref[t]))
        assert np.array_equal(np.isnan(got[t]), np.isnan(ref[t]))
        assert (got[t][ref[t] == 0] == 0).all()
    # what the forward says of the same rows
    assert np.isnan(weights[1]).all() and np.isnan(got[1][ids[1]]).all()
