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


@pytest.mark.parametrize("wtype", [inputs.F16, inputs.Q8_0, inputs.Q4_0])
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("large", [True, False])
def test_weights_beside_magnitudes(rg, wtype, fwd, large):
    """A slot's weight times its row's power of two (2^109 or 2^-120) passes F32's range: 2^19 2^109, 2^-40 2^-120.  The
    sum times both does not: a row has one value, 2^123 or 2^-106, beside weights W of about 2^-20 or 2^14.  The
    streaming form gives the result; the tiles report a factor that is too large, and lose 2^-135 of W to one that is
    too small."""
    for tokens in (2, 150):
        s = _stack(rg, wtype, tokens)
        W = s.W.view(np.uint8).copy()
        if wtype == inputs.F16:
            W = (W.view(np.float16).astype(np.float32) * (2.0 ** -14 if large else 2.0 ** 19)).astype(np.float16)
        else:  # the blocks' scale: 2^-24, or what brings the largest values to 2^15
            d = 2.0 ** -24 if large else 2.0 ** 8 if wtype == inputs.Q8_0 else 2.0 ** 12
            W.reshape(-1, 34 if wtype == inputs.Q8_0 else 18)[:, :2] = np.float16([d]).view(np.uint8)
        s.W = W.reshape(-1).view(np.uint8)
        s.W_d = torch.from_numpy(s.W).cuda()
        wide = 512 if fwd else 72
        x = np.zeros((s.slots, wide), np.float32)
        x[np.arange(s.slots), s.rng.integers(0, wide, s.slots)] = 2.0 ** 123 if large else 2.0 ** -106
        weights = ((2.0 ** 19 if large else 2.0 ** -40) * (1 + 0.25 * s.rng.random(s.slots))).astype(np.float32)
        ref, mag = oracle.product_id(fwd, wtype, s.W, 4, 72, 512, s.ids, 2, x, False, weights)
        assert 2.0 ** -134 < mag.max() < 3e38
        few = fwd and tokens == 2
        if large and not few:
            out, st = torch.empty(s.slots, s.N if fwd else s.K, device="cuda:0"), torch.cuda.current_stream()
            call = rg.rg_mul_mat_id if fwd else rg.rg_out_prod_id
            rg.check(call(wtype, s.W_d, s.N, s.K, s.batch, F32, s.put(x, F32), wide, SLOT, out, out.shape[1], SLOT,
                          torch.from_numpy(weights).cuda(), 0.0, st))
            assert rg.rg_check(st) == rg.RG_ERR_RANGE
            continue
        got = s.run(fwd, F32, x, SLOT, SLOT, weights)
        # (the helper's bound without its floor of 1e-30; a subnormal result is rounded to a multiple of 2^-149)
        tol = product_tolerance(wtype, 512, wide, F32, mag, ref) - 1e-30 + 2.0 ** -149
        if not few:
            w = np.abs(oracle.dequant(wtype, s.W, 4 * 72, 512).astype(np.float64).reshape(4, 72, 512)[s.ids])
            tol = tol + 2.0 ** -135 * w.sum(2 if fwd else 1)
        assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("wtype", [inputs.F16, inputs.Q8_0, inputs.Q6_K, inputs.MXFP4])
@pytest.mark.parametrize("fwd", [True, False])
def test_an_infinity_beside_large_values(rg, wtype, fwd):
    """A row with one infinity gives infinities of the signs of its weights (NaN for zeros), whatever else it holds: its
    finite values beyond the operands' range are not infinite."""
    for tokens in (2, 150):
        s = _stack(rg, wtype, tokens, K=2048)
        wide = 2048 if fwd else 72
        x = s.act(s.slots, wide, F32, 1e30)
        x[1, 5] = np.inf
        got = s.run(fwd, F32, x, SLOT, SLOT)
        w = oracle.dequant(wtype, s.W.reshape(4, -1)[s.ids[1]], 72, 2048)
        along = w[:, 5] if fwd else w[5]
        big = np.abs(along) > 2.0 ** -14   # (a decoded operand is a normal fp16 there)
        assert big.any() and np.array_equal(got[1][big], np.inf * np.sign(along[big]))
        assert np.isnan(got[1][along == 0]).all()
