"""Entries of order that are no slots, in every route of the experts' products on a GB300: reported wherever they stand."""
import numpy as np
import pytest

from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from id_common import BF16, F32, SLOT, TOKEN, Stack  # noqa: E402


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("wtype,tokens", [(F32, 5), (F32, 200), (inputs.Q8_0, 5), (inputs.Q8_0, 200), (inputs.BF16, 1),
                                          (inputs.Q4_K, 900)])
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("out_of", [SLOT, TOKEN])
@pytest.mark.parametrize("where", ["first", "in a range", "behind the ranges"])
def test_order_outside_the_slots(rg, wtype, tokens, fwd, out_of, where):
    """One entry spoiled, up or down; the other slots' rows (and the sums of other tokens) are those of the whole call."""
    ids = np.arange(2 * tokens) % 3
    ids[-1] = -1
    for value in (2 * tokens, -1, -(1 << 31)):
        s = Stack(torch, rg, wtype, 3, 64, 256, ids, 2)
        wide, width = (256, 64) if fwd else (64, 256)
        x = s.act(tokens, wide, BF16)
        good = s.run(fwd, BF16, x, TOKEN, out_of)
        at = {"first": 0, "in a range": s.slots // 2 - 1, "behind the ranges": s.slots - 1}[where]
        lost = int(s.order[at])
        s.order_d[at] = value
        x_d, out = s.put(x, BF16), s.put(np.full(good.shape, np.nan), BF16)
        call, st = (rg.rg_mul_mat_id if fwd else rg.rg_out_prod_id), torch.cuda.current_stream()
        rg.check(call(wtype, s.W_d, 64, 256, s.batch, BF16, x_d, wide, TOKEN, out, width, out_of, None, 0.0, st))
        assert rg.rg_check(st) == rg.RG_ERR_INDEX
        got = out.float().cpu().numpy()
        keep = np.arange(len(good)) != (lost if out_of == SLOT else lost // 2)
        assert np.array_equal(got[keep], good[keep], equal_nan=True)
        if out_of == SLOT:
            assert np.isnan(got[lost]).all()
