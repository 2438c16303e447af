"""A call that fails is no later call's failure."""
import pytest

from quantized_weight_out_gb300 import inputs

from kv_common import RG_F32, Setup
from test_gpu_kv_attend import rg  # noqa: F401  (the fixture)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_a_failed_allocation_is_not_the_next_calls(rg):  # noqa: F811
    """rg_out_prod refuses a workspace of 35 TB (nothing is launched); the calls after it
    are good and say so."""
    s = torch.cuda.current_stream()
    x = torch.zeros(4096, device="cuda")
    su = Setup(torch, rg, inputs.F16, 64, 1, 16, [(1, 1)], atype=RG_F32)
    k, q, out = (torch.ones(64, device="cuda") for _ in range(3))

    def fail():
        return rg.rg_out_prod_variant(rg.RG_VARIANT_TC, inputs.Q8_0, x, 1 << 20, 256, x, 1 << 24, x, 0.0, s)

    for good in (lambda: rg.rg_kv_write(su.cache, su.batch, RG_F32, k, 64, 64, k, 64, 64, s),
                 lambda: rg.rg_kv_read(su.cache, su.batch, RG_F32, out, 64, 64, None, 64, 64, s),
                 lambda: rg.rg_kv_attend(su.cache, su.batch, RG_F32, q, 64, 64, 1, out, 64, 64, 0.125, 0, s),
                 lambda: rg.rg_dequant_async(inputs.F32, x, 8, 64, torch.empty(512, device="cuda"), s)):
        assert fail() == rg.RG_ERR_CUDA
        assert good() == rg.RG_OK
    rg.check(rg.rg_check(s), "rg_check")
    assert torch.equal(out, torch.ones_like(out))


def test_workspace_of_a_refused_batch(rg):  # noqa: F811
    """0 for what rg_kv_attend refuses: more rows a sequence than 2^30."""
    su = Setup(torch, rg, inputs.Q8_0, 64, 1, 16, [(1, 1)], atype=RG_F32)
    x = torch.zeros(64, device="cuda")
    for max_new, ok in ((1 << 20, True), ((1 << 20) + 1, False)):
        b = rg.kv_batch(su.start_d, su.len_d, su.table_d, 1 << 30, max_new)
        assert (rg.rg_kv_attend_workspace_bytes(su.cache, b, 1024) > 0) == ok
        if not ok:
            assert rg.rg_kv_attend(su.cache, b, RG_F32, x, 64, 64, 1024, x, 64, 64, 0.1, 0,
                                   torch.cuda.current_stream()) == rg.RG_ERR_ARG
