"""Which form an experts' product takes, without a GPU: the streaming form of a product by slot needs no workspace for
tiles, so the workspace query tells."""
import pytest

from quantized_weight_out_gb300 import binding as rg
from quantized_weight_out_gb300 import build as rgbuild
from quantized_weight_out_gb300 import inputs as i

BAD = 0x1000  # never followed


@pytest.fixture(scope="module")
def lib():
    rgbuild.build()
    return rg.load()


def _streams(wtype, experts, N, K, slots):
    return rg.rg_mul_mat_id_workspace_bytes(wtype, N, K, rg.rg_id_batch(experts, 1, slots, BAD, BAD), 0) == 0


# (type, experts, N, K, the most slots that stream): every type on large experts, on small ones, and on long rows, of
# which fewer fit a chunk
@pytest.mark.parametrize("wtype,experts,N,K,most", [
    (i.Q4_K, 8, 14336, 4096, 40), (i.Q4_K, 64, 2048, 2048, 320), (i.Q4_K, 8, 4096, 14336, 24), (i.Q4_K, 8, 4096, 8192, 40),
    (i.Q8_0, 8, 14336, 4096, 40), (i.Q8_0, 8, 4096, 14336, 24), (i.Q4_0, 64, 2048, 1536, 320), (i.Q4_0, 8, 4096, 14336, 24),
    (i.MXFP4, 8, 14336, 4096, 40), (i.MXFP4, 8, 4096, 14336, 16), (i.MXFP4, 8, 4096, 8192, 26),
    (i.Q4_1, 64, 2048, 1536, 320), (i.Q4_1, 8, 4096, 14336, 16), (i.Q2_K, 8, 14336, 4096, 40), (i.Q2_K, 8, 4096, 14336, 16),
    (i.Q6_K, 32, 4096, 4096, 256), (i.Q6_K, 8, 4096, 14336, 24), (i.Q3_K, 8, 4096, 8192, 40), (i.Q3_K, 64, 2048, 2048, 512),
    (i.Q5_0, 64, 2048, 2048, 128), (i.Q5_0, 8, 4096, 14336, 12), (i.Q5_1, 8, 14336, 4096, 8), (i.Q5_1, 64, 2048, 1536, 64),
    (i.Q5_K, 8, 14336, 4096, 8), (i.Q5_K, 64, 2048, 2048, 64),
    (i.F16, 8, 14336, 4096, 8), (i.F16, 64, 2048, 2048, 8), (i.F16, 32, 4096, 4096, 16), (i.F16, 8, 4096, 14336, 4),
    (i.BF16, 8, 14336, 4096, 8), (i.BF16, 64, 2048, 1536, 8), (i.BF16, 128, 1536, 2048, 16), (i.BF16, 8, 768, 1024, 4),
    (i.NVFP4, 8, 14336, 4096, 2), (i.NVFP4, 64, 2048, 2048, 2), (i.F32, 64, 2048, 2048, 0)])
def test_the_most_slots_that_stream(lib, wtype, experts, N, K, most):
    if i.row_bytes(wtype, K) % 16:
        pytest.skip("rows off 16 bytes are copied to the workspace in both forms")
    assert most == 0 or all(_streams(wtype, experts, N, K, s) for s in (1, 2, most))
    assert not any(_streams(wtype, experts, N, K, s) for s in (most + 1, 2 * most + 2, 1 << 14))
