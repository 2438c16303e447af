"""The 16-bit operands that products by slot decode of the types with a minimum, on a GB300: one-hot rows bring them out
one by one."""
import numpy as np
import pytest

from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from id_common import F32, SLOT, Stack  # noqa: E402


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


# (the middle c of the codes, their number, scales and minima a super-block, their number)
TYPES = {inputs.Q4_K: (8, 16, 8, 64), inputs.Q5_K: (16, 32, 8, 64), inputs.Q2_K: (2, 4, 16, 16)}


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("centred", [True, False])
def test_operands(rg, wtype, fwd, centred):
    """A value s q - t (s = d sc, t = dmin m) is formed as fp16(fp16(s) (q - c) + fp16(c s - t)): half a step of 2^-11 for
    each of the three, of s |q - c|, of |c s - t| and of the value."""
    c, codes, subs, scales = TYPES[wtype]
    N, K = 136, 1024
    rng = np.random.default_rng(wtype)
    nb = N * K // 256
    d = (2.0 ** -8 * (1 + rng.random(nb))).astype(np.float16)
    sc = rng.integers(1, scales, (nb, subs))
    if centred:  # values around zero, as trained weights have them
        dmin, m = ((codes - 1) / 2 * d.astype(np.float32)).astype(np.float16), sc
    else:
        dmin, m = (2.0 ** -8 * (1 + rng.random(nb))).astype(np.float16), rng.integers(0, scales, (nb, subs))
    q = rng.integers(0, codes, (nb, 256))
    pack = {inputs.Q4_K: inputs.pack_q4_k, inputs.Q5_K: inputs.pack_q5_k, inputs.Q2_K: inputs.pack_q2_k}[wtype]
    W = pack(d.view(np.uint16), dmin.view(np.uint16), sc, m, q).reshape(-1)
    s, t = (np.repeat(a.astype(np.float64)[:, None] * b, 256 // subs, 1).reshape(N, K) for a, b in ((d, sc), (dmin, m)))
    codes_of = q.reshape(N, K)
    wide = K if fwd else N
    stack = Stack(torch, rg, wtype, 1, N, K, [0] * wide, 1, W=W)
    got = stack.run(fwd, F32, np.eye(wide, dtype=np.float32), SLOT, SLOT)
    got = got.T if fwd else got
    value = s * codes_of - t
    tol = 2.0 ** -11 * (s * np.abs(codes_of - c) + np.abs(c * s - t) + np.abs(value)) * (1 + 2.0 ** -9) + 3 * 2.0 ** -25
    assert (np.abs(got - value) <= tol).all()
