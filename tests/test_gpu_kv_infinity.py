"""An infinity among the values: what the definition gives, in every dimension, where a
sequence is shared by many CTAs and its parts are joined."""
import numpy as np
import pytest

import oracle
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


@pytest.mark.parametrize("wtype", [inputs.F16, inputs.BF16])
@pytest.mark.parametrize("n", [1, 9, 150])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("L", [160, 9011])
@pytest.mark.parametrize("window", [0, 20])
def test_scores_of_minus_infinity(rg, wtype, n, D, L, window):  # noqa: F811
    """Keys of -inf under positive queries.  Rows that see others too: as without those keys.
    Rows that see nothing else: 0 / 0.  Rows that see nothing at all: zeros."""
    G, L, short = 2, max(L, n), 5
    seqs = [(n, L), (n, L), (n, max(0, n // 2))]
    su = Setup(torch, rg, wtype, D, 1, 64, seqs, seed=8, atype=RG_F32)
    k, v = _contexts(su, 0.0)
    q = np.abs(su.rng.standard_normal((su.tokens, G, D))).astype(np.float32)
    only = np.arange(L) % 3 == 1       # sequence 0: every third key; sequence 1: all but the last token's
    k[:L][only, 0, 5] = -np.inf
    k[L:2 * L - short, 0, 5] = -np.inf
    su.fill(k, v)
    got = _attend(rg, su, q, G, D ** -0.5, window)
    # _reference's bound, with the sums of magnitudes over the finite keys only
    ref, bound = [], []
    u, lo = (2.0 ** -8 if wtype == inputs.BF16 else 2.0 ** -11), 0
    for s, (n_s, L_s) in enumerate(seqs):
        K, V = (oracle.kv_values(wtype, x[lo:lo + L_s]).astype(np.float64) for x in (k, v))
        lo += L_s
        qq = q[su.start[s]:su.start[s] + n_s].astype(np.float64)
        with np.errstate(all="ignore"):
            out, mag = oracle.kv_attend(qq, K, V, su.positions(s), D ** -0.5, window)
        S = np.einsum("ihd,jd->ihj", np.abs(qq), np.abs(np.where(np.isinf(K), 0, K))[:, 0]).max(-1, initial=0)[..., None]
        eta = np.expm1(D ** -0.5 * S * (u + D * 2.0 ** -23 + 2.0 ** -22)) + 2.0 ** -21
        b = mag * (2 * eta + u + 2 * L_s * 2.0 ** -24) + L_s * 2.0 ** -32 * np.abs(V).max(initial=0)
        ref.append(out)
        bound.append(b + (np.abs(out) + b) * 2.0 ** -22 + 1e-7)
    ref, bound = np.concatenate(ref), np.concatenate(bound)
    nan = np.isnan(ref)
    assert nan.any() == (n > short) and (np.isnan(got) == nan).all()
    assert (np.abs(got - ref) <= bound)[~nan].all()
    assert (got[su.start[2]:su.start[2] + n - n // 2] == 0).all()

