"""rg_kv_attend against the oracle's sums in 64 bits.

The bound of an output is derived from the roundings that the header states.
With z_j the score, B = sum_j w_j |v_j| / sum_j w_j and u the unit roundoff of
the operand type (fp16 2^-11, bf16 2^-8):
  - a score's error is at most scale * S_j * (r u + D 2^-23), S_j = sum_d |q_d||k_jd|,
    r the number of its operands that are rounded (decoded keys; F32 queries, or
    queries of the other 16-bit type), and |z_j| 2^-22 from the F32 scaling and the
    exponential's argument; a weight's relative error is then at most expm1 of it
    plus 2^-21 (the exponential), and the quotient's twice that times B;
  - the probability's rounding adds u B, a decoded value's u B, F32 sums of L terms
    at most L 2^-24 B (each side), a probability below fp16's normal range 2^-32 max|v|
    a token (probabilities are scaled so that the largest is at least 2^7);
  - the result's own rounding.
"""
import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

from kv_common import RG_BF16, RG_F16, RG_F32, Setup, to_act

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
F16, BF16, Q8, Q4 = inputs.F16, inputs.BF16, inputs.Q8_0, inputs.Q4_0


@pytest.fixture(scope="module")
def rg():
    from quantized_weight_out_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def _contexts(su, strong=3.0):
    total = int(np.maximum(su.len, 0).sum())
    ch = 1 + (su.rng.random((1, su.H, su.D)) < 0.05) * strong
    k = (su.rng.standard_normal((total, su.H, su.D)) * ch).astype(np.float32)
    v = su.rng.standard_normal((total, su.H, su.D)).astype(np.float32)
    return k, v


def _attend(rg, su, q, heads, scale, window=0, stream=None, out=None, check=True):
    stream = stream or torch.cuda.current_stream()
    D = su.D
    qd = su.tensor(q)
    if out is None:
        out = torch.full((max(su.tokens, 1), heads, D), 5.0, device=su.dev, dtype=qd.dtype)
    rg.check(rg.rg_kv_attend(su.cache, su.batch, su.atype, qd, heads * D, D, heads, out, heads * D, D, scale, window,
                             stream), "rg_kv_attend")
    if check:
        rg.check(rg.rg_check(stream), "rg_check")
    return out.float().cpu().numpy()[:su.tokens].astype(np.float64)


def _reference(su, q, k, v, scale, window=0):
    """(out, bound) of the batch's rows; q as the activations hold it, k and v F32."""
    ks, vs = oracle.kv_values(su.wtype, k), oracle.kv_values(su.wtype, v)
    start = np.concatenate([[0], np.cumsum(np.maximum(su.len, 0))])
    u = 2.0 ** -8 if su.wtype == BF16 else 2.0 ** -11
    quant = su.wtype in (Q8, Q4)
    rounded_q = su.atype == RG_F32 or (su.atype == RG_BF16) != (su.wtype == BF16)
    outs, bounds = [], []
    for s, (n, L) in enumerate(su.seqs):
        lo = int(start[s])
        K, V = ks[lo:lo + max(L, 0)], vs[lo:lo + max(L, 0)]
        qq = q[su.start[s]:su.start[s] + n]
        out, mag = oracle.kv_attend(qq, K, V, su.positions(s), scale, window)
        if len(K):
            G = q.shape[1] // su.H
            S = np.einsum("ihgd,jhd->ihgj", np.abs(qq.astype(np.float64)).reshape(n, su.H, G, su.D),
                          np.abs(K.astype(np.float64))).max(-1).reshape(n, q.shape[1], 1)
            err = abs(scale) * S * ((quant + rounded_q) * u + su.D * 2.0 ** -23 + 2.0 ** -22)
            eta = np.expm1(err) + 2.0 ** -21
            b = mag * (2 * eta + u * (1 + quant) + 2 * len(K) * 2.0 ** -24) + len(K) * 2.0 ** -32 * np.abs(V).max()
        else:
            b = np.zeros_like(out)
        act = {RG_F32: 2.0 ** -22, RG_F16: 2.0 ** -11, RG_BF16: 2.0 ** -8}[su.atype]
        outs.append(out)
        bounds.append(b + (np.abs(out) + b) * act + 1e-7)
    return np.concatenate(outs), np.concatenate(bounds)


def _case(rg, wtype, atype, D, H, G, P, seqs, window=0, seed=1, scale=None, fill=None):
    su = Setup(torch, rg, wtype, D, H, P, seqs, seed=seed, atype=atype, fill=fill)
    k, v = _contexts(su)
    su.fill(k, v)
    q = to_act(su.rng.standard_normal((su.tokens, H * G, D)).astype(np.float32), atype)
    scale = D ** -0.5 if scale is None else scale
    got = _attend(rg, su, q, H * G, scale, window)
    ref, bound = _reference(su, q, k, v, scale, window)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / bound)))
    return su, k, v, q


DECODE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 333), (1, 1000)]
CHUNKS = [(2, 2), (7, 40), (3, 3), (33, 100), (64, 64), (20, 333), (0, 12), (1, 70)]


@pytest.mark.parametrize("wtype", [F16, BF16, Q8, Q4])
@pytest.mark.parametrize("atype", [RG_F32, RG_F16, RG_BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", ["decode", "chunk"])
def test_types_and_dims(rg, wtype, atype, D, form):
    """Every storage type, activation type and head size; the pool's other bytes are NaN."""
    _case(rg, wtype, atype, D, 2, 3, 32, DECODE if form == "decode" else CHUNKS)


@pytest.mark.parametrize("H,G", [(1, 1), (5, 1), (2, 4), (1, 7), (1, 16), (2, 17), (1, 40), (3, 8)])
@pytest.mark.parametrize("form", ["decode", "chunk"])
def test_head_layouts(rg, H, G, form):
    _case(rg, Q8, RG_BF16, 128, H, G, 16, DECODE if form == "decode" else CHUNKS)


@pytest.mark.parametrize("P", [16, 48, 64, 256])
@pytest.mark.parametrize("window", [1, 5, 16, 64, 100, 4000])
def test_windows_and_pages(rg, P, window):
    _case(rg, Q8, RG_F16, 64, 2, 2, P, [(1, 500), (9, 301), (130, 400), (3, 3), (1, 1)], window=window)


@pytest.mark.parametrize("wtype", [F16, BF16, Q8, Q4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts(rg, wtype, D):
    """Whole prompts packed behind one another, ragged, beside a decoding sequence."""
    _case(rg, wtype, RG_BF16, D, 2, 4, 64, [(300, 300), (129, 129), (1, 200), (257, 700), (16, 16)])


@pytest.mark.parametrize("wtype,D", [(Q8, 128), (Q4, 64), (BF16, 128), (F16, 256)])
def test_long_context_is_split_and_joined(rg, wtype, D):
    """One sequence's tiles shared by every CTA."""
    _case(rg, wtype, RG_BF16, D, 2, 4, 64, [(1, 20011)])
    _case(rg, wtype, RG_BF16, D, 1, 4, 64, [(6, 9001), (1, 130)])
    _case(rg, wtype, RG_F32, D, 1, 4, 64, [(40, 9001), (1, 130)])


def test_maxima_that_rise_along_the_keys(rg):
    """Scores that grow by tens along the cache, so that the running reference moves
    in every tile: the accumulators are rescaled again and again."""
    for D, n in ((128, 1), (128, 90), (256, 90), (64, 90)):
        L, G = 1200, 4
        su = Setup(torch, rg, F16, D, 1, 64, [(n, L)], atype=RG_F32)
        k, v = _contexts(su, 0.0)
        q = np.repeat(su.rng.standard_normal((1, G, D)), n, 0).astype(np.float16).astype(np.float32)
        k += (np.arange(L)[:, None, None] / L * 6).astype(np.float32) * q[0, :1]
        su.fill(k, v)
        got = _attend(rg, su, q, G, 0.4)
        ref, bound = _reference(su, q, k, v, 0.4)
        assert (np.abs(got - ref) <= bound).all(), (D, n)


@pytest.mark.parametrize("n", [1, 40, 200])
@pytest.mark.parametrize("D", [64, 256])
def test_rows_that_see_nothing(rg, n, D):
    """Lengths below the new tokens' number, of zero too: zeros for the rows before
    the cache's start, and no error."""
    su, *_ = _case(rg, Q8, RG_F32, D, 2, 2, 16, [(n, n // 2), (1, 0), (n, 0), (1, 33), (3, 2)])
    assert su.seqs


@pytest.mark.parametrize("wtype", [F16, BF16, Q8, Q4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(4, 2), (20, 2), (150, 2)])
@pytest.mark.parametrize("window", [0, 9])
def test_hidden_values_do_not_reach_a_row(rg, wtype, D, n, G, window):
    """Keys and values that are not finite at positions that some of the new tokens
    see and others do not: the others' results are as without them, the tokens that
    see them get what the definition gives (NaN, or an infinity from a value)."""
    H, L = 1, n + 37
    su = Setup(torch, rg, wtype, D, H, 16, [(n, L)], seed=4, atype=RG_F32)
    k, v = _contexts(su)
    q = su.rng.standard_normal((n, G, D)).astype(np.float32)
    at_v, at_k = L - n // 2, L - max(1, n // 4)
    at_v = min(at_v, at_k - 1)
    clean_k, clean_v = k.copy(), v.copy()
    v[at_v, 0, 7] = np.inf
    k[at_k, 0, 3] = np.nan
    su.fill(k, v)
    got = _attend(rg, su, q, G, D ** -0.5, window)
    ref, bound = _reference(su, q, clean_k, clean_v, D ** -0.5, window)
    pos = su.positions(0)
    see = lambda p: (pos >= p) & ((pos < p + window) if window else True)  # noqa: E731
    sees_v, sees_k = see(at_v), see(at_k)
    none = ~sees_v & ~sees_k
    assert none.any() and sees_k.any()
    assert (np.abs(got - ref) <= bound)[none].all()
    assert np.isnan(got[sees_k]).all()
    only_v = sees_v & ~sees_k
    block = slice(0, 32) if wtype in (Q8, Q4) else slice(7, 8)  # a block with an infinity is NaN whole
    assert not np.isfinite(got[only_v][..., block]).any()
    rest = np.ones(D, bool)
    rest[block] = False
    assert (np.abs(got - ref) <= bound)[only_v][..., rest].all()


def test_large_scores_and_far_maxima(rg):
    """Scores of hundreds, with the maximum late, early or shared by two tokens."""
    D, L = 128, 1500
    for at in ([3], [L - 1], [10, 1200]):
        su = Setup(torch, rg, F16, D, 1, 64, [(1, L)], atype=RG_F32)
        k, v = _contexts(su, 0.0)
        q = su.rng.standard_normal((1, 4, D)).astype(np.float16).astype(np.float32)
        k[at] = q[0, 0] * 4
        su.fill(k, v)
        got = _attend(rg, su, q, 4, 0.5)
        ref, bound = _reference(su, q, k, v, 0.5)
        assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("n", [1, 150])
def test_a_window_of_any_length(rg, n):
    """Windows past every length hide nothing, the largest int included."""
    su = Setup(torch, rg, Q8, 64, 2, 16, [(n, n + 300), (n, n // 2)], atype=RG_F32)
    k, v = _contexts(su)
    su.fill(k, v)
    q = su.rng.standard_normal((su.tokens, 4, 64)).astype(np.float32)
    none = _attend(rg, su, q, 4, 0.125)
    ref, bound = _reference(su, q, k, v, 0.125)
    assert (np.abs(none - ref) <= bound).all()
    for window in (n + 400, 1 << 20, 2 ** 31 - 1):
        assert (np.abs(_attend(rg, su, q, 4, 0.125, window) - ref) <= bound).all()


def test_negative_and_zero_scale(rg):
    _case(rg, Q8, RG_F32, 64, 2, 2, 16, [(1, 100), (30, 90)], scale=0.0)
    _case(rg, Q8, RG_F32, 64, 2, 2, 16, [(1, 100), (30, 90)], scale=-0.2)


def test_strides(rg):
    """Queries inside a fused row, results head-major."""
    D, H, G = 64, 2, 3
    su = Setup(torch, rg, Q8, D, H, 16, [(5, 30), (1, 77), (40, 41)], atype=RG_BF16)
    k, v = _contexts(su)
    su.fill(k, v)
    T, Hq = su.tokens, H * G
    q = to_act(su.rng.standard_normal((T, Hq, D)).astype(np.float32), RG_BF16)
    fused = torch.zeros((T, (Hq + 3) * D), device=su.dev, dtype=torch.bfloat16)
    fused[:, D:(Hq + 1) * D] = su.tensor(q).view(T, -1)
    out = torch.zeros((Hq, T, D + 8), device=su.dev, dtype=torch.bfloat16)
    s = torch.cuda.current_stream()
    rg.check(rg.rg_kv_attend(su.cache, su.batch, RG_BF16, fused[:, D:], fused.stride(0), D, Hq, out, D + 8,
                             T * (D + 8), D ** -0.5, 0, s))
    rg.check(rg.rg_check(s))
    ref, bound = _reference(su, q, k, v, D ** -0.5)
    got = out.float().cpu().numpy()
    assert (np.abs(got[..., :D].transpose(1, 0, 2) - ref) <= bound).all() and (got[..., D:] == 0).all()


@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("D", [64, 256])
def test_bad_numbers_are_reported_not_followed(rg, n, D):
    """A page outside the pool hides its tokens, a bad length or row range empties
    its sequence; the others' results stand."""
    H, G, P = 2, 2, 16
    seqs = [(n, n + 60), (n, n + 9), (n, n + 30)]
    su = Setup(torch, rg, Q8, D, H, P, seqs, atype=RG_F32)
    k, v = _contexts(su)
    su.fill(k, v)
    q = su.rng.standard_normal((su.tokens, H * G, D)).astype(np.float32)
    ref, bound = _reference(su, q, k, v, D ** -0.5)
    table = su.table.copy()
    table[0, 0] = 1 << 20
    lens = su.len.copy()
    lens[1] = -3
    su.table_d.copy_(torch.from_numpy(table))
    su.len_d.copy_(torch.from_numpy(lens))
    got = _attend(rg, su, q, H * G, D ** -0.5, check=False)
    s = torch.cuda.current_stream()
    assert rg.rg_check(s) == rg.RG_ERR_INDEX and rg.rg_check(s) == rg.RG_OK
    assert (np.abs(got - ref) <= bound)[2 * n:].all()
    assert (got[n:2 * n] == 5.0).all()
    ks, vs = oracle.kv_values(Q8, k[P:n + 60]), oracle.kv_values(Q8, v[P:n + 60])
    want, mag = oracle.kv_attend(q[:n], ks, vs, su.positions(0) - P, D ** -0.5)
    assert (np.abs(got[:n] - want) <= 2e-2 * mag + 1e-6).all()


def test_streams_graphs_workspace_and_repeats(rg):
    """The same words on another stream, in a replayed graph whose lengths grow, with
    a caller's workspace, and time after time; launches are counted."""
    D, H, G = 128, 2, 4
    su = Setup(torch, rg, Q8, D, H, 32, [(1, 3000), (1, 700), (1, 64)], atype=RG_BF16)
    k, v = _contexts(su)
    su.fill(k, v)
    q = to_act(su.rng.standard_normal((3, H * G, D)).astype(np.float32), RG_BF16)
    first = _attend(rg, su, q, H * G, 0.1)
    before = rg.rg_launch_count()
    assert np.array_equal(first, _attend(rg, su, q, H * G, 0.1))
    assert rg.rg_launch_count() - before in (1, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert np.array_equal(first, _attend(rg, su, q, H * G, 0.1, stream=side))
    need = rg.rg_kv_attend_workspace_bytes(su.cache, su.batch, H * G)
    ws = torch.empty(need, dtype=torch.uint8, device=su.dev)
    qd = su.tensor(q)
    out = torch.zeros((3, H * G, D), device=su.dev, dtype=torch.bfloat16)
    s = torch.cuda.current_stream()
    args = (su.cache, su.batch, RG_BF16, qd, H * G * D, D, H * G, out, H * G * D, D, 0.1, 0)
    rg.check(rg.rg_kv_attend_ws(*args, ws, need, s))
    assert np.array_equal(first, out.float().cpu().numpy())
    if need:
        assert rg.rg_kv_attend_ws(*args, ws, need - 1, s) == rg.RG_ERR_ARG
        assert rg.rg_kv_attend_ws(*args, ws.data_ptr() + 16, need, s) == rg.RG_ERR_ALIGN
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rg.check(rg.rg_kv_attend_ws(*args, ws, need, torch.cuda.current_stream()))
    out.zero_()
    graph.replay()
    assert np.array_equal(first, out.float().cpu().numpy())
    su.len_d.copy_(torch.tensor([2500, 701 - 5, 10], dtype=torch.int32))
    graph.replay()
    again = out.float().cpu().numpy()
    assert np.array_equal(again, _attend(rg, su, q, H * G, 0.1)) and not np.array_equal(again, first)


def test_query_beyond_fp16_is_reported(rg):
    su = Setup(torch, rg, Q8, 64, 1, 16, [(1, 20)], atype=RG_F32)
    k, v = _contexts(su)
    su.fill(k, v)
    q = np.ones((1, 2, 64), np.float32)
    q[0, 1, 5] = 1e6
    _attend(rg, su, q, 2, 0.1, check=False)
    s = torch.cuda.current_stream()
    assert rg.rg_check(s) == rg.RG_ERR_RANGE and rg.rg_check(s) == rg.RG_OK
