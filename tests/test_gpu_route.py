"""The router on a GB300 against the definition in 64 bits."""
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


def _route(rg, logits, top, mode, scale=1.0, pad=0, plan=True):
    T, E = logits.shape
    l = torch.full((T, E + pad), 9e9, device="cuda:0")
    l[:, :E] = torch.from_numpy(logits).cuda()
    ids = torch.full((T, top), 77, dtype=torch.int32, device="cuda:0")
    w = torch.full((T, top), 7.0, device="cuda:0")
    start = torch.full((E + 1,), 77, dtype=torch.int32, device="cuda:0")
    order = torch.full((T * top,), 77, dtype=torch.int32, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_route(l, E + pad, T, E, top, mode, scale, ids, w, start if plan else None, order if plan else None, s))
    assert rg.rg_check(s) == 0
    return [x.cpu().numpy() for x in (ids, w, start, order)]


def _check(rg, logits, top, mode, scale=1.0, pad=0):
    ids, w, start, order = _route(rg, logits, top, mode, scale, pad)
    ref_i, ref_w = oracle.route(logits, top, mode, scale)
    assert np.array_equal(ids, ref_i)
    # each exp is within 2 ulp, its argument (a difference of F32 values) half an ulp of itself, the sum one half step
    # a term, the quotient and the product one each
    far = float(np.abs(np.where(np.isfinite(logits), logits, 0)).max())
    tol = (logits.shape[1] + 8 + 2 * min(2 * far, 104)) * 2.0 ** -24
    fine = np.isfinite(ref_w)
    assert np.array_equal(np.isnan(w), np.isnan(ref_w))
    assert (np.abs(w - ref_w)[fine] <= tol * np.abs(ref_w[fine]) + 1e-37).all()
    s, o = oracle.group(ref_i, logits.shape[1])
    assert np.array_equal(start, s) and np.array_equal(order, o)


@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (1, 8, 2), (1, 8, 8), (7, 33, 32), (300, 60, 4), (1000, 128, 8),
                                     (65, 256, 8), (33, 257, 6), (40, 1024, 32), (2049, 64, 1)])
@pytest.mark.parametrize("mode", [0, 1])
def test_route(rg, T, E, top, mode):
    _check(rg, (np.random.default_rng(E + T).standard_normal((T, E)) * 2).astype(np.float32), top, mode, 1.0 + mode, pad=3)


@pytest.mark.parametrize("mode", [0, 1])
def test_ties_and_masks(rg, mode):
    """Equal logits, zeros of either sign, the type's lowest value, -inf, NaN, +inf, rows that leave nothing."""
    E = 40
    rows = np.zeros((10, E), np.float32)
    rows[1, ::2] = -0.0
    rows[2] = np.finfo(np.float32).min
    rows[2, 30] = 1.0
    rows[3] = -np.inf
    rows[4] = np.nan
    rows[5] = -np.inf
    rows[5, [39, 3]] = 2.0
    rows[6, 5], rows[6, 6] = np.nan, 3.0
    rows[7, 9] = np.inf
    rows[8] = np.finfo(np.float32).min
    rows[9] = np.linspace(-1000, 1000, E)
    _check(rg, rows, 4, mode)


@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (5, 8, 2), (300, 60, 4), (65, 256, 8), (17, 1024, 32)])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("masked", [False, True])
def test_back(rg, T, E, top, mode, masked):
    """Against the formula, and the formula against differences of the definition."""
    rng = np.random.default_rng(T + E)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if masked:
        logits[rng.random((T, E)) < 0.3] = -np.inf
        logits[0] = -np.inf
        logits[T // 2, 0] = np.nan
    ids, _ = oracle.route(logits, top, mode, 1.5)
    dw = rng.standard_normal((T, top)).astype(np.float32)
    dl = torch.full((T, E + 2), 7.0, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_route_back(torch.from_numpy(logits).cuda(), E, T, E, top, mode, 1.5, torch.from_numpy(ids).cuda(),
                              torch.from_numpy(dw).cuda(), dl, E + 2, s))
    assert rg.rg_check(s) == 0
    got = dl.cpu().numpy()
    assert (got[:, E:] == 7.0).all()
    ref = oracle.route_back(logits, ids, mode, 1.5, dw)
    most = np.abs(dw).max()
    assert (np.abs(got[:, :E] - ref) <= (E + 64) * 2.0 ** -24 * 1.5 * 2 * most).all()
    if not masked:
        t, h = T // 2, 1e-5
        for e in (int(ids[t, 0]), 0, E - 1):
            f = []
            for sign in (1, -1):
                z = logits[t].astype(np.float64).copy()
                z[e] += sign * h
                among = ids[t] if mode == 0 else np.arange(E)
                f.append(1.5 * np.dot(np.exp(z[ids[t]]) / np.exp(z[among]).sum(), dw[t]))
            assert abs((f[0] - f[1]) / (2 * h) - ref[t, e]) <= 1e-6 * (1 + most)


def test_back_reports_ids_outside(rg):
    l, dw = torch.zeros(2, 4, device="cuda:0"), torch.ones(2, 2, device="cuda:0")
    ids = torch.tensor([[0, 4], [-1, 3]], dtype=torch.int32, device="cuda:0")
    dl = torch.zeros(2, 4, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_route_back(l, 4, 2, 4, 2, 1, 1.0, ids, dw, dl, 4, s))
    assert rg.rg_check(s) == rg.RG_ERR_INDEX
    ref = oracle.route_back(np.zeros((2, 4)), ids.cpu().numpy(), 1, 1.0, np.ones((2, 2)))
    assert np.allclose(dl.cpu().numpy(), ref, rtol=0, atol=1e-6)


@pytest.mark.parametrize("n,groups", [(0, 3), (1, 1), (31, 5), (1000, 1024), (5000, 1), (70001, 60), (33000, 1023)])
def test_group(rg, n, groups):
    rng = np.random.default_rng(n)
    ids = rng.integers(-1, groups, n).astype(np.int32)
    start = torch.full((groups + 1,), 77, dtype=torch.int32, device="cuda:0")
    order = torch.full((n + 1,), 77, dtype=torch.int32, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_group(torch.from_numpy(ids).cuda(), n, groups, start, order, s))
    assert rg.rg_check(s) == 0
    a, b = oracle.group(ids, groups)
    assert np.array_equal(start.cpu().numpy(), a) and np.array_equal(order.cpu().numpy(), np.append(b, 77))


def test_group_reports_ids_outside(rg):
    ids = torch.tensor([2, 3, -5, 1 << 30, 0], dtype=torch.int32, device="cuda:0")
    start, order = (torch.zeros(n, dtype=torch.int32, device="cuda:0") for n in (4, 5))
    s = torch.cuda.current_stream()
    rg.check(rg.rg_group(ids, 5, 3, start, order, s))
    assert rg.rg_check(s) == rg.RG_ERR_INDEX
    assert start.tolist() == [0, 1, 1, 2] and order.tolist() == [4, 0, 1, 2, 3]


def test_no_tokens(rg):
    """An empty batch leaves an empty plan."""
    start = torch.full((5,), 77, dtype=torch.int32, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_route(None, 4, 0, 4, 2, 0, 1.0, None, None, start, None, s))
    assert rg.rg_check(s) == 0 and start.tolist() == [0] * 5


def test_captured_router(rg):
    rng = np.random.default_rng(3)
    a, b = (rng.standard_normal((50, 16)).astype(np.float32) for _ in range(2))
    l = torch.zeros(50, 16, device="cuda:0")
    ids, order = (torch.zeros(100, dtype=torch.int32, device="cuda:0") for _ in range(2))
    w, start = torch.zeros(100, device="cuda:0"), torch.zeros(17, dtype=torch.int32, device="cuda:0")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rg.check(rg.rg_route(l, 16, 50, 16, 2, 0, 1.0, ids, w, start, order, torch.cuda.current_stream()))
    for x in (a, b):
        l.copy_(torch.from_numpy(x))
        graph.replay()
        torch.cuda.synchronize()
        ref, _ = oracle.route(x, 2, 0, 1.0)
        s, o = oracle.group(ref, 16)
        assert np.array_equal(ids.cpu().numpy().reshape(50, 2), ref)
        assert np.array_equal(start.cpu().numpy(), s) and np.array_equal(order.cpu().numpy(), o)
