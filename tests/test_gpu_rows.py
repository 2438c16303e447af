"""Table rows by token and their gradient on a GB300 against the definition in 64 bits."""
import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from id_common import BF16, F16, F32, HALF_STEP, SMALLEST, torch_act  # noqa: E402
from kv_common import to_act  # noqa: E402


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


def _get(rg, wtype, W, N, K, ids, scale, atype, pad=0, status=0):
    out = torch.full((len(ids), K + pad), 7.0, dtype=torch_act(torch, atype), device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_get_rows(wtype, torch.from_numpy(np.ascontiguousarray(W).view(np.uint8).reshape(-1)).cuda(), N, K,
                            torch.tensor(ids, dtype=torch.int32, device="cuda:0"), len(ids), scale, atype, out, K + pad,
                            s))
    assert rg.rg_check(s) == status
    got = out.float().cpu().numpy()
    assert (got[:, K:] == 7.0).all()
    return got[:, :K]


@pytest.mark.parametrize("wtype", inputs.ALL_TYPES)
@pytest.mark.parametrize("atype", [F32, F16, BF16])
def test_get_rows(rg, wtype, atype):
    """Every type, several widths, scales, padding ids, the same id twice: the decoded value times the scale, rounded
    once in F32 and once to atype."""
    for N, K, n, scale, pad in [(1, 256, 1, 1.0, 0), (50, 768, 33, 64.0, 8), (301, 2048, 129, 0.3, 0)]:
        W = inputs.gen_weight(wtype, N, K, seed=N, stream=1)
        rng = np.random.default_rng(n)
        ids = rng.integers(0, N, n)
        ids[n // 2:n // 2 + 2] = ids[0]
        if n > 8:
            ids[3] = -1
        got = _get(rg, wtype, W, N, K, ids, scale, atype, pad)
        ref = oracle.get_rows(wtype, W, N, K, ids, scale)
        tol = HALF_STEP[atype] * np.abs(ref) * 1.001 + 2.0 ** -24 * np.abs(ref) + SMALLEST[atype]
        assert (np.abs(got - ref) <= tol).all()
        if n > 8:
            assert (got[3] == 0).all()


def test_get_rows_by_itself_is_dequant(rg):
    """With scale 1 an F32 row is the decoded row, bit for bit."""
    for wtype in inputs.ALL_TYPES:
        W = inputs.gen_weight(wtype, 40, 512, seed=3, stream=1)
        assert np.array_equal(_get(rg, wtype, W, 40, 512, np.arange(40), 1.0, F32), oracle.dequant(wtype, W, 40, 512))


def test_get_rows_past_the_table(rg):
    W = inputs.gen_weight(inputs.Q4_K, 10, 256, seed=3, stream=1)
    got = _get(rg, inputs.Q4_K, W, 10, 256, [9, 10, 1 << 30, -1, -(1 << 31)], 1.0, BF16, status=rg.RG_ERR_INDEX)
    assert (got[1:] == 0).all() and (got[0] != 0).any()


def test_get_rows_far(rg):
    """A row beyond 2^32 bytes, and outputs beyond 2^31 values."""
    N, K = (1 << 20) + 5, 4096
    W = torch.zeros(N * K * 2, dtype=torch.uint8, device="cuda:0")
    last = np.random.default_rng(0).standard_normal(K).astype(np.float16)
    W[(N - 1) * K * 2:] = torch.from_numpy(last.view(np.uint8)).cuda()
    n = (1 << 19) + 3
    ids = torch.zeros(n, dtype=torch.int32, device="cuda:0")
    ids[-1] = N - 1
    out = torch.empty(n, K, dtype=torch.float16, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_get_rows(inputs.F16, W, N, K, ids, n, 1.0, F16, out, K, s))
    assert rg.rg_check(s) == 0
    assert np.array_equal(out[-1].cpu().numpy(), last) and not bool(out[:-1].any())


def _back(rg, atype, dY, ids, scale, G, beta, pad=0, ws=False, status=0):
    n, K = dY.shape
    N = G.shape[0]
    d = torch.full((n, K + pad), 3.0, dtype=torch_act(torch, atype), device="cuda:0")
    d[:, :K] = torch.from_numpy(dY).cuda().to(d.dtype)
    g = torch.full((N, K + pad), 7.0, device="cuda:0")
    g[:, :K] = torch.from_numpy(G).cuda()
    i = torch.tensor(ids, dtype=torch.int32, device="cuda:0")
    s = torch.cuda.current_stream()
    if ws:
        size = rg.rg_get_rows_back_workspace_bytes(n, N, K)
        work = torch.full((size + 256,), ws, dtype=torch.uint8, device="cuda:0")
        rg.check(rg.rg_get_rows_back_ws(atype, d, K + pad, i, n, scale, g, K + pad, N, K, beta, work, size, s))
        assert rg.rg_check(s) == status
        assert bool((work[size:] == ws).all())
    else:
        rg.check(rg.rg_get_rows_back(atype, d, K + pad, i, n, scale, g, K + pad, N, K, beta, s))
        assert rg.rg_check(s) == status
    got = g.cpu().numpy()
    assert (got[:, K:] == 7.0).all()
    return got[:, :K]


@pytest.mark.parametrize("atype", [F32, F16, BF16])
@pytest.mark.parametrize("N,K,n,beta,scale", [
    (1, 8, 1, 0.0, 1.0), (7, 8, 500, 0.0, 0.5), (1000, 264, 63, 1.0, 2.0), (3000, 64, 4097, 0.5, 1.0),
    (5, 1032, 1000, 1.0, -3.0), (70000, 16, 2000, 0.0, 1.0), (1025, 2048, 129, 0.0, 1.0), (2000000, 8, 300, 0.0, 1.0)])
def test_rows_back(rg, atype, N, K, n, beta, scale):
    """Runs of one token to thousands, tables smaller and larger than one digit of the sort, every kind of beta."""
    rng = np.random.default_rng(N + n)
    ids = np.minimum((N ** rng.random(n)).astype(np.int64) - 1, N - 1)
    ids[rng.random(n) < 0.05] = -1
    dY = to_act((rng.standard_normal((n, K)) * 1e-3).astype(np.float32), atype)
    G = rng.standard_normal((N, K)).astype(np.float32) if beta else np.full((N, K), np.nan, np.float32)
    ref, mag = oracle.get_rows_back(dY, ids, scale, G, beta)
    runs = np.bincount(ids[ids >= 0], minlength=N)[:, None] if (ids >= 0).any() else np.zeros((N, 1))
    got = _back(rg, atype, dY, ids, scale, G, beta, pad=8)
    assert (np.abs(got - ref) <= (runs + 4) * 2.0 ** -24 * mag * 1.01 + 1e-30).all()
    if beta == 1.0:
        assert np.array_equal(got[runs[:, 0] == 0], G[runs[:, 0] == 0])
    # the same bits, whatever the workspace holds
    for fill in (0xFF, 0x01):
        assert np.array_equal(_back(rg, atype, dY, ids, scale, G, beta, pad=8, ws=fill), got)


def test_rows_back_ids_outside(rg):
    rng = np.random.default_rng(0)
    dY = rng.standard_normal((6, 16)).astype(np.float32)
    ids = [2, 5, 6, -1, 1 << 30, 2]
    got = _back(rg, F32, dY, ids, 1.0, np.zeros((6, 16), np.float32), 0.0, status=rg.RG_ERR_INDEX)
    ref, _ = oracle.get_rows_back(dY, ids, 1.0, np.zeros((6, 16), np.float32), 0.0)
    assert np.allclose(got, ref, rtol=0, atol=1e-6)


def test_rows_back_of_nothing(rg):
    G = np.random.default_rng(0).standard_normal((20, 16)).astype(np.float32)
    none = np.zeros((0, 16), np.float32)
    assert np.array_equal(_back(rg, F32, none, [], 1.0, G, 1.0), G)
    assert (_back(rg, F32, none, [], 1.0, G, 0.0) == 0).all()
    assert np.array_equal(_back(rg, F32, none, [], 1.0, G, 0.5), G * np.float32(0.5))
    assert np.array_equal(_back(rg, F32, np.ones((3, 16), np.float32), [-1] * 3, 1.0, G, 1.0), G)


def test_lookup_and_its_gradient_together(rg):
    """A table's forward and gradient agree: the sum of dY * out is the sum of table * G (both linear in the table)."""
    rng = np.random.default_rng(4)
    N, K, n = 300, 64, 777
    table = rng.standard_normal((N, K)).astype(np.float32)
    ids = rng.integers(-1, N, n)
    dY = rng.standard_normal((n, K)).astype(np.float32)
    out = _get(rg, F32, table, N, K, ids, 0.25, F32).astype(np.float64)
    G = _back(rg, F32, dY, ids, 0.25, np.zeros((N, K), np.float32), 0.0).astype(np.float64)
    a, b = (dY * out).sum(), (table * G).sum()
    assert abs(a - b) <= 16 * 2.0 ** -24 * np.abs(dY * out).sum()


def test_rows_back_captured(rg):
    """One graph serves other tokens and gradients."""
    rng = np.random.default_rng(6)
    N, K, n = 500, 72, 333
    dY = [rng.standard_normal((n, K)).astype(np.float32) for _ in range(2)]
    ids = [rng.integers(0, 1 + 40 * i, n) for i in range(2)]
    want = [_back(rg, F32, d, i, 1.0, np.zeros((N, K), np.float32), 0.0) for d, i in zip(dY, ids)]
    d_d, i_d = torch.zeros(n, K, device="cuda:0"), torch.zeros(n, dtype=torch.int32, device="cuda:0")
    g_d = torch.zeros(N, K, device="cuda:0")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rg.check(rg.rg_get_rows_back(F32, d_d, K, i_d, n, 1.0, g_d, K, N, K, 0.0, torch.cuda.current_stream()))
    for d, i, w in zip(dY, ids, want):
        d_d.copy_(torch.from_numpy(d))
        i_d.copy_(torch.from_numpy(i.astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(g_d.cpu().numpy(), w)
