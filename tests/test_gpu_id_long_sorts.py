"""Long sorts of ids on a GB300: slots by group and a table's gradient by token, past the lengths at which a warp's part
is walked twice and a cluster has sixteen blocks."""
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


# A sort has 1 block of 32 warps for up to 2048 ids, 8 up to 16384, then 16: a warp keeps its ids' places in registers
# while it has at most 256 of them (131072 in all).
@pytest.mark.parametrize("n", [2047, 2049, 16384, 16385, 131071, 131072, 131073, 140001, 1000003])
@pytest.mark.parametrize("groups", [8, 1023])
def test_group(rg, n, groups):
    rng = np.random.default_rng(n)
    # (a popular group, padding, and runs of one id)
    ids = np.where(rng.random(n) < 0.3, groups // 2, rng.integers(-1, groups, n)).astype(np.int32)
    ids[n // 3:n // 3 + n // 5] = groups - 1
    start = torch.full((groups + 1,), 77, dtype=torch.int32, device="cuda:0")
    order = torch.full((n + 1,), 77, dtype=torch.int32, device="cuda:0")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_group(torch.from_numpy(ids).cuda(), n, groups, start, order, s))
    assert rg.rg_check(s) == 0
    a, b = oracle.group(ids, groups)
    assert np.array_equal(start.cpu().numpy(), a) and np.array_equal(order.cpu().numpy(), np.append(b, 77))


# tables whose ids take one, two, three and four passes (10 bits of an id at most a pass)
@pytest.mark.parametrize("N", [1000, 32000, (1 << 20) + 7, (1 << 21) + 5])
@pytest.mark.parametrize("n", [2049, 16387, 131075, 300001])
@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_rows_back(rg, N, n, beta):
    """Against a 64-bit sum by token: small ids in long runs, large ones once or twice, padding."""
    K = 8
    rng = np.random.default_rng(N + n)
    ids = np.minimum((N ** rng.random(n)).astype(np.int64) - 1, N - 1)
    ids[rng.random(n) < 0.02] = -1
    ids[0], ids[n - 1] = N - 1, N - 1
    i_d = torch.from_numpy(ids.astype(np.int32)).cuda()
    g = torch.Generator(device="cuda:0").manual_seed(n)
    dY = torch.randn(n, K, generator=g, device="cuda:0")
    G = torch.randn(N, K, generator=g, device="cuda:0") if beta else torch.full((N, K), float("nan"), device="cuda:0")
    real = i_d >= 0
    at = i_d[real].long()
    old = G.double() if beta else torch.zeros(N, K, dtype=torch.float64, device="cuda:0")
    # (the order of a 64-bit sum moves it by far less than the bound)
    ref = old.index_add(0, at, dY[real].double())
    mag = old.abs().index_add(0, at, dY[real].double().abs())
    runs = torch.bincount(at, minlength=N)[:, None].double()
    s = torch.cuda.current_stream()
    size = rg.rg_get_rows_back_workspace_bytes(n, N, K)
    first = None
    for fill in (0xFF, 0x01):
        out = G.clone()
        work = torch.full((size + 256,), fill, dtype=torch.uint8, device="cuda:0")
        rg.check(rg.rg_get_rows_back_ws(2, dY.bfloat16(), K, i_d, 0, 1.0, out, K, N, K, 1.0, work, size, s))  # no ids
        rg.check(rg.rg_get_rows_back_ws(11, dY, K, i_d, n, 1.0, out, K, N, K, beta, work, size, s))
        assert rg.rg_check(s) == 0
        assert bool((work[size:] == fill).all())
        # a piece is summed in order in windows of 32, the windows' sums in order: at most one half step a term
        assert bool(((out.double() - ref).abs() <= (runs + 4) * 2.0 ** -24 * mag * 1.01 + 1e-30).all())
        first = out if first is None else first
        assert torch.equal(out, first)
