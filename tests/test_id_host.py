"""The indexed calls without a GPU: refusals before any CUDA call, what has nothing to do, sizes, and the oracle's pins."""
import ctypes

import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import binding as rg
from quantized_weight_out_gb300 import build as rgbuild
from quantized_weight_out_gb300 import inputs

BAD = 0x1000  # never followed: every case below is refused, or has nothing to do
F32, F16, BF16, Q8 = inputs.F32, inputs.F16, inputs.BF16, inputs.Q8_0


@pytest.fixture(scope="module")
def lib():
    rgbuild.build()
    return rg.load()


ROWS = dict(wtype=Q8, W=BAD, N=10, K=256, ids=BAD, n=3, scale=1.0, atype=BF16, out=BAD, out_row=256)


@pytest.mark.parametrize("change,status", [
    (dict(wtype=0), rg.RG_ERR_TYPE), (dict(wtype=16), rg.RG_ERR_TYPE), (dict(atype=Q8), rg.RG_ERR_TYPE),
    (dict(K=200), rg.RG_ERR_SHAPE), (dict(wtype=F16, K=12), rg.RG_ERR_SHAPE), (dict(N=-1), rg.RG_ERR_ARG),
    (dict(n=-1), rg.RG_ERR_ARG), (dict(n=1 << 31), rg.RG_ERR_ARG), (dict(W=None), rg.RG_ERR_ARG),
    (dict(ids=None), rg.RG_ERR_ARG), (dict(out=None), rg.RG_ERR_ARG), (dict(out_row=248), rg.RG_ERR_ARG),
    (dict(out_row=260), rg.RG_ERR_ALIGN), (dict(atype=F32, out_row=258), rg.RG_ERR_ALIGN),
    (dict(W=BAD + 8), rg.RG_ERR_ALIGN), (dict(ids=BAD + 2), rg.RG_ERR_ALIGN), (dict(out=BAD + 8), rg.RG_ERR_ALIGN),
    (dict(K=(1 << 30) + 256, out_row=1 << 31), rg.RG_ERR_ARG),
    (dict(n=0, W=None, ids=None, out=None), rg.RG_OK), (dict(K=0, W=None, out=None), rg.RG_OK),
])
def test_get_rows_refusals(lib, change, status):
    assert rg.rg_get_rows(*dict(ROWS, **change).values()) == status


BACK = dict(atype=BF16, dY=BAD, dy_row=64, ids=BAD, n=3, scale=1.0, G=BAD, g_row=64, N=10, K=64, beta=0.0)


@pytest.mark.parametrize("change,status", [
    (dict(atype=0), rg.RG_ERR_TYPE), (dict(K=60), rg.RG_ERR_SHAPE), (dict(N=-1), rg.RG_ERR_ARG),
    (dict(n=-1), rg.RG_ERR_ARG), (dict(K=1 << 31), rg.RG_ERR_ARG), (dict(G=None), rg.RG_ERR_ARG),
    (dict(dY=None), rg.RG_ERR_ARG), (dict(ids=None), rg.RG_ERR_ARG), (dict(dy_row=56), rg.RG_ERR_ARG),
    (dict(g_row=56), rg.RG_ERR_ARG), (dict(dy_row=68), rg.RG_ERR_ALIGN), (dict(g_row=66), rg.RG_ERR_ALIGN),
    (dict(G=BAD + 4), rg.RG_ERR_ALIGN), (dict(dY=BAD + 8), rg.RG_ERR_ALIGN), (dict(ids=BAD + 1), rg.RG_ERR_ALIGN),
    (dict(K=65535 * 1024 + 8, dy_row=1 << 28, g_row=1 << 28), rg.RG_ERR_ARG),
    (dict(N=0, G=None, dY=None), rg.RG_OK), (dict(K=0, G=None, dY=None), rg.RG_OK),
])
def test_rows_back_refusals(lib, change, status):
    args = list(dict(BACK, **change).values())
    assert rg.rg_get_rows_back(*args) == status
    assert rg.rg_get_rows_back_ws(*args, BAD, 1 << 40) == status


def test_rows_back_workspace(lib):
    assert rg.rg_get_rows_back_workspace_bytes(0, 10, 64) == 0
    assert rg.rg_get_rows_back_workspace_bytes(3, 10, 60) == 0
    assert rg.rg_get_rows_back_workspace_bytes(3, 10, 1 << 31) == 0
    # order, the sorted ids, the rows' first places and one window's sums
    assert rg.rg_get_rows_back_workspace_bytes(3, 10, 64) >= 3 * 8 + 10 * 4 + 64 * 4


ROUTE = dict(logits=BAD, l_row=8, T=4, experts=8, top=2, mode=0, scale=1.0)


@pytest.mark.parametrize("change,status", [
    (dict(mode=2), rg.RG_ERR_TYPE), (dict(mode=-1), rg.RG_ERR_TYPE), (dict(T=-1), rg.RG_ERR_ARG),
    (dict(T=1 << 31), rg.RG_ERR_ARG), (dict(T=1 << 30), rg.RG_ERR_ARG), (dict(experts=0), rg.RG_ERR_ARG),
    (dict(experts=1025, l_row=1025), rg.RG_ERR_SHAPE), (dict(top=0), rg.RG_ERR_ARG), (dict(top=9), rg.RG_ERR_SHAPE),
    (dict(experts=64, l_row=64, top=33), rg.RG_ERR_SHAPE), (dict(l_row=7), rg.RG_ERR_ARG),
    (dict(logits=None), rg.RG_ERR_ARG), (dict(logits=BAD + 2), rg.RG_ERR_ALIGN), (dict(scale=float("nan")), rg.RG_ERR_ARG),
    (dict(scale=float("inf")), rg.RG_ERR_ARG),
])
def test_route_refusals(lib, change, status):
    args = list(dict(ROUTE, **change).values())
    assert rg.rg_route(*args, BAD, BAD, BAD, BAD) == status
    assert rg.rg_route_back(*args, BAD, BAD, BAD, 2000) == status


def test_route_outputs(lib):
    a = list(ROUTE.values())
    assert rg.rg_route(*a, None, BAD, BAD, BAD) == rg.RG_ERR_ARG
    assert rg.rg_route(*a, BAD, None, BAD, BAD) == rg.RG_ERR_ARG
    assert rg.rg_route(*a, BAD, BAD, BAD, None) == rg.RG_ERR_ARG   # both of the plan's arrays, or neither
    assert rg.rg_route(*a, BAD, BAD, None, BAD) == rg.RG_ERR_ARG
    assert rg.rg_route(*a, BAD + 2, BAD, BAD, BAD) == rg.RG_ERR_ALIGN
    assert rg.rg_route(None, 8, 0, 8, 2, 0, 1.0, None, None, None, None) == rg.RG_OK
    assert rg.rg_route_back(*a, BAD, BAD, BAD, 7) == rg.RG_ERR_ARG
    assert rg.rg_route_back(*a, BAD, None, BAD, 8) == rg.RG_ERR_ARG
    assert rg.rg_route_back(None, 8, 0, 8, 2, 0, 1.0, None, None, None, 0) == rg.RG_OK


def test_group_refusals(lib):
    assert rg.rg_group(BAD, -1, 4, BAD, BAD) == rg.RG_ERR_ARG
    assert rg.rg_group(BAD, 5, 0, BAD, BAD) == rg.RG_ERR_ARG
    assert rg.rg_group(BAD, 5, 1025, BAD, BAD) == rg.RG_ERR_SHAPE
    assert rg.rg_group(None, 5, 4, BAD, BAD) == rg.RG_ERR_ARG
    assert rg.rg_group(BAD, 5, 4, None, BAD) == rg.RG_ERR_ARG
    assert rg.rg_group(BAD, 5, 4, BAD, None) == rg.RG_ERR_ARG
    assert rg.rg_group(BAD + 2, 5, 4, BAD, BAD) == rg.RG_ERR_ALIGN


BATCH = dict(experts=4, per_token=2, slots=6, start=BAD, order=BAD)
BATCHES = [
    (dict(experts=-1), rg.RG_ERR_ARG), (dict(experts=1025), rg.RG_ERR_SHAPE), (dict(per_token=0), rg.RG_ERR_ARG),
    (dict(per_token=4), rg.RG_ERR_SHAPE), (dict(slots=-2), rg.RG_ERR_ARG), (dict(slots=1 << 31), rg.RG_ERR_ARG),
    (dict(start=None), rg.RG_ERR_ARG), (dict(order=None), rg.RG_ERR_ARG), (dict(start=BAD + 2), rg.RG_ERR_ALIGN),
    (dict(order=BAD + 2), rg.RG_ERR_ALIGN), (dict(experts=0), rg.RG_ERR_SHAPE), (dict(slots=0, start=None), rg.RG_OK),
]
CALLS = [
    (dict(wtype=0), rg.RG_ERR_TYPE), (dict(wtype=99), rg.RG_ERR_TYPE), (dict(atype=Q8), rg.RG_ERR_TYPE),
    (dict(N=-8), rg.RG_ERR_ARG), (dict(N=1 << 31), rg.RG_ERR_ARG), (dict(N=60), rg.RG_ERR_SHAPE),
    (dict(K=200), rg.RG_ERR_SHAPE), (dict(wtype=F16, K=12), rg.RG_ERR_SHAPE), (dict(W=None), rg.RG_ERR_ARG),
    (dict(W=BAD + 8), rg.RG_ERR_ALIGN), (dict(x=None), rg.RG_ERR_ARG), (dict(x=BAD + 8), rg.RG_ERR_ALIGN),
    (dict(x_row=56), rg.RG_ERR_ARG), (dict(x_row=1004), rg.RG_ERR_ALIGN), (dict(x_of=2), rg.RG_ERR_ARG),
    (dict(y=None), rg.RG_ERR_ARG), (dict(y=BAD + 4), rg.RG_ERR_ALIGN), (dict(y_row=56), rg.RG_ERR_ARG),
    (dict(y_row=1004), rg.RG_ERR_ALIGN), (dict(y_of=-1), rg.RG_ERR_ARG), (dict(weights=BAD + 2), rg.RG_ERR_ALIGN),
    (dict(N=(1 << 30) + 8), rg.RG_ERR_ARG), (dict(K=(1 << 30) + 256), rg.RG_ERR_ARG),
]
CALL = dict(wtype=Q8, W=BAD, N=64, K=256, batch=None, atype=BF16, x=BAD, x_row=256, x_of=0, y=BAD, y_row=256, y_of=0,
            weights=None, beta=0.0)


def _calls(lib, batch, change, status):
    b = rg.rg_id_batch(*dict(BATCH, **batch).values())
    args = list(dict(CALL, batch=b, **change).values())
    assert rg.rg_mul_mat_id(*args) == status
    assert rg.rg_out_prod_id(*args) == status
    assert rg.rg_mul_mat_id_ws(*args, BAD, 1 << 40) == status
    assert rg.rg_out_prod_id_ws(*args, BAD, 1 << 40) == status


@pytest.mark.parametrize("batch,status", BATCHES)
def test_product_batch_refusals(lib, batch, status):
    _calls(lib, batch, {}, status)


@pytest.mark.parametrize("change,status", CALLS)
def test_product_refusals(lib, change, status):
    _calls(lib, {}, change, status)


def test_the_plain_routes_widest_rows(lib):
    b = rg.rg_id_batch(*BATCH.values())
    wide = 65535 * 64 + 8
    a = dict(CALL, batch=b, wtype=F32, N=wide, K=8, x_row=wide, y_row=wide)
    assert rg.rg_mul_mat_id(*a.values()) == rg.RG_ERR_ARG
    a = dict(CALL, batch=b, wtype=F32, N=8, K=wide, x_row=wide, y_row=wide)
    assert rg.rg_out_prod_id(*a.values()) == rg.RG_ERR_ARG


def test_product_without_a_batch(lib):
    args = list(CALL.values())
    assert rg.rg_mul_mat_id(*args) == rg.RG_ERR_ARG
    assert rg.rg_out_prod_id(*args) == rg.RG_ERR_ARG
    assert rg.rg_mul_mat_id_workspace_bytes(Q8, 64, 256, None, 0) == 0


def test_product_workspace(lib):
    """The queries need no device; refused and empty calls need no memory."""
    b = rg.rg_id_batch(4, 2, 600, BAD, BAD)
    for query in (rg.rg_mul_mat_id_workspace_bytes, rg.rg_out_prod_id_workspace_bytes):
        by_slot, by_token = (query(Q8, 64, 256, b, of) for of in (0, 1))
        assert by_token >= by_slot + 600 * 4 * 64 > 0
        assert query(0, 64, 256, b, 0) == 0 and query(Q8, 60, 256, b, 0) == 0 and query(Q8, 64, 256, b, 2) == 0
        assert query(Q8, 64, 256, rg.rg_id_batch(4, 2, 0, BAD, BAD), 0) == 0
        # rows of 210 bytes get a copy with rows of 224; no stack has 2^46 bytes
        assert query(inputs.Q6_K, 64, 256, b, 0) >= query(Q8, 64, 256, b, 0) + 4 * 64 * 224
        assert query(inputs.Q6_K, 1 << 30, 1 << 20, b, 0) == 0
    assert ctypes.sizeof(rg.rg_id_batch) == 32


def test_the_oracles_router():
    """Choices, ties and weights by hand."""
    l = np.array([[1.0, 3.0, 3.0, 2.0], [-np.inf, 0.0, np.nan, -np.inf]], np.float32)
    ids, w = oracle.route(l, 2, oracle.ROUTE_TOP, 1.0)
    assert ids.tolist() == [[1, 2], [1, -1]] and np.allclose(w, [[0.5, 0.5], [1.0, 0.0]])
    start, order = oracle.group(ids, 4)
    assert start.tolist() == [0, 0, 2, 3, 3] and order.tolist() == [0, 2, 1, 3]
    _, w = oracle.route(l, 2, oracle.ROUTE_ALL, 2.0)
    assert np.isclose(w[0, 0], 2 * np.exp(3) / (np.exp(1) + 2 * np.exp(3) + np.exp(2)))


def test_the_oracles_router_gradient():
    """The formula against differences of the definition."""
    rng = np.random.default_rng(0)
    l = rng.standard_normal((3, 7))
    dw = rng.standard_normal((3, 2))
    for mode in (oracle.ROUTE_TOP, oracle.ROUTE_ALL):
        ids, _ = oracle.route(l, 2, mode, 1.0)
        g = oracle.route_back(l, ids, mode, 1.0, dw)
        for t in range(3):
            for e in range(7):
                d = []
                for s in (1e-6, -1e-6):
                    z = l.copy()
                    z[t, e] += s
                    d.append((oracle.route(z, 2, mode, 1.0)[1] * dw).sum())
                assert abs((d[0] - d[1]) / 2e-6 - g[t, e]) < 1e-7


def test_the_oracles_products_are_transposes():
    rng = np.random.default_rng(0)
    W = inputs.gen_weight(Q8, 3 * 16, 256, seed=0, stream=1)
    ids = np.array([2, 0, -1, 2, 1, 0])
    x, up = rng.standard_normal((3, 256)), rng.standard_normal((6, 16))
    y, _ = oracle.product_id(True, Q8, W, 3, 16, 256, ids, 2, x, True, None)
    d, _ = oracle.product_id(False, Q8, W, 3, 16, 256, ids, 2, up, False, None)
    assert np.isclose((y * up).sum(), (x * d.reshape(3, 2, 256).sum(1)).sum())
    assert (y[2] == 0).all()
