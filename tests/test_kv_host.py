"""The paged cache without a GPU: refusals before any CUDA call, sizes, and the
oracle's own pins."""
import ctypes

import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import binding as rg
from quantized_weight_out_gb300 import build as rgbuild
from quantized_weight_out_gb300 import inputs

BAD = 0x1000  # never followed: every case below is refused, or has nothing to do
F16, BF16, F32, Q8, Q4 = inputs.F16, inputs.BF16, inputs.F32, inputs.Q8_0, inputs.Q4_0


@pytest.fixture(scope="module")
def lib():
    rgbuild.build()
    return rg.load()


def _cache(type=Q8, head_dim=128, kv_heads=8, page_tokens=64, pages=10, data=BAD):
    return rg.rg_kv_cache(type, head_dim, kv_heads, page_tokens, pages, data)


def _batch(seqs=2, max_pages=4, max_new=3, tokens=5, new_start=BAD, kv_len=BAD, page_table=BAD):
    return rg.rg_kv_batch(seqs, max_pages, max_new, 0, tokens, new_start, kv_len, page_table)


CACHES = [
    (dict(type=inputs.Q4_K), rg.RG_ERR_TYPE), (dict(type=F32), rg.RG_ERR_TYPE), (dict(type=0), rg.RG_ERR_TYPE),
    (dict(head_dim=96), rg.RG_ERR_SHAPE), (dict(head_dim=0), rg.RG_ERR_SHAPE), (dict(page_tokens=24), rg.RG_ERR_SHAPE),
    (dict(page_tokens=8192), rg.RG_ERR_SHAPE), (dict(page_tokens=0), rg.RG_ERR_ARG), (dict(kv_heads=0), rg.RG_ERR_ARG),
    (dict(kv_heads=5000), rg.RG_ERR_ARG), (dict(pages=-1), rg.RG_ERR_ARG), (dict(pages=1 << 31), rg.RG_ERR_ARG),
    (dict(data=None), rg.RG_ERR_ARG), (dict(data=BAD + 8), rg.RG_ERR_ALIGN),
]
BATCHES = [
    (dict(seqs=-1), rg.RG_ERR_ARG), (dict(max_pages=-1), rg.RG_ERR_ARG), (dict(max_new=-1), rg.RG_ERR_ARG),
    (dict(tokens=-1), rg.RG_ERR_ARG), (dict(tokens=1 << 31), rg.RG_ERR_ARG), (dict(max_pages=1 << 30), rg.RG_ERR_ARG),
    (dict(max_pages=(1 << 24) + 1), rg.RG_ERR_ARG),
    (dict(new_start=None), rg.RG_ERR_ARG), (dict(kv_len=None), rg.RG_ERR_ARG), (dict(page_table=None), rg.RG_ERR_ARG),
    (dict(kv_len=BAD + 2), rg.RG_ERR_ALIGN),
    (dict(seqs=0, new_start=None, kv_len=None, page_table=None), rg.RG_OK), (dict(tokens=0), rg.RG_OK),
    (dict(max_new=0), rg.RG_OK),
]


def _store(call, cache, batch, **kw):
    a = dict(atype=F32, k=BAD, k_t=1024, k_h=128, v=BAD, v_t=1024, v_h=128)
    a.update(kw)
    return call(cache, batch, a["atype"], a["k"], a["k_t"], a["k_h"], a["v"], a["v_t"], a["v_h"])


def _attend(cache, batch, **kw):
    a = dict(atype=BF16, q=BAD, q_t=4096, q_h=128, heads=32, out=BAD, o_t=4096, o_h=128, scale=0.1, window=0)
    a.update(kw)
    return rg.rg_kv_attend(cache, batch, a["atype"], a["q"], a["q_t"], a["q_h"], a["heads"], a["out"], a["o_t"],
                           a["o_h"], a["scale"], a["window"])


@pytest.mark.parametrize("change,status", CACHES)
def test_cache_refusals(lib, change, status):
    c, b = _cache(**change), _batch()
    assert _store(rg.rg_kv_write, c, b) == status
    assert _store(rg.rg_kv_read, c, b) == status
    assert _attend(c, b) == status
    assert rg.rg_kv_attend_workspace_bytes(c, b, 32) == 0


@pytest.mark.parametrize("change,status", BATCHES)
def test_batch_refusals(lib, change, status):
    c, b = _cache(), _batch(**change)
    assert _store(rg.rg_kv_write, c, b) == status
    assert _store(rg.rg_kv_read, c, b) == status
    assert _attend(c, b) == status


@pytest.mark.parametrize("change,status", [
    (dict(atype=Q8), rg.RG_ERR_TYPE), (dict(k=None, v=None), rg.RG_ERR_ARG), (dict(k=BAD + 4), rg.RG_ERR_ALIGN),
    (dict(v=BAD + 8), rg.RG_ERR_ALIGN), (dict(k_t=1022), rg.RG_ERR_ALIGN), (dict(atype=F16, k_t=1028), rg.RG_ERR_ALIGN),
    (dict(k_h=64), rg.RG_ERR_ARG), (dict(v_t=64), rg.RG_ERR_ARG), (dict(v_h=-128), rg.RG_ERR_ARG),
])
def test_store_refusals(lib, change, status):
    for call in (rg.rg_kv_write, rg.rg_kv_read):
        assert _store(call, _cache(), _batch(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(atype=4), rg.RG_ERR_TYPE), (dict(heads=0), rg.RG_ERR_ARG), (dict(heads=31), rg.RG_ERR_SHAPE),
    (dict(heads=8 * 1025), rg.RG_ERR_SHAPE), (dict(window=-1), rg.RG_ERR_ARG), (dict(scale=float("inf")), rg.RG_ERR_ARG),
    (dict(scale=float("nan")), rg.RG_ERR_ARG), (dict(q=None), rg.RG_ERR_ARG), (dict(out=None), rg.RG_ERR_ARG),
    (dict(q=BAD + 2), rg.RG_ERR_ALIGN), (dict(out=BAD + 8), rg.RG_ERR_ALIGN), (dict(o_t=4100), rg.RG_ERR_ALIGN),
    (dict(q_h=64), rg.RG_ERR_ARG), (dict(o_t=-4096), rg.RG_ERR_ARG),
])
def test_attend_refusals(lib, change, status):
    assert _attend(_cache(), _batch(), **change) == status


def test_missing_descriptions(lib):
    assert lib.rg_kv_write(None, ctypes.addressof(_batch()), F32, BAD, 1024, 128, BAD, 1024, 128, None) == rg.RG_ERR_ARG
    assert lib.rg_kv_attend(ctypes.addressof(_cache()), None, F32, BAD, 4096, 128, 32, BAD, 4096, 128, 0.1, 0,
                            None) == rg.RG_ERR_ARG
    c, b = _cache(), _batch()
    assert rg.rg_kv_attend_ws(c, b, F32, BAD, 4096, 128, 32, BAD, 4096, 128, 0.1, 0, None, 0) == rg.RG_ERR_ARG
    assert ctypes.sizeof(rg.rg_kv_cache) == 32 and ctypes.sizeof(rg.rg_kv_batch) == 48
    assert rg.strerror(rg.RG_ERR_INDEX) != "unknown status"


def test_page_bytes(lib):
    for t in (F16, BF16, Q8, Q4):
        for d in (64, 128, 256):
            for h, p in ((1, 16), (8, 64), (5, 4096)):
                assert rg.rg_kv_page_bytes(t, d, h, p) == oracle.kv_page_bytes(t, d, h, p)
    assert rg.rg_kv_page_bytes(Q8, 96, 8, 64) == 0 and rg.rg_kv_page_bytes(inputs.Q6_K, 128, 8, 64) == 0
    assert rg.rg_kv_page_bytes(Q8, 128, 0, 64) == 0 and rg.rg_kv_page_bytes(Q8, 128, 8, 40) == 0


def test_oracle_places_fill_a_granule():
    """Every code and scale has a place of its own, and together they are the granule."""
    for t in (F16, BF16, Q8, Q4):
        for d in (64, 128, 256):
            for kind in (0, 1):
                bits = np.zeros(16 * oracle.kv_row_bytes(t, d) * 2, int)  # by half byte
                for j in range(16):
                    at, half, scale = oracle.kv_places(t, d, kind, j)
                    for a, h in zip(at, half):
                        wide = {F16: 4, BF16: 4, Q8: 2, Q4: 1}[t]
                        bits[2 * a + h:2 * a + h + wide] += 1
                    for a in (scale if scale is not None else ()):
                        bits[2 * a:2 * a + 4] += 1
                assert (bits == 1).all()


def test_oracle_quantises_by_hand():
    x = np.zeros(32, np.float32)
    x[:4] = [12.7, -12.7, 6.35, 0.05]
    codes, d = oracle.kv_quantise(Q8, x)
    assert float(d[0]) == float(np.float16(np.float32(12.7) / np.float32(127)))
    assert list(codes[:4].view(np.int8)) == [127, -127, 64, 0]      # 63.5 and 0.5 to even
    x[:3] = [4.0, -4.0, 1.0]                                         # tie: the first value's sign counts
    codes, d = oracle.kv_quantise(Q4, x)
    assert float(d[0]) == -0.5 and list(codes[:4]) == [0, 15, 6, 8]
    x[0] = np.nan
    assert np.isnan(oracle.kv_values(Q4, x)).all() and np.isnan(oracle.kv_values(Q8, x)).all()
    assert (oracle.kv_values(Q8, np.full(32, 1e-9, np.float32)) == 0).all()


def test_oracle_attention_by_hand():
    """Equal scores average what is visible; a window hides the rest; nothing visible: zeros."""
    V = np.arange(6.0).reshape(6, 1, 1).repeat(64, 2)
    K, q = np.zeros((6, 1, 64)), np.ones((3, 2, 64))
    out, mag = oracle.kv_attend(q, K, V, [-1, 3, 5], 1.0)
    assert (out[0] == 0).all() and np.allclose(out[1], 1.5) and np.allclose(out[2], 2.5) and np.allclose(mag, out)
    out, _ = oracle.kv_attend(q, K, V, [0, 3, 5], 1.0, window=2)
    assert np.allclose(out[:, 0, 0], [0, 2.5, 4.5])
    K[4] = 10.0
    assert np.allclose(oracle.kv_attend(q[:1], K, V, [5], 1.0)[0], 4.0)
