"""rg_kv_write and rg_kv_read against the oracle: every byte of the pool."""
import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

from kv_common import RG_BF16, RG_F16, RG_F32, Setup, to_act

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
TYPES = [inputs.F16, inputs.BF16, inputs.Q8_0, inputs.Q4_0]
ACTS = [RG_F32, RG_F16, RG_BF16]


@pytest.fixture(scope="module")
def rg():
    from quantized_weight_out_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def _write(su, k, v, rg, kt=None, kh=None):
    HD = su.H * su.D
    return rg.rg_kv_write(su.cache, su.batch, su.atype, k, HD, su.D, v, HD, su.D, torch.cuda.current_stream())


def _expect(su, k, v):
    """The pool after the write, by the oracle's placement."""
    pool = su.pool.copy()
    for s, (n, L) in enumerate(su.seqs):
        for i, p in enumerate(su.positions(s)):
            if p < 0:
                continue
            page = su.table[s, p // su.P]
            for h in range(su.H):
                for kind, x in ((0, k), (1, v)):
                    oracle.kv_store(pool, su.wtype, su.D, su.H, su.P, page, int(p), kind, h,
                                    x[su.start[s] + i, h])
    return pool


SEQS = [
    [(1, 1)],                                   # the first token of all
    [(1, 16), (1, 17), (1, 33), (1, 5)],        # single tokens at granule ends and starts
    [(40, 40), (3, 50), (0, 20), (17, 18)],     # whole granules, pieces, nothing new
    [(5, 3), (1, 0), (2, 70)],                  # tokens before the cache's start
    [(100, 100)],
]


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("atype", ACTS)
@pytest.mark.parametrize("shape", [(64, 3, 16), (128, 2, 32), (256, 1, 48)])
@pytest.mark.parametrize("case", range(len(SEQS)))
def test_write_every_byte_and_read_back(rg, wtype, atype, shape, case):
    """The pool's bytes after a write are the oracle's, stale ones around the
    new tokens included, and reading gives what the codes stand for."""
    D, H, P = shape
    su = Setup(torch, rg, wtype, D, H, P, SEQS[case], seed=case, atype=atype, fill="random")
    k, v = (to_act(su.rng.standard_normal((su.tokens, H, D)).astype(np.float32) *
                   10.0 ** su.rng.integers(-3, 2, (su.tokens, H, 1)), atype) for _ in range(2))
    rg.check(_write(su, su.tensor(k), su.tensor(v), rg))
    got = su.pool_d.cpu().numpy()
    rg.check(rg.rg_check(torch.cuda.current_stream()))
    want = _expect(su, k, v)
    assert np.array_equal(got, want), int((got != want).sum())
    out = [torch.full((su.tokens, H, D), 7.0, device=su.dev, dtype=su.tensor(k).dtype) for _ in range(2)]
    rg.check(rg.rg_kv_read(su.cache, su.batch, atype, out[0], H * D, D, out[1], H * D, D,
                           torch.cuda.current_stream()))
    rg.check(rg.rg_check(torch.cuda.current_stream()))
    for x, o in zip((k, v), out):
        ref = to_act(oracle.kv_values(wtype, x), atype)
        for s in range(len(su.seqs)):
            ref[su.start[s]:su.start[s + 1]][su.positions(s) < 0] = 0
        assert np.array_equal(o.float().cpu().numpy(), ref)


@pytest.mark.parametrize("wtype", TYPES)
def test_special_values(rg, wtype):
    """Zeros, subnormal blocks, ties of the largest magnitude with both signs,
    exact halves between codes, infinities and NaN; a value beyond fp16 is
    reported (not for a BF16 cache), and the next check is clean."""
    D, H, P = 64, 1, 16
    su = Setup(torch, rg, wtype, D, H, P, [(20, 20)], atype=RG_F32, fill="random")
    k = np.zeros((20, H, D), np.float32)
    k[1] = 1e-9
    k[2, 0, :32] = np.where(np.arange(32) % 3 == 0, -2.0, 2.0)
    k[3, 0, :32] = np.where(np.arange(32) % 3 == 1, -2.0, 2.0)
    k[4, 0, :] = np.arange(64) - 31.5
    k[5, 0, 5] = np.inf
    k[6, 0, 40] = np.nan
    k[7, 0, 0], k[7, 0, 1] = -np.inf, np.nan
    k[8, 0, :32] = np.linspace(-127, 127, 32)
    k[9] = 3e-5
    k[10] = -1e-41
    v = k[::-1].copy()
    rg.check(_write(su, su.tensor(k), su.tensor(v), rg))
    got = su.pool_d.cpu().numpy()
    rg.check(rg.rg_check(torch.cuda.current_stream()))
    out = [torch.empty((20, H, D), device=su.dev) for _ in range(2)]
    rg.check(rg.rg_kv_read(su.cache, su.batch, RG_F32, out[0], D, D, out[1], D, D, torch.cuda.current_stream()))
    for x, o in zip((k, v), out):
        assert np.array_equal(o.cpu().numpy(), oracle.kv_values(wtype, x), equal_nan=True)
    if wtype in (inputs.Q8_0, inputs.Q4_0):
        assert np.array_equal(got, _expect(su, k, v))
    k[0, 0, 3] = 7e4
    rg.check(_write(su, su.tensor(k), su.tensor(v), rg))
    st = rg.rg_check(torch.cuda.current_stream())
    assert st == (rg.RG_OK if wtype == inputs.BF16 else rg.RG_ERR_RANGE)
    assert rg.rg_check(torch.cuda.current_stream()) == rg.RG_OK


@pytest.mark.parametrize("wtype", [inputs.F16, inputs.BF16, inputs.Q8_0, inputs.Q4_0])
def test_the_largest_values(rg, wtype):
    """What is stored without a report is finite as an fp16 operand: in a Q8_0 block of
    65504 d rounds up to 516, and 516 * 127 does not fit."""
    for x, ok in ((65500.0, True), (65502.0, wtype != inputs.Q8_0), (65504.0, wtype != inputs.Q8_0),
                  (-65504.0, wtype != inputs.Q8_0), (65508.0, wtype == inputs.BF16)):
        su = Setup(torch, rg, wtype, 64, 1, 16, [(1, 1)], atype=RG_F32)
        k = np.ones((1, 1, 64), np.float32)
        k[0, 0, 40] = x
        t = su.tensor(k)
        rg.check(_write(su, t, t, rg))
        st = rg.rg_check(torch.cuda.current_stream())
        assert st == (rg.RG_OK if ok else rg.RG_ERR_RANGE), x
        stored = oracle.kv_values(wtype, k)
        if ok and wtype != inputs.BF16:
            with np.errstate(over="ignore"):
                assert np.isfinite(stored.astype(np.float16)).all()


@pytest.mark.parametrize("wtype", [inputs.F16, inputs.Q4_0])
def test_strides_and_one_side_only(rg, wtype):
    """Head-major arrays and parts of a fused row, keys or values alone; the
    gaps of the result arrays keep their contents."""
    D, H, P, seqs = 64, 3, 16, [(21, 30), (2, 2)]
    su = Setup(torch, rg, wtype, D, H, P, seqs, atype=RG_F16, fill="random")
    T = su.tokens
    k, v = (to_act(su.rng.standard_normal((T, H, D)).astype(np.float32), RG_F16) for _ in range(2))
    fused = torch.zeros((T, 5 * D + 2 * H * D), device=su.dev, dtype=torch.float16)
    fused[:, 5 * D:(5 + H) * D] = su.tensor(k).view(T, H * D)
    headed = su.tensor(v).transpose(0, 1).contiguous()          # [H, T, D]
    s = torch.cuda.current_stream()
    rg.check(rg.rg_kv_write(su.cache, su.batch, RG_F16, fused[:, 5 * D:], fused.stride(0), D, None, 0, 0, s))
    half = su.pool_d.cpu().numpy()
    rg.check(rg.rg_kv_write(su.cache, su.batch, RG_F16, None, 0, 0, headed, D, T * D, s))
    rg.check(rg.rg_check(s))
    want = _expect(su, k, v)
    assert np.array_equal(su.pool_d.cpu().numpy(), want)
    keys = su.page_bytes // 2
    assert np.array_equal(half[:, :keys], want[:, :keys]) and np.array_equal(half[:, keys:], su.pool[:, keys:])
    wide = torch.full((T, H, D + 8), 3.0, device=su.dev, dtype=torch.float16)
    rg.check(rg.rg_kv_read(su.cache, su.batch, RG_F16, None, 0, 0, wide, H * (D + 8), D + 8, s))
    ref = oracle.kv_values(wtype, v).astype(np.float16).astype(np.float32)
    got = wide.float().cpu().numpy()
    assert np.array_equal(got[..., :D], ref) and (got[..., D:] == 3).all()


def test_bad_numbers_are_reported_not_followed(rg):
    """Page numbers outside the pool, lengths and rows outside the batch: RG_ERR_INDEX,
    the pool and the other sequences' results as they should be."""
    D, H, P = 64, 2, 16
    seqs = [(4, 20), (2, 10), (3, 40), (1, 6)]
    su = Setup(torch, rg, inputs.Q8_0, D, H, P, seqs, atype=RG_F32, fill="random")
    k, v = (su.rng.standard_normal((su.tokens, H, D)).astype(np.float32) for _ in range(2))
    s = torch.cuda.current_stream()
    want = _expect(su, k, v)
    table = su.table.copy()
    table[0, 1] = su.pages                      # sequence 0's new tokens 16 .. 19
    table[1, 0] = -5
    lens = su.len.copy()
    lens[2] = su.width * P + 1
    su.table_d.copy_(torch.from_numpy(table))
    su.len_d.copy_(torch.from_numpy(lens))
    rg.check(_write(su, su.tensor(k), su.tensor(v), rg))
    assert rg.rg_check(s) == rg.RG_ERR_INDEX and rg.rg_check(s) == rg.RG_OK
    got = su.pool_d.cpu().numpy()
    mine = su.table[3, 0]
    assert np.array_equal(got[mine], want[mine])
    others = [p for p in range(su.pages) if p != mine]
    assert np.array_equal(got[others], su.pool[others])
    out = torch.full((su.tokens, H, D), 9.0, device=su.dev)
    rg.check(rg.rg_kv_read(su.cache, su.batch, RG_F32, out, H * D, D, None, 0, 0, s))
    assert rg.rg_check(s) == rg.RG_ERR_INDEX
    o = out.cpu().numpy()
    assert (o[:6] == 0).all() and (o[6:9] == 9).all()
    assert np.array_equal(o[9:], oracle.kv_values(inputs.Q8_0, k[9:]))


def test_pool_past_four_gigabytes(rg):
    """Pages whose bytes lie past 2^32 from the pool's start."""
    D, H, P = 128, 8, 64
    wtype = inputs.Q8_0
    pb = oracle.kv_page_bytes(wtype, D, H, P)
    pages = (5 << 30) // pb
    pool = torch.zeros(pages * pb, dtype=torch.uint8, device="cuda:0")
    table = torch.tensor([[pages - 1, 3, pages - 7]], dtype=torch.int32, device="cuda:0")
    n = 150
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda:0")
    ln = torch.tensor([n], dtype=torch.int32, device="cuda:0")
    cache, batch = rg.kv_cache(wtype, D, H, P, pages, pool), rg.kv_batch(start, ln, table, n, n)
    x = np.random.default_rng(3).standard_normal((2, n, H, D)).astype(np.float32)
    kd, vd = (torch.from_numpy(a).cuda() for a in x)
    s = torch.cuda.current_stream()
    rg.check(rg.rg_kv_write(cache, batch, RG_F32, kd, H * D, D, vd, H * D, D, s))
    out = torch.empty_like(kd), torch.empty_like(vd)
    rg.check(rg.rg_kv_read(cache, batch, RG_F32, out[0], H * D, D, out[1], H * D, D, s))
    rg.check(rg.rg_check(s))
    for a, o in zip(x, out):
        assert np.array_equal(o.cpu().numpy(), oracle.kv_values(wtype, a))
    assert not pool[4 * pb:(pages - 7) * pb].any()
    q = torch.from_numpy(x[0][-1:, :, :].copy()).cuda()
    o = torch.empty((1, H, D), device="cuda:0")
    b1 = rg.kv_batch(torch.tensor([0, 1], dtype=torch.int32, device="cuda:0"), ln, table, 1, 1)
    rg.check(rg.rg_kv_attend(cache, b1, RG_F32, q, H * D, D, H, o, H * D, D, 0.1, 0, s))
    rg.check(rg.rg_check(s))
    ref, mag = oracle.kv_attend(x[0][-1:], oracle.kv_values(wtype, x[0]), oracle.kv_values(wtype, x[1]), [n - 1], 0.1)
    assert (np.abs(o.cpu().numpy() - ref) <= 2e-2 * mag).all()
