"""Experts' products by slot on a GB300 against the definition in 64 bits."""
import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from id_common import BF16, F16, F32, SLOT, TOKEN, Stack, product_tolerance  # noqa: E402

TYPES = inputs.ALL_TYPES


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


def _ids(rng, tokens, top, experts, pad=0.0):
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(tokens)])
    ids[rng.random(tokens) < pad] = -1
    return ids.reshape(-1)


def test_smallest(rg):
    """One slot, one expert, one block of weights."""
    s = Stack(torch, rg, inputs.Q8_0, 1, 8, 256, [0], 1)
    s.check(True, F32, SLOT, SLOT)
    s.check(False, F32, SLOT, SLOT)


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("fwd", [True, False])
def test_types(rg, wtype, fwd):
    """Every weight type, rows of 16-byte multiples and (where the type has them) others, few slots an expert and many."""
    rng = np.random.default_rng(wtype)
    for K, tokens in ((2048, 3), (2048, 10), (2048, 14), (2048, 70), (2048, 400), (768, 10), (768, 300)):
        s = Stack(torch, rg, wtype, 5, 136, K, _ids(rng, tokens, 3, 5, 0.1), 3, seed=K)
        s.check(fwd, BF16, TOKEN, SLOT)


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("x_of,out_of", [(SLOT, SLOT), (TOKEN, TOKEN)])
def test_fewest(rg, wtype, x_of, out_of):
    """Fewer slots than experts, apart or all of one expert: the form of the fewest, whatever the type."""
    for ids, per in (([30, 2], 2), ([7] * 22, 1), ([0, 31, 0, 4, -1, 0, 31, 5, 0, 6, 0, 0, 0, 0, 0, 0], 2)):
        s = Stack(torch, rg, wtype, 32, 72, 2048, ids, per)
        s.check(True, BF16, x_of, out_of, weigh=out_of == TOKEN, beta=0.5, pad=8)


@pytest.mark.parametrize("wtype", [inputs.Q4_K, inputs.Q6_K, inputs.BF16, inputs.MXFP4])
@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("atype", [F32, F16, BF16])
@pytest.mark.parametrize("x_of,out_of", [(SLOT, SLOT), (TOKEN, SLOT), (SLOT, TOKEN), (TOKEN, TOKEN)])
def test_forms(rg, wtype, fwd, atype, x_of, out_of):
    """Whose rows go in and come out, weights, beta, padded rows, a caller's workspace; few slots an expert, tiles of
    single CTAs and of pairs."""
    rng = np.random.default_rng(7)
    one = Stack(torch, rg, wtype, 4, 264, 2048, _ids(rng, 6, 2, 4, 0.2), 2)
    one.check(fwd, atype, x_of, out_of, weigh=True, beta=-1.5, pad=8, ws=True)
    few = Stack(torch, rg, wtype, 4, 264, 2048, _ids(rng, 37, 2, 4, 0.2), 2)
    few.check(fwd, atype, x_of, out_of, weigh=True, beta=0.5, pad=16, ws=True)
    many = Stack(torch, rg, wtype, 3, 264, 2048, _ids(rng, 301, 2, 3, 0.05), 2)
    many.check(fwd, atype, x_of, out_of, weigh=False, pad=8)


@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("counts", [
    [0, 300, 0, 1], [128, 128, 256, 0], [127, 129, 255, 257], [0, 0, 0, 512], [1, 1, 1, 1], [513, 0, 31, 33],
    [0, 0, 20, 0], [0, 32, 0, 0], [8, 9, 7, 1], [16, 1, 0, 15]])
def test_ragged(rg, fwd, counts):
    """Groups that fill tiles exactly, miss by one, or are empty."""
    ids = np.repeat(np.arange(len(counts)), counts)
    ids = np.random.default_rng(3).permutation(ids)
    Stack(torch, rg, inputs.Q4_0, len(counts), 392, 512, ids, 1).check(fwd, BF16, SLOT, SLOT)


@pytest.mark.parametrize("fwd", [True, False])
def test_nobody_routed(rg, fwd):
    """Every slot without an expert: rows by slot stay, rows by token become beta times themselves."""
    s = Stack(torch, rg, inputs.Q8_0, 4, 64, 256, [-1] * 10, 2)
    s.check(fwd, BF16, SLOT, SLOT, beta=0.5)
    s.check(fwd, BF16, SLOT, TOKEN, beta=0.5)
    s.check(fwd, BF16, SLOT, TOKEN)


@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("scale", [1e-30, 1e-9, 1e4, 1e30])
def test_magnitudes(rg, fwd, scale):
    """Rows of any magnitude keep the operands' 11 bits, in every route."""
    rng = np.random.default_rng(1)
    for tokens in (3, 300):
        Stack(torch, rg, inputs.Q8_0, 4, 128, 512, _ids(rng, tokens, 2, 4), 2).check(fwd, F32, TOKEN, SLOT, scale=scale)


@pytest.mark.parametrize("tokens", [3, 200])
@pytest.mark.parametrize("fwd", [True, False])
def test_infinities_stay_in_their_rows(rg, tokens, fwd):
    """An infinity or NaN in one slot's row reaches that slot's result and no other."""
    rng = np.random.default_rng(2)
    s = Stack(torch, rg, inputs.Q8_0, 3, 72, 256, _ids(rng, tokens, 2, 3), 2)
    wide = 256 if fwd else 72
    x = s.act(s.slots, wide, BF16)
    clean = s.run(fwd, BF16, x, SLOT, SLOT)
    x[1, 5], x[4, 0] = np.inf, np.nan
    got = s.run(fwd, BF16, x, SLOT, SLOT)
    assert np.isnan(got[4]).all() and not np.isfinite(got[1]).any()
    keep = np.ones(s.slots, bool)
    keep[[1, 4]] = False
    assert np.array_equal(got[keep], clean[keep])


@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("tokens", [2, 150])
def test_same_bits_and_graphs(rg, fwd, tokens):
    """The same bits every time; a captured call serves other slots and values, beside one on another stream."""
    rng = np.random.default_rng(5)
    a, b = (_ids(rng, tokens, 2, 6, 0.1) for _ in range(2))
    s, s2 = (Stack(torch, rg, inputs.Q4_K, 6, 256, 512, i, 2, seed=9) for i in (a, b))
    wide, width = (512, 256) if fwd else (256, 512)
    xs = [s.act(tokens, wide, BF16) for _ in range(2)]
    want = [z.run(fwd, BF16, x, TOKEN, TOKEN) for z, x in zip((s, s2), xs)]
    assert np.array_equal(want[0], s.run(fwd, BF16, xs[0], TOKEN, TOKEN))
    x_d = s.put(xs[0], BF16)
    out = s.put(np.zeros((tokens, width)), BF16)
    call = rg.rg_mul_mat_id if fwd else rg.rg_out_prod_id
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rg.check(call(s.wtype, s.W_d, s.N, s.K, s.batch, BF16, x_d, wide, TOKEN, out, width, TOKEN, None, 0.0,
                      torch.cuda.current_stream()))
    for z, x, w in 4 * list(zip((s, s2), xs, want)):
        s.start_d.copy_(torch.from_numpy(z.start))
        s.order_d.copy_(torch.from_numpy(z.order))
        x_d.copy_(s.put(x, BF16))
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            graph.replay()
        beside = s2.run(fwd, BF16, xs[1], TOKEN, TOKEN)
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().numpy(), w)
        assert np.array_equal(beside, want[1])


@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("wtype", [inputs.Q8_0, inputs.BF16])
def test_long_rows(rg, fwd, wtype):
    """Input rows longer than a warp's share of the copy, many slots and few."""
    rng = np.random.default_rng(6)
    for tokens in (5, 90):
        N, K = (72, 17 * 256) if fwd else (4488, 256)
        Stack(torch, rg, wtype, 2, N, K, _ids(rng, tokens, 2, 2, 0.1), 2).check(fwd, BF16, TOKEN, SLOT, scale=1e-3)


@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("wtype", [inputs.Q4_K, inputs.Q8_0, inputs.MXFP4])
def test_long_pipelines_same_bits(rg, wtype, fwd):
    """Several items a unit of a hundred and more stages each, over and over: the copies' order of arrival changes, the
    result does not (and is right)."""
    rng = np.random.default_rng(13)
    N, K = (512, 6656) if fwd else (6952, 512)
    s = Stack(torch, rg, wtype, 16, N, K, _ids(rng, 2300, 5, 16, 0.01), 5, W=_tiled(wtype, 16, N, K))
    x = s.act(s.slots, K if fwd else N, BF16, 0.1)
    x_d = s.put(x, BF16)
    out = torch.zeros(s.slots, N if fwd else K, dtype=torch.bfloat16, device=s.dev)
    call, st = (rg.rg_mul_mat_id if fwd else rg.rg_out_prod_id), torch.cuda.current_stream()
    first = None
    for _ in range(60):
        rg.check(call(wtype, s.W_d, N, K, s.batch, BF16, x_d, x.shape[1], SLOT, out, out.shape[1], SLOT, None, 0.0, st))
        first = out.clone() if first is None else first
        assert torch.equal(out, first)
    assert rg.rg_check(st) == 0
    some = rng.choice(np.nonzero(s.ids >= 0)[0], 40, replace=False)
    few = np.full(s.slots, -1)
    few[some] = s.ids[some]
    ref, mag = oracle.product_id(fwd, wtype, s.W, 16, N, K, few, 5, x, False, None)
    tol = product_tolerance(wtype, K, x.shape[1], BF16, mag[some], ref[some])
    assert (np.abs(first.float().cpu().numpy()[some] - ref[some]) <= tol).all()


def _tiled(wtype, experts, N, K):
    """A stack from a few generated rows, each expert's in an order of its own."""
    rows = inputs.gen_weight(wtype, 64, K, seed=3, stream=1)
    rows = np.ascontiguousarray(rows).view(np.uint8).reshape(64, -1)
    pick = np.random.default_rng(5).integers(0, 64, experts * N)
    return rows[pick].reshape(-1)


def test_bad_indices(rg):
    """Ranges and slots outside the batch are reported and count as none; nothing else is touched."""
    ids = np.array([0, 1, 2, 1, 0, 2], np.int32)
    for fwd in (True, False):
        for spoil in ("order", "range", "long", "overlap"):
            s = Stack(torch, rg, inputs.Q8_0, 3, 64, 256, ids, 1)
            x = s.act(6, 256 if fwd else 64, BF16)
            good = s.run(fwd, BF16, x, SLOT, SLOT)
            if spoil == "order":
                s.order_d[0], s.order_d[3] = 99, -5
                lost = [s.order[0], s.order[3]]
            elif spoil == "range":
                s.start_d[1] = -7   # the ranges of experts 0 and 1 are none
                lost = [0, 4, 1, 3]
            elif spoil == "long":
                s.start_d[3] = 1 << 30
                lost = [2, 5]
            else:
                s.start_d.copy_(torch.tensor([0, 6, 0, 6], dtype=torch.int32))
                lost = list(range(6))
            out = s.put(np.full(good.shape, np.nan), BF16)
            x_d = s.put(x, BF16)
            st = torch.cuda.current_stream()
            call = rg.rg_mul_mat_id if fwd else rg.rg_out_prod_id
            rg.check(call(s.wtype, s.W_d, 64, 256, s.batch, BF16, x_d, x.shape[1], SLOT, out, good.shape[1], SLOT, None,
                          0.0, st))
            assert rg.rg_check(st) == rg.RG_ERR_INDEX
            got = out.float().cpu().numpy()
            keep = [i for i in range(6) if i not in lost]
            assert np.array_equal(got[keep], good[keep])
            if spoil != "overlap":
                assert np.isnan(got[lost]).all()


@pytest.mark.parametrize("wtype", [inputs.Q6_K, inputs.Q3_K, inputs.Q2_K, inputs.MXFP4])
@pytest.mark.parametrize("K", [256, 768, 1280, 1536])
@pytest.mark.parametrize("fwd", [True, False])
def test_rows_off_sixteen_bytes(rg, wtype, K, fwd):
    """Rows of W that are not multiples of 16 bytes, at every phase of them: one row block and several, few slots,
    tiles and pairs, experts without slots, a caller's workspace."""
    rng = np.random.default_rng(K)
    for N, tokens in ((8, 2), (104, 3), (72, 40), (264, 330)):
        ids = _ids(rng, tokens, 2, 5, 0.1)
        ids[ids == 3] = -1
        Stack(torch, rg, wtype, 5, N, K, ids, 2, seed=N).check(fwd, BF16, TOKEN, SLOT, ws=tokens != 3)


def test_far_expert(rg):
    """The last of a stack of more than 2^32 bytes."""
    E, N, K = 66, 8192, 4096
    need = E * N * K * 2
    assert need > 1 << 32
    W = torch.zeros(need, dtype=torch.uint8, device="cuda:0")
    last = inputs.gen_weight(inputs.BF16, N, K, seed=4, stream=1)
    W[(E - 1) * N * K * 2:] = torch.from_numpy(np.ascontiguousarray(last).view(np.uint8).reshape(-1)).to("cuda:0")
    for fwd, slots in ((True, 3), (True, 70), (False, 3)):  # slots streamed past W, and tiles of them
        s = Stack(torch, rg, inputs.BF16, 1, N, K, [0] * slots, 1, W=last)
        wide = K if fwd else N
        x = s.act(slots, wide, BF16)
        ref, mag = oracle.product_id(fwd, inputs.BF16, last, 1, N, K, s.ids, 1, x, False, None)
        start = torch.tensor([0] * E + [slots], dtype=torch.int32, device="cuda:0")
        batch = rg.id_batch(E, 1, start, s.order_d)
        out = s.put(np.full(ref.shape, np.nan), BF16)
        st = torch.cuda.current_stream()
        call = rg.rg_mul_mat_id if fwd else rg.rg_out_prod_id
        rg.check(call(inputs.BF16, W, N, K, batch, BF16, s.put(x, BF16), x.shape[1], SLOT, out, ref.shape[1], SLOT, None,
                      0.0, st))
        assert rg.rg_check(st) == 0
        err = np.abs(out.float().cpu().numpy() - ref)
        assert (err <= product_tolerance(inputs.BF16, K, wide, BF16, mag, ref)).all()


def test_gradient_is_the_forwards(rg):
    """rg_out_prod_id's result against differences of the forward (F32 weights, whose route is exact to F32)."""
    rng = np.random.default_rng(8)
    s = Stack(torch, rg, F32, 3, 24, 16, _ids(rng, 5, 2, 3), 2)
    x, up = s.act(5, 16, F32), s.act(5, 24, F32)
    w = rng.random(s.slots).astype(np.float32)
    grad = s.run(False, F32, up, TOKEN, TOKEN, weights=w)
    h = np.float32(2.0 ** -6)
    # the forward is linear: a central difference has no error but the F32 sums'
    for t, k in [(0, 0), (2, 7), (4, 15)]:
        d = []
        for sign in (1, -1):
            z = x.copy()
            z[t, k] += sign * h
            d.append((s.run(True, F32, z, TOKEN, TOKEN, weights=w).astype(np.float64) * up).sum())
        slope = (d[0] - d[1]) / (2 * h)
        scale = np.abs(up[t]).sum() * 8
        assert abs(slope - grad[t, k]) <= scale * 64 * 2.0 ** -24 / h + 1e-6


def test_random(rg):
    """Seeded batches over the ranges."""
    for seed in range(24):
        rng = np.random.default_rng(1000 + seed)
        wtype = TYPES[seed % len(TYPES)]
        E = int(rng.integers(1, 40))
        top = int(rng.integers(1, min(E, 6) + 1))
        tokens = int(np.exp(rng.uniform(0, np.log(200))))
        N, K = 8 * int(rng.integers(1, 60)), 256 * int(rng.integers(1, 5))
        s = Stack(torch, rg, wtype, E, N, K, _ids(rng, tokens, top, E, rng.choice([0, 0.3])), top, seed=seed)
        s.check(bool(rng.integers(2)), int(rng.choice([F32, F16, BF16])), int(rng.integers(2)), int(rng.integers(2)),
                weigh=bool(rng.integers(2)), beta=float(rng.choice([0, 1, -0.25])), pad=int(rng.choice([0, 8])))
