"""The ends of what the paged cache's calls take: many query heads a kv head, hundreds of
sequences, batches that mix prompts and single tokens, host threads side by side, graphs."""
import threading

import numpy as np
import pytest

import oracle
from quantized_weight_out_gb300 import inputs

from kv_common import RG_BF16, RG_F32, Setup, to_act
from test_gpu_kv_attend import _attend, _case, _contexts, rg  # noqa: F401  (rg: the fixture)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
F16, BF16, Q8, Q4 = inputs.F16, inputs.BF16, inputs.Q8_0, inputs.Q4_0


@pytest.mark.parametrize("G", [64, 65, 128, 513, 1024])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window", [0, 50])
def test_wide_groups(rg, G, D, window):  # noqa: F811
    """From 65 heads a kv head on a single token is a tile's work; above 512 it is several items'."""
    _case(rg, Q8, RG_BF16, D, 1, G, 16, [(1, 300), (2, 77), (0, 5), (3, 3), (1, 1)], window=window)
    _case(rg, F16, RG_F32, D, 2, G, 32, [(1, 129)], window=window)


@pytest.mark.parametrize("seqs", [
    [(1, 1 + 7 * s % 90) for s in range(700)],                                       # decoding
    [(40 + s % 3, 40 + s % 50) for s in range(300)],                                 # more than 64 rows each
    [(80, 80 + s % 30) if s % 37 == 5 else (s % 4, 4 + s % 60) for s in range(600)],  # both, and nothing new
])
def test_hundreds_of_sequences(rg, seqs):  # noqa: F811
    _case(rg, Q8, RG_BF16, 64, 1, 2, 16, [(n, max(n, L)) for n, L in seqs])


def _launches(rg, su, G):  # noqa: F811
    q = to_act(su.rng.standard_normal((su.tokens, su.H * G, su.D)).astype(np.float32), su.atype)
    before = rg.rg_launch_count()
    _attend(rg, su, q, su.H * G, 0.1)
    return rg.rg_launch_count() - before


@pytest.mark.parametrize("G,seqs,count", [
    (4, [(1, 100), (16, 40)], 2),              # few rows: their kernel and its join
    (4, [(100, 100)], 2),                      # one long sequence: the tile kernel and its join
    (4, [(100, 100), (1, 70), (1, 3)], 4),     # both
    (65, [(1, 100), (1, 40)], 2),              # no sequence can be a short one
])
def test_launches(rg, G, seqs, count):  # noqa: F811
    su = Setup(torch, rg, Q8, 64, 1, 16, seqs, atype=RG_BF16)
    k, v = _contexts(su)
    su.fill(k, v)
    assert _launches(rg, su, G) == count


def test_host_threads_side_by_side(rg):  # noqa: F811
    """Threads with streams and batches of their own, workspaces from the library's pool."""
    jobs = []
    for i, seqs in enumerate(([(1, 900), (1, 77)], [(130, 400)], [(1, 50), (90, 90), (3, 1000)], [(5, 5000)])):
        su = Setup(torch, rg, (Q8, F16, Q4, BF16)[i], 128, 2, 32, seqs, seed=i, atype=RG_BF16)
        k, v = _contexts(su)
        su.fill(k, v)
        q = su.tensor(to_act(su.rng.standard_normal((su.tokens, 8, 128)).astype(np.float32), RG_BF16))
        outs = [torch.empty_like(q) for _ in range(30)]
        jobs.append((su, q, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []

    def work(su, q, outs, stream):
        for out in outs:
            st = rg.rg_kv_attend(su.cache, su.batch, RG_BF16, q, 1024, 128, 8, out, 1024, 128, 0.1, 0, stream)
            if st != rg.RG_OK:
                failed.append(st)

    for su, q, outs, stream in jobs:  # alone first
        work(su, q, outs[:1], stream)
    torch.cuda.synchronize()
    want = [outs[0].clone() for _, _, outs, _ in jobs]
    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    rg.check(rg.rg_check(torch.cuda.current_stream()), "rg_check")
    for (_, _, outs, _), w in zip(jobs, want):
        assert not torch.isnan(w).any() and all(torch.equal(o, w) for o in outs)


@pytest.mark.parametrize("wtype", [F16, BF16, Q8, Q4])
def test_write_and_read_in_a_replayed_graph(rg, wtype):  # noqa: F811
    """One captured store and read-back serves steps of other tokens at other lengths."""
    D, H, S = 64, 2, 5
    su = Setup(torch, rg, wtype, D, H, 16, [(1, 200)] * S, seed=3, atype=RG_F32)
    HD = H * D
    k, v, ko, vo = (torch.zeros(S, H, D, device="cuda") for _ in range(4))

    def step(stream):
        rg.check(rg.rg_kv_write(su.cache, su.batch, RG_F32, k, HD, D, v, HD, D, stream), "rg_kv_write")
        rg.check(rg.rg_kv_read(su.cache, su.batch, RG_F32, ko, HD, D, vo, HD, D, stream), "rg_kv_read")

    step(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        su.len_d -= 1
        step(torch.cuda.current_stream())
    rows = []
    for _ in range(40):
        k.normal_()
        v.normal_()
        graph.replay()
        torch.cuda.synchronize()
        rows.append([x.cpu().numpy() for x in (k, v, ko, vo)])
    for kk, vv, k2, v2 in rows:
        assert np.array_equal(k2, oracle.kv_values(wtype, kk)) and np.array_equal(v2, oracle.kv_values(wtype, vv))
    # all of them are there: positions 198 down to 159
    b, start = su.whole()
    su.len_d.fill_(200)
    whole = torch.zeros(int(start[-1]), H, D, device="cuda")
    s = torch.cuda.current_stream()
    rg.check(rg.rg_kv_read(su.cache, b, RG_F32, whole, HD, D, None, HD, D, s), "rg_kv_read")
    rg.check(rg.rg_check(s), "rg_check")
    whole = whole.view(S, 200, H, D).cpu().numpy()
    for i, (_, _, k2, _) in enumerate(rows):
        assert np.array_equal(whole[:, 198 - i], k2)
