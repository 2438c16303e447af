"""What a cache's memory holds where nothing has been stored, or where no row may look,
changes neither a result of rg_kv_attend nor, by much, its time."""
import numpy as np
import pytest

from quantized_weight_out_gb300 import inputs

from kv_common import RG_BF16, Setup
from test_gpu_kv_attend import rg  # noqa: F401  (the fixture)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
F16, BF16, Q8, Q4 = inputs.F16, inputs.BF16, inputs.Q8_0, inputs.Q4_0


class Call:
    """A batch over a cache whose memory was `fill` before the contexts were stored."""

    def __init__(self, rg, wtype, D, H, G, P, seqs, fill, window=0, spoil=None):  # noqa: F811
        self.rg, self.G, self.window = rg, G, window
        self.su = su = Setup(torch, rg, wtype, D, H, P, seqs, seed=2, atype=RG_BF16)
        su.pool_d.fill_(fill)
        g = torch.Generator(device="cuda").manual_seed(7)
        k, v = (torch.randn(int(su.len.sum()), H, D, generator=g, device=su.dev) for _ in range(2))
        if spoil:
            spoil(su, k, v)
        rg.check(rg.rg_kv_write(su.cache, su.whole()[0], inputs.F32, k, H * D, D, v, H * D, D,
                                torch.cuda.current_stream()), "rg_kv_write")
        self.q = torch.randn(su.tokens, H * G, D, generator=g, device=su.dev).bfloat16()
        self.out = torch.empty_like(self.q)
        need = rg.rg_kv_attend_workspace_bytes(su.cache, su.batch, H * G)
        self.ws = torch.empty(need, dtype=torch.uint8, device=su.dev)

    def go(self):
        su, rg, row = self.su, self.rg, self.su.H * self.G * self.su.D
        rg.check(rg.rg_kv_attend_ws(su.cache, su.batch, RG_BF16, self.q, row, su.D, su.H * self.G, self.out, row, su.D,
                                    su.D ** -0.5, self.window, self.ws, self.ws.numel(), torch.cuda.current_stream()),
                 "rg_kv_attend")

    def result(self):
        self.go()
        torch.cuda.synchronize()
        return self.out.view(torch.int16).cpu().numpy()

    def time(self, replays=20):
        """us of a call inside a replayed graph, the least of several."""
        self.go()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.go()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = float("inf")
        for _ in range(replays):
            torch.cuda.synchronize()
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) * 1e3)
        return best


# Bytes 0xFF are a NaN as a scale and as a 16-bit value.  Twice the time allows for noise;
# where such bytes were taken for values that rows miss, the calls took 180 times as long and more.
@pytest.mark.parametrize("wtype", [F16, BF16, Q8, Q4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs,window", [([(1001, 1001)], 0), ([(301, 5005)], 0), ([(301, 5005)], 700)])
def test_prompts_over_stale_memory(rg, wtype, D, seqs, window):  # noqa: F811
    zero, stale = (Call(rg, wtype, D, 2, 4, 64, seqs, fill, window) for fill in (0, 255))
    assert np.array_equal(zero.result(), stale.result())
    t0, t1 = zero.time(), stale.time()
    assert t1 <= 2 * t0, (t0, t1)


# (A decode's last granule alone is looked at: 2.5 times the time where its stale bytes counted.)
@pytest.mark.parametrize("wtype", [F16, BF16, Q8, Q4])
@pytest.mark.parametrize("seqs,window", [([(1, 1001)], 0), ([(1, 1001)], 500), ([(1, 1001), (3, 70), (1, 5)], 0)])
def test_decoding_over_stale_memory(rg, wtype, seqs, window):  # noqa: F811
    zero, stale = (Call(rg, wtype, 256, 4, 4, 64, seqs, fill, window) for fill in (0, 255))
    assert np.array_equal(zero.result(), stale.result())
    t0, t1 = zero.time(60), stale.time(60)
    assert t1 <= 1.5 * t0, (t0, t1)


# A value of +inf (a NaN block in Q8_0) at one of the newest tokens: the rows behind it see it,
# those before it must not.  The call looks for it among the tiles at the diagonal, and where a
# page is missing among all of an item's; neither may take so long that another wait of the kernel
# runs out.  Looked for row by row and value by value it took 180 to 900 times as long.
@pytest.mark.parametrize("wtype", [BF16, Q8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hole", [False, True])
def test_a_visible_infinity_costs_little(rg, wtype, D, hole):  # noqa: F811
    n, L, at = 301, 9011, 8900

    def spoil(su, k, v):
        v[at, 1, 3] = float("inf")

    clean, call = (Call(rg, wtype, D, 2, 4, 64, [(n, L)], 0, spoil=how) for how in (None, spoil))
    if hole:
        for c in (clean, call):
            c.su.table_d[0, 5] = 1 << 20
    clean.go()
    call.go()
    s = torch.cuda.current_stream()
    assert rg.rg_check(s) == (rg.RG_ERR_INDEX if hole else rg.RG_OK)
    want, got = clean.out.float(), call.out.float()
    see = torch.arange(L - n, L, device="cuda") >= at
    spoilt = torch.zeros_like(want, dtype=torch.bool)
    spoilt[see, 4:, 0 if wtype == Q8 else 3:32 if wtype == Q8 else 4] = True
    assert (torch.isnan(got[spoilt]) if wtype == Q8 else got[spoilt] == float("inf")).all()
    assert torch.equal(got[~spoilt], want[~spoilt])
    t0, t1 = clean.time(), call.time()
    rg.rg_check(s)
    assert t1 <= 5 * t0, (t0, t1)
