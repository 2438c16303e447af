"""A paged cache and a batch for the tests, on both sides: numpy arrays for the
oracle, device tensors and descriptions for the library."""
import numpy as np

import oracle
from quantized_weight_out_gb300 import inputs

RG_F32, RG_F16, RG_BF16 = inputs.F32, inputs.F16, inputs.BF16


def to_act(x, atype):
    """F32 values as atype holds them (numpy F32)."""
    if atype == RG_F16:
        return x.astype(np.float16).astype(np.float32)
    if atype == RG_BF16:
        return oracle.kv_values(RG_BF16, x)
    return x.astype(np.float32)


class Setup:
    """seqs: (new tokens, length with them) pairs."""

    def __init__(self, torch, rg, wtype, D, H, P, seqs, seed=0, atype=RG_F32, extra_pages=2, fill=None, table_pad=1):
        self.torch, self.rg = torch, rg
        self.wtype, self.D, self.H, self.P, self.atype = wtype, D, H, P, atype
        self.seqs, self.rng = seqs, np.random.default_rng(seed)
        self.dev = torch.device("cuda:0")
        held = [-(-max(0, L) // P) for _, L in seqs]
        self.pages = sum(held) + extra_pages
        self.width = max(held + [1]) + table_pad
        order = self.rng.permutation(self.pages)
        self.table = np.full((len(seqs), self.width), -1, np.int32)
        at = 0
        for s, n in enumerate(held):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.page_bytes = oracle.kv_page_bytes(wtype, D, H, P)
        # stale bytes everywhere: every 16-bit word a NaN, or random ones
        if fill is None:
            self.pool = np.full((self.pages, self.page_bytes), 0xFF, np.uint8)
        else:
            self.pool = self.rng.integers(0, 256, (self.pages, self.page_bytes)).astype(np.uint8)
        self.new = [n for n, _ in seqs]
        self.tokens = sum(self.new)
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.len = np.array([L for _, L in seqs], np.int32)
        self.pool_d = torch.from_numpy(self.pool).to(self.dev)
        self.start_d, self.len_d, self.table_d = (torch.from_numpy(x).to(self.dev)
                                                  for x in (self.start, self.len, self.table))
        self.cache = rg.kv_cache(wtype, D, H, P, self.pages, self.pool_d)
        self.batch = rg.kv_batch(self.start_d, self.len_d, self.table_d, self.tokens, max(self.new + [0]))

    def tensor(self, x, atype=None):
        t = self.torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(self.dev)
        atype = self.atype if atype is None else atype
        return t.to({RG_F32: self.torch.float32, RG_F16: self.torch.float16, RG_BF16: self.torch.bfloat16}[atype])

    def whole(self):
        """The same sequences with every token new, for filling the cache: (batch, start)."""
        start = np.concatenate([[0], np.cumsum(np.maximum(self.len, 0))]).astype(np.int32)
        sd = self.torch.from_numpy(start).to(self.dev)
        b = self.rg.kv_batch(sd, self.len_d, self.table_d, int(start[-1]), int(max(self.len.max(), 0)))
        b._keep = sd
        return b, start

    def fill(self, k, v):
        """Stores whole contexts k, v [sum of lengths, H, D] F32 through rg_kv_write."""
        rg, b = self.rg, self.whole()[0]
        kd, vd = self.tensor(k, RG_F32), self.tensor(v, RG_F32)
        HD = self.H * self.D
        rg.check(rg.rg_kv_write(self.cache, b, RG_F32, kd, HD, self.D, vd, HD, self.D,
                                self.torch.cuda.current_stream()), "rg_kv_write")

    def positions(self, s):
        n, L = self.seqs[s]
        return np.arange(L - n, L)
