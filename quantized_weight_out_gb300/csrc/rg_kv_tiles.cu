// rg_kv_tiles.cu - attention of many rows a sequence over the paged cache:
// prompts and chunks of prompts, on the 5th-generation tensor cores.
//
// An item is 512 rows (new tokens x the query heads of one kv head) of a
// sequence, two streams of 256, against its 128-token key tiles.  A pair of CTAs
// (a cluster, two SMs) works on it, 128 rows of each stream a CTA:
//   S = Q K^T           tcgen05.mma.cta_group::2, M = 256: both operands in shared
//                       memory, S in TMEM
//   P = 2^(S c - m)     one thread a row, TMEM -> registers -> TMEM (16 bits, over S)
//   O += P V            tcgen05.mma.cta_group::2, P read from TMEM, V^T from shared memory
// Each CTA decodes and holds one half of a tile (64 tokens' keys; half the values'
// dimensions) for both: one CTA alone, reading whole tiles for its 256 rows and writing
// them itself, saturated its shared memory.  While one stream's softmax runs, the tensor
// cores work for the other.  Warps of each CTA:
//   0 - 7    softmax, a warpgroup a stream; they also load Q and write the result
//   8 - 15   decoders: half a granule (16 tokens) of keys and of values of each tile a
//            warp, global memory -> registers -> operand tiles (128-byte swizzle),
//            loaded a tile ahead
//   16       issues the matrix instructions (of the pair: the even CTA's)
//   17       scheduler: page numbers and masks of the next tiles (18, 19 idle:
//            registers are handed out by warpgroups)
// The running maximum is a reference that moves only when a score passes it by
// 2^8 (as in rg_kv_rows.cu), so O is rescaled, which needs the tensor core's
// previous product finished, a few times an item.
// All items' key tiles form one line that is cut into equal shares, one a pair:
// causal items of different lengths and ragged sequences balance, and a short
// prompt over a long cache uses every SM.  An item cut by a border leaves F32
// parts that a second kernel joins in a fixed order.
// Measured: 1021 tokens of 32 heads over a Q8_0 context of 15,000 (8 kv heads of 128)
// 233 us, 1.11 PFLOP/s, 0.59 of the measured burst bf16 rate; four packed prompts of
// 700 to 4,099 tokens, bf16 cache, 443 us, 0.85 PFLOP/s (one item's rows are written
// and the next one's first tile started in about 11,000 cycles of 3,300 a tile); 16
// heads of 256, the same prompts, 557 us a call.  The tensor pipe is active 54 % of the time:
// a stream's chain (scores complete, softmax 1,200 cycles, probabilities stored 250,
// waits 400, products and next scores 1,400) is longer than the other stream covers.
#include "rg_kv_attend.cuh"

namespace rg {
namespace kv {
namespace {

constexpr int BN = 128;          // tokens of a key tile
constexpr int kSoftWarps = 8, kDecWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + kDecWarps + 4);
constexpr int kMmaWarp = kSoftWarps + kDecWarps;
// Registers a thread: 96 at launch (640 threads), 61440 in all; then 256 x 168 for
// the softmax, 256 x 56 for the decoders and 128 x 32 for the rest, the same.
constexpr int kRegsSoft = 168, kRegsDec = 56, kRegsMma = 32;
template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr int kScan = 256;       // sequences counted at a time

template <int D>
struct Cfg {
  // streams of 256 rows: two of up to 128 dimensions; of 256 one, whose accumulators take half of
  // tensor memory and which has two score tiles in the other half, used in turn
  static constexpr int NS = D <= 128 ? 2 : 1;
  static constexpr int BM = 256 * NS;        // rows of an item
  static constexpr int Q = 128 * D * 2;      // a CTA's queries of one stream
  static constexpr int KV = 64 * D * 2;      // its half of a tile's keys, or values
  static constexpr int SMEM = NS * Q + 4 * KV + 1024;
  static constexpr int CHUNK = 128 * 128;    // queries: 128 rows x 64 dimensions
  static constexpr int KCHUNK = 64 * 128;    // keys: 64 tokens x 64 dimensions
  static constexpr int VCHUNK = D / 2 * 128; // values: D / 2 dimensions x 64 tokens
};

// --- the line of key tiles ----------------------------------------------------

struct Block {
  int t0, nt;          // first tile, tiles
  int minpos, maxpos;  // positions of the block's first and last row
  int rows;
};
template <int BM>
__device__ __forceinline__ Block block_of(const Seq& q, int group, int window, int rb) {
  Block b;
  const int first = q.len - q.n, r0 = rb * BM;
  b.rows = min(BM, q.n * group - r0);
  b.minpos = first + r0 / group;
  b.maxpos = first + (r0 + b.rows - 1) / group;
  b.t0 = window ? max(0, b.minpos - window + 1) / BN : 0;
  b.nt = max(1, (max(0, min(q.len, b.maxpos + 1)) + BN - 1) / BN - b.t0);
  return b;
}
template <int BM>
__device__ __forceinline__ int blocks_of(const Seq& q, int group, int max_rows) {
  return q.n * group > max_rows ? (q.n * group + BM - 1) / BM : 0;
}

// A CTA's part of an item: tiles begin .. end - 1 of nt.
struct Segment {
  Seq sq;
  Block b;
  int seq, head, rb, begin, end;
  bool holes;      // a page that is not there
  long long last;  // the line's index of the item's last tile
};
// Walks a CTA's share (the scheduler warp).
struct Walk {
  long long at, hi;
  int seq, head, rb, tile, nrb;
  Seq sq;
  template <int BM>
  __device__ __forceinline__ bool next(const Cache& c, const Batch& b, const Attend& a, Segment& s) {
    if (at >= hi) return false;
    while (nrb == 0) {  // a new sequence
      if (++seq >= b.seqs) return false;
      sq = load_seq(b, c.page_tokens, seq, nullptr);
      nrb = blocks_of<BM>(sq, a.group, a.rows_limit);
    }
    s.sq = sq;
    s.seq = seq;
    s.head = head;
    s.rb = rb;
    s.b = block_of<BM>(sq, a.group, a.window, rb);
    s.begin = tile;
    s.end = static_cast<int>(min(static_cast<long long>(s.b.nt), tile + (hi - at)));
    s.last = at + (s.b.nt - tile) - 1;
    at += s.end - tile;
    tile = 0;
    if (++rb == nrb) {
      rb = 0;
      if (++head == c.kv_heads) {
        head = 0;
        nrb = 0;
      }
    }
    return true;
  }
};

__device__ __forceinline__ bool tile_masked(const Block& b, int window, int t) {
  return t * BN + BN - 1 > b.minpos || (window && t * BN <= b.maxpos - window);
}

// --- tensor memory --------------------------------------------------------------

// The matrix instructions and commits are executed by the whole warp with one
// lane's predicate set, not in a branch of that lane: in converged code their
// operands stay in uniform registers.  (In a branch each instruction took about
// 150 cycles to issue, against the 64 that the tensor core needs for it.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc,
                                       uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc,
                                       uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc), "r"(one)
      : "memory");
}
// (arrives on the barrier at this offset in both CTAs of the pair)
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(
          bar),
      "r"(one), "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23,"
      " %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// The load without its wait, and the wait, after which r may be used.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  // (an asm statement takes 30 operands at most)
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// two F32 at once
__device__ __forceinline__ uint64_t pack_f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// What the decoders need to know of a tile, written by the scheduler a few tiles
// ahead, so that they wait for no page number and walk nothing.
struct TileInfo {
  long long off[8];   // byte offset of each granule's keys
  int flags;          // kEnd: no more tiles; kClean: values are checked, some row may not see them all
  int ord;            // segment
  int valid;          // bit g: granule g's tokens are there, or hidden by position
  uint16_t seen[8];   // bit j: token j of the granule is there, and some row of the item may see it
};
constexpr int kEnd = 1, kClean = 2;
constexpr int kRing = 8, kSegs = 4;
// Flags of values left out, by segment.  Both CTAs' decoders write both CTAs' flags, and a CTA
// is held back by its own segments' release only, so it may be kSegs segments ahead of the
// other, which may itself have kSegs that are not released: a flag read late is not yet written
// for a later segment with twice as many.
constexpr int kFlags = 2 * kSegs;

template <int TYPE, int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attend_tiles_kernel(Cache c, Batch b, Attend a, Desc* desc, float* parts, WaitCtl ctl) {
  using C = Cfg<D>;
  constexpr bool BF = TYPE == RG_BF16;
  constexpr int BM = C::BM, NS = C::NS;
  constexpr int HALF = D / 64, GB = granule_bytes(TYPE, D);  // HALF: blocks of 32 dimensions in half a row
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[13 + 2 * kRing + 2 * kSegs];
  __shared__ TileInfo ring[kRing];
  __shared__ Segment segs[kSegs];                       // begin -1: no more
  __shared__ uint8_t valid[8];                          // by tile ordinal: TileInfo's valid
  __shared__ int poison[kFlags];                        // by segment ordinal: values left out of the product
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ Walk sh_walk;
  __shared__ long long sh_tiles[kScan];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, sK = base + NS * C::Q, sV = sK + 2 * C::KV;
  const int rank = static_cast<int>(cluster_ctarank()), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto bar = [&](int i) { return smem_addr(&bars[i]); };
  auto lead = [&](int i) { return mapa_shared(bar(i), 0); };  // the even CTA's
  // barriers: two of each kind
  constexpr int FULL = 0, FREE = 2, SFULL = 4, PFULL = 6, ODONE = 8, QFULL = 10, DRAIN = 12, RFULL = 13,
                RFREE = RFULL + kRing, GFULL = RFREE + kRing, GFREE = GFULL + kSegs;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(FULL + i), 2 * kDecWarps);   // (used in the even CTA)
      mbar_init(bar(FREE + i), 1);
      mbar_init(bar(SFULL + i), 1);
      mbar_init(bar(PFULL + i), 8);               // (in the even CTA)
      mbar_init(bar(ODONE + i), 1);
      mbar_init(bar(QFULL + i), 8);               // (in the even CTA)
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar(RFULL + i), 1);
      mbar_init(bar(RFREE + i), kDecWarps);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar(GFULL + i), 1);
      mbar_init(bar(GFREE + i), 4 * NS + (rank == 0));
    }
    mbar_init(bar(DRAIN), 1);
    abort_flag = 0;
    for (int i = 0; i < kFlags; ++i) poison[i] = -1;
    fence_mbar_init();
  }
  pdl_launch_dependents();  // (the joining kernel waits for this one's end before it reads)
  if (warp == kMmaWarp) {
    tmem_alloc2(smem_addr(&tmem_slot), kTmemCols);
    tmem_relinquish2();
  }

  // This CTA's share of the line: every sequence's tiles are counted by a warp
  // (lanes over its blocks), kScan sequences at a time.
  auto count_tiles = [&](int s0, int* status) {
    for (int s = s0 + warp; s < min(b.seqs, s0 + kScan); s += kThreads / 32) {
      const Seq q = load_seq(b, c.page_tokens, s, status);
      const int nrb = blocks_of<BM>(q, a.group, a.rows_limit);
      long long all = 0;  // (2^21 blocks of 2^23 tiles at most)
      for (int rb = lane; rb < nrb; rb += 32) all += block_of<BM>(q, a.group, a.window, rb).nt;
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
      if (lane == 0) sh_tiles[s - s0] = all * c.kv_heads;
    }
  };
  long long total = 0;
  for (int s0 = 0; s0 < b.seqs; s0 += kScan) {
    if (s0) __syncthreads();
    count_tiles(s0, ctl.status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long sum = 0;
    for (int s = lane; s < min(b.seqs - s0, kScan); s += 32) sum += sh_tiles[s];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    total += sum;
  }
  const uint32_t tmem = tmem_slot;
  const long long per = (total + pairs - 1) / pairs;
  const long long lo = per * pair, hi = min(total, lo + per);
  // where it begins
  long long before = 0;
  bool found = lo >= hi;
  for (int s0 = 0; s0 < b.seqs && !found; s0 += kScan) {
    if (b.seqs > kScan) {
      __syncthreads();
      count_tiles(s0, nullptr);
      __syncthreads();
    }
    const int here = min(b.seqs - s0, kScan);
    for (int s1 = 0; s1 < here && !found; s1 += 32) {
      const long long v = s1 + lane < here ? sh_tiles[s1 + lane] : 0;
      long long inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + inc > lo);
      if (past) {
        found = true;
        if (warp == 0) {
          const int l = __ffs(past) - 1;
          const long long one = __shfl_sync(0xFFFFFFFFu, v, l) / c.kv_heads;
          long long rel = lo - before - __shfl_sync(0xFFFFFFFFu, inc - v, l);
          Walk w;
          w.at = lo;
          w.hi = hi;
          w.seq = s0 + s1 + l;
          w.sq = load_seq(b, c.page_tokens, w.seq, nullptr);
          w.nrb = blocks_of<BM>(w.sq, a.group, a.rows_limit);
          w.head = static_cast<int>(rel / one);
          rel -= w.head * one;
          for (int rb0 = 0;; rb0 += 32) {  // the block, 32 at a time
            const int nt = rb0 + lane < w.nrb ? block_of<BM>(w.sq, a.group, a.window, rb0 + lane).nt : 0;
            int sum = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
              if (lane >= o) sum += u;
            }
            const uint32_t in = __ballot_sync(0xFFFFFFFFu, sum > rel);
            if (in || rb0 + 32 >= w.nrb) {
              const int k = in ? __ffs(in) - 1 : 0;
              w.rb = rb0 + k;
              w.tile = static_cast<int>(rel) - __shfl_sync(0xFFFFFFFFu, sum - nt, k);
              break;
            }
            rel -= __shfl_sync(0xFFFFFFFFu, sum, 31);
          }
          if (lane == 0) sh_walk = w;
        }
      }
      before += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
  }
  // (also: the barriers and tensor memory of both CTAs are there)
  tc_fence_before();
  cluster_sync();
  tc_fence_after();

  if (lo < hi) {
    if (warp < 4 * NS) {
      // ---------------- softmax: a row a thread ----------------
      more_regs<kRegsSoft>();
      const int h = warp >> 2, r = (warp & 3) * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tO = tmem + lanes + kColO + h * 128;
      // (a scale of zero stands for a tiny one: hidden scores are -inf, and -inf x 0 is NaN)
      const float cz = fmaxf(fabsf(a.scale_log2), 1e-37f);
      const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
      uint32_t n_s = 0, n_seg = 0;  // tiles and segments this stream has had
      uint32_t tile_no = 0;         // tiles of the CTA
      bool ok = true, headed = false;
      auto segment = [&](int ord) -> const Segment& { return segs[ord % kSegs]; };
      auto wait_segment = [&](int ord) {
        ok = ok && __all_sync(0xFFFFFFFFu, wait_bar(bar(GFULL + ord % kSegs), (ord / kSegs) & 1, ctl, &abort_flag));
        return ok && segment(ord).begin >= 0;
      };
      auto release = [&](int ord) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(GFREE + ord % kSegs));
      };
      auto mine = [&](int ord) { return h == 0 || segment(ord).b.rows > 256; };
      const int row = h * 256 + rank * 128 + r;  // of the item
      // a segment's queries into shared memory: the lanes of a group take a row's 16-byte words
      auto load_queries = [&](const Segment& sg) {
        constexpr int LR = D / 8, RI = 32 / LR;  // lanes a row, rows at a time
        const int grow = sg.rb * BM + row;
        const int64_t at = (sg.sq.start + grow / a.group) * a.q_t + (sg.head * a.group + grow % a.group) * a.q_h;
        const int real = row < sg.b.rows;
        auto put = [&](int from, uint4 v) {
          const int at_row = (warp & 3) * 32 + from, word = lane % LR;
          sts128(sQ + h * C::Q + (word >> 3) * C::CHUNK + at_row * 128 + (((word & 7) ^ (at_row & 7)) << 4), v.x ^ flip,
                 v.y ^ flip, v.z ^ flip, v.w ^ flip);
        };
        if (a.atype == (BF ? RG_BF16 : RG_F16)) {
          // already the operand type: eight loads at a time (rows that do not exist read
          // the segment's first instead, and become zeros)
          const int64_t first = sg.sq.start * a.q_t + static_cast<int64_t>(sg.head) * a.group * a.q_h;
#pragma unroll 1
          for (int k0 = 0; k0 < 32 / RI; k0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int from = (k0 + k) * RI + lane / LR;
              const int64_t src = __shfl_sync(0xFFFFFFFFu, real ? at : first, from) + 8 * (lane % LR);
              v[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + src));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int from = (k0 + k) * RI + lane / LR;
              const bool there = __shfl_sync(0xFFFFFFFFu, real, from);
              put(from, there ? v[k] : make_uint4(0, 0, 0, 0));
            }
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < 32 / RI; ++k) {
            const int from = k * RI + lane / LR;
            const int64_t src = __shfl_sync(0xFFFFFFFFu, at, from);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (__shfl_sync(0xFFFFFFFFu, real, from)) v = query8<BF>(a, src + 8 * (lane % LR), ctl.status);
            put(from, v);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(QFULL + h));
      };
      bool loaded = false;
      for (int ord = 0; wait_segment(ord); ++ord) {
        const Segment& sg = segment(ord);
        const int begin = sg.begin, end = sg.end, t0 = sg.b.t0, minpos = sg.b.minpos, maxpos = sg.b.maxpos;
        if (!mine(ord)) {
          tile_no += end - begin;
          release(ord);
          continue;
        }
        if (!loaded) load_queries(sg);
        loaded = false;
        const bool holes = sg.holes;
        const int grow = sg.rb * BM + row;
        const bool real = row < sg.b.rows;
        const int pos = real ? sg.sq.len - sg.sq.n + grow / a.group : -1;
        float m_ref = kNone, l = 0.0f;
        for (int i = begin; i < end; ++i, ++tile_no, ++n_s) {
          const int t = t0 + i;
          // this tile's scores: the stream's, or every other tile's
          const int turn = NS == 2 ? h : n_s & 1;
          const uint32_t tS = tmem + lanes + turn * 128;
          ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(SFULL + turn), (NS == 2 ? n_s : n_s >> 1) & 1, ctl, &abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (holes || t * BN + BN - 1 > minpos || (a.window && t * BN <= maxpos - a.window)) {
            // hidden scores become -inf in tensor memory: the pass below has no mask
            const uint32_t granules = holes ? *reinterpret_cast<const volatile uint8_t*>(&valid[tile_no & 7]) : 0xFFu;
            // columns (lim_lo, lim_hi] of the tile are visible to this row
            const int lim_hi = pos - t * BN, lim_lo = a.window ? pos - a.window - t * BN : -1;
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 32) {
              const bool g0 = (granules >> (c0 / 16)) & 1, g1 = (granules >> (c0 / 16 + 1)) & 1;
              const int to = lim_hi - c0, from = lim_lo - c0;
              uint32_t s[32];
              tmem_ld_32x32b_x32(tS + c0, s);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k > to || k <= from || !(k < 16 ? g0 : g1)) s[k] = 0xFF800000u;
              tmem_st32(tS + c0, s);
            }
            tmem_wait_st();
          }
          // Probabilities relative to the reference so far, and the tile's maximum on the
          // way; where it passes the reference by too much, once more with a new one.
          uint32_t p[BN / 2];
          float sum;
          for (;;) {
            const float off = kHead - m_ref;
            const uint64_t cz2 = pack_f2(cz, cz), off2 = pack_f2(off, off);
            float top = kNone;
            uint64_t sum2 = 0;
            auto take = [&](const uint32_t (&x)[32], int c0) {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float s0 = __uint_as_float(x[2 * k]), s1 = __uint_as_float(x[2 * k + 1]);
                top = fmaxf(top, fmaxf(s0, s1));
                float e0, e1;
                unpack_f2(fma_f2(pack_f2(s0, s1), cz2, off2), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                sum2 = add_f2(sum2, pack_f2(e0, e1));
                p[c0 / 2 + k] = pack16<BF>(e0, e1);
              }
            };
            uint32_t x0[32], x1[32], y0[32], y1[32];
            tmem_ld32(tS, x0);
            tmem_ld32(tS + 32, x1);
            tmem_wait_ld(x0);
            tmem_wait_ld(x1);
            tmem_ld32(tS + 64, y0);
            tmem_ld32(tS + 96, y1);
            take(x0, 0);
            take(x1, 32);
            tmem_wait_ld(y0);
            tmem_wait_ld(y1);
            take(y0, 64);
            take(y1, 96);
            float sx, sy;
            unpack_f2(sum2, sx, sy);
            sum = sx + sy;
            top = top <= kNone ? kNone : top * cz;
            if (!__any_sync(0xFFFFFFFFu, top > m_ref + kSlack)) break;
            const float v = fmaxf(top, m_ref), f = ex2(m_ref - v);
            m_ref = v;
            if (i > begin) {
              // rescale what has been accumulated (two streams: the last product was issued
              // before this tile's scores, whose commit covers it)
              if constexpr (NS == 1) {
                ok = __all_sync(0xFFFFFFFFu,
                                wait_bar(bar(ODONE + ((n_s - 1) & 1)), ((n_s - 1) >> 1) & 1, ctl, &abort_flag));
                if (!ok) break;
                tc_fence_after();
              }
              l *= f;
#pragma unroll 1
              for (int k = 0; k < D / 32; ++k) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(tO + 32 * k, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(tO + 32 * k, o);
              }
            }
          }
          if (!ok) break;
          l += sum;
          tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(p));
          tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(p + 32));
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(lead(PFULL + turn));
        }
        if (!ok) break;
        // the next segment's queries (this one's have been read: its last scores are in)
        if (wait_segment(ord + 1) && mine(ord + 1)) {
          load_queries(segment(ord + 1));
          loaded = true;
        }
        // the result, or this CTA's part of it
        ok = ok && __all_sync(0xFFFFFFFFu,
                              NS == 2 ? wait_bar(bar(ODONE + h), n_seg++ & 1, ctl, &abort_flag)
                                      : wait_bar(bar(ODONE + ((n_s - 1) & 1)), ((n_s - 1) >> 1) & 1, ctl, &abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (__any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(&poison[ord % kFlags]) == ord)) {
          // Values that are not finite were left out of the products of tiles that some row sees
          // in part.  What this row sees of them in dimensions 32 k .. + 31: an infinity of either
          // sign a bit (both: NaN).  The warp looks at a token's 32 dimensions together.  (The
          // segment is read again, past the compiler: with its copies in registers for this, rare,
          // the tiles' loop took 2 to 5 % longer.)
          const volatile Segment& v = *const_cast<const volatile Segment*>(&sg);
          const int* table = b.table + static_cast<int64_t>(v.seq) * b.max_pages;
          const int low = v.b.minpos, high = v.b.maxpos, head = v.head;
          const int at = real ? v.sq.len - v.sq.n + (v.rb * BM + row) / a.group : -1;  // this row's position
          const int past = min((v.b.t0 + v.end) * BN, high + 1);
          const bool all = v.holes;
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t plus = 0, minus = 0;
#pragma unroll 1
            for (int j0 = (v.b.t0 + v.begin) * BN; j0 < past; j0 += kGranule) {
              const int t = j0 / BN * BN;
              if (!(all || t + BN - 1 > low || (a.window && t <= high - a.window))) continue;  // (as tile_masked())
              if (a.window && j0 + kGranule - 1 <= low - a.window) continue;
              const int page = table[j0 / c.page_tokens];
              if (page < 0 || page >= c.pages) continue;
              const uint8_t* src = c.data + granule_offset(c, page, 1, head, j0, GB);
              // (mostly there is none in the granule's block)
              ValueWords<TYPE> vw;
              load_words<TYPE, D>(vw, src, k, lane);
              uint32_t vb[4][2];
              value_operand(vw, vb);
              const uint32_t every[2] = {~0u, ~0u};
              if (!__any_sync(0xFFFFFFFFu, clean_operand<TYPE>(vb, every))) continue;
#pragma unroll 1
              for (int j = 0; j < kGranule; ++j) {
                const float x = value_not_finite<TYPE, D>(src, j, 32 * k + lane);
                const uint32_t up = __ballot_sync(0xFFFFFFFFu, !(x <= 0.0f)), down = __ballot_sync(0xFFFFFFFFu, !(x >= 0.0f));
                if (j0 + j <= at && !(a.window && j0 + j <= at - a.window)) {
                  plus |= up;
                  minus |= down;
                }
              }
            }
            uint32_t any = plus | minus;
#pragma unroll
            for (int i = 16; i; i >>= 1) any |= __shfl_xor_sync(0xFFFFFFFFu, any, i);
#pragma unroll 1
            for (; any; any &= any - 1) {
              const int e = __ffs(any) - 1;
              uint32_t o;
              asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                           : "=r"(o) : "r"(tO + 32 * k + e) : "memory");
              float x = __uint_as_float(o);
              if (plus >> e & 1) x += INFINITY;
              if (minus >> e & 1) x -= INFINITY;
              asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(tO + 32 * k + e),
                           "r"(__float_as_uint(x))
                           : "memory");
              tmem_wait_st();
            }
          }
        }
        const bool starts = begin == 0, ends = end == sg.b.nt;
        if (m_ref == kNone && sees_any(c, b.table + static_cast<int64_t>(sg.seq) * b.max_pages, a.window, pos,
                                       (t0 + begin) * BN, (t0 + end) * BN))
          m_ref = kMinusInf;
        const int64_t to = (sg.sq.start + grow / a.group) * a.o_t + (sg.head * a.group + grow % a.group) * a.o_h;
        float* part = parts + (static_cast<int64_t>(pair) * 2 + (starts ? 1 : 0)) * part_floats(BM, D);
        const float inv = starts && ends ? row_factor(m_ref, l) : 1.0f;
        if (!(starts && ends) && real) {
          part[row] = m_ref;
          part[BM + row] = l;
        }
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + 32 * k, o);
          if (real && !(starts && ends)) {
            float4* to4 = reinterpret_cast<float4*>(part + 2 * BM + row * D + 32 * k);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              to4[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          } else if (real) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v[8];
#pragma unroll
              for (int u = 0; u < 8; ++u) v[u] = __uint_as_float(o[8 * e + u]) * inv;
              const int64_t at = to + 32 * k + 8 * e;
              if (a.atype == RG_F32)
                store8<RG_F32>(a.out, at, v);
              else if (a.atype == RG_F16)
                store8<RG_F16>(a.out, at, v);
              else
                store8<RG_BF16>(a.out, at, v);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
        if (tid == 0 && rank == 0 && starts && !ends) {
          headed = true;
          desc[pair] = Desc{static_cast<int>(sg.last / per), sg.b.rows, sg.sq.start + sg.rb * BM / a.group,
                                  sg.rb * BM % a.group, sg.head};
        }
        release(ord);
      }
      if (tid == 0 && rank == 0 && !headed) desc[pair].last = -1;
    } else if (warp >= kSoftWarps && warp < kSoftWarps + kDecWarps) {
      // ---------------- decoders ----------------
      // Warp w of CTA `rank`: the keys of granule 4 rank + w / 2, half w % 2 of the dimensions;
      // the values of granule w, half `rank` of the dimensions.  In pairs: the values of tile
      // j - 1 and the keys of tile j, the order in which the tensor cores need them; the next
      // pair's words are loaded before the wait for its slots.
      if constexpr (NS == 2) fewer_regs<kRegsDec>();  // (one stream: 96 stay, the second warpgroup gives its own)
      const int w = warp - kSoftWarps, g = lane >> 2, t4 = lane & 3;
      const int kg = 4 * rank + (w >> 1), kb0 = (w & 1) * HALF, vb0 = rank * HALF;
      const int key0 = 16 * (w >> 1) + 4 * (g >> 1) + (g & 1);
      const long long to_values = c.kv_heads * c.slab_bytes;
      KeyWords<TYPE> kw[HALF] = {};
      ValueWords<TYPE> vw[HALF] = {};
      auto load_keys = [&](long long off) {
#pragma unroll
        for (int k = 0; k < HALF; ++k) load_words<TYPE, D>(kw[k], c.data + off, kb0 + k, lane);
      };
      const bool pages = c.pages > 0;
      bool any = __all_sync(0xFFFFFFFFu, wait_bar(bar(RFULL), 0, ctl, &abort_flag)) && !(ring[0].flags & kEnd);
      if (any && pages) load_keys(ring[0].off[kg]);
      bool clean = false;
      int ord = 0;
      const uint32_t full[2] = {lead(FULL), lead(FULL + 1)};
      for (uint32_t j = 0; any || j > 0; ++j) {
        const TileInfo& x = ring[j % kRing];
        if (j >= 2 &&
            !__all_sync(0xFFFFFFFFu, wait_bar(bar(FREE + (j & 1)), ((j - 2) >> 1) & 1, ctl, &abort_flag)))
          break;
        if (j > 0) {
          bool bad = false;
          const uint32_t to = sV + ((j - 1) & 1) * C::KV + (w >> 2) * C::VCHUNK + (t4 & 1) * 8;
          const int chunk = (w & 3) * 2 + (t4 >> 1);
#pragma unroll
          for (int k = 0; k < HALF; ++k) {
            uint32_t vb[4][2];
            value_operand(vw[k], vb);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row = 32 * k + 8 * q + g;
              sts64(to + row * 128 + ((chunk ^ (row & 7)) << 4), vb[q][0], vb[q][1]);
            }
          }
          if (clean) {  // again over what this lane has stored: rare, and no register above
            // Operands that are not finite become zero.  They are reported where a row of the
            // item may see them; elsewhere (past the newest token, before every window, a
            // page that is not there) they are bytes of anything, which nobody misses.
            const uint32_t seen = ring[(j - 1) % kRing].seen[w] >> (4 * t4);  // of this lane's four tokens
            const uint32_t seen_x = (seen & 1 ? 0xFFFFu : 0u) | (seen & 2 ? 0xFFFF0000u : 0u);
            const uint32_t seen_y = (seen & 4 ? 0xFFFFu : 0u) | (seen & 8 ? 0xFFFF0000u : 0u);
#pragma unroll 1
            for (int n = 0; n < 4 * HALF; ++n) {
              const int row = 8 * n + g;
              const uint32_t at = to + row * 128 + ((chunk ^ (row & 7)) << 4);
              uint2 u = lds64(at);
              const uint32_t out_x = clean_pair<TYPE>(u.x), out_y = clean_pair<TYPE>(u.y);
              if (out_x | out_y) {
                sts64(at, u.x, u.y);
                bad |= ((out_x & seen_x) | (out_y & seen_y)) != 0;
              }
            }
          }
          if (bad) {  // both CTAs' rows need these dimensions
#pragma unroll
            for (int r2 = 0; r2 < 2; ++r2)
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_addr(&poison[ord % kFlags]), r2)),
                           "r"(ord)
                           : "memory");
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
          }
        }
        if (any) {
          const uint32_t to = sK + (j & 1) * C::KV;
          if constexpr (HALF >= 2) {
            // Two blocks (the 128 bytes of a row's chunk) at a time: a quarter warp's stores
            // are two rows' four words each; where the odd row stores its other block first,
            // they fall on all eight 16-byte columns.
#pragma unroll
            for (int k = 0; k < HALF; k += 2) {
              uint32_t kb[2][2][4];
              key_operand(kw[k], kb[0]);
              key_operand(kw[k + 1 < HALF ? k + 1 : k], kb[1]);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int row = key0 + 2 * q;
                const uint32_t at = to + ((w & 1) * (HALF / 2) + k / 2) * C::KCHUNK + row * 128;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const int blk = u ^ (g & 1);
                  const bool odd = g & 1;
                  sts128(at + (((blk * 4 + t4) ^ (row & 7)) << 4), odd ? kb[u ^ 1][q][0] : kb[u][q][0],
                         odd ? kb[u ^ 1][q][1] : kb[u][q][1], odd ? kb[u ^ 1][q][2] : kb[u][q][2],
                         odd ? kb[u ^ 1][q][3] : kb[u][q][3]);
                }
              }
            }
          } else {
            uint32_t kb[2][4];
            key_operand(kw[0], kb);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int row = key0 + 2 * q;
              sts128(to + row * 128 + ((((w & 1) * 4 + t4) ^ (row & 7)) << 4), kb[q][0], kb[q][1], kb[q][2], kb[q][3]);
            }
          }
          if (lane == 0 && w == 0)
            *reinterpret_cast<volatile uint8_t*>(&valid[j & 7]) = static_cast<uint8_t>(x.valid);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(full[j & 1]);
          if (j > 0) mbar_arrive(bar(RFREE + (j - 1) % kRing));
        }
        if (!any) break;
        // the next pair: this tile's values, the next tile's keys
        clean = x.flags & kClean;
        ord = x.ord;
        if (pages) {
          const uint8_t* src = c.data + x.off[w] + to_values;
#pragma unroll
          for (int k = 0; k < HALF; ++k) load_words<TYPE, D>(vw[k], src, vb0 + k, lane);
        }
        if (!__all_sync(0xFFFFFFFFu, wait_bar(bar(RFULL + (j + 1) % kRing), ((j + 1) / kRing) & 1, ctl, &abort_flag)))
          break;
        any = !(ring[(j + 1) % kRing].flags & kEnd);
        if (any && pages) load_keys(ring[(j + 1) % kRing].off[kg]);
      }
    } else {
      fewer_regs<kRegsMma>();
    }
    if (warp == kMmaWarp + 1) {
      // ---------------- the scheduler: a granule of each tile a lane ----------------
      Walk walk = sh_walk;
      Segment sg;
      uint32_t n = 0;
      int ord = 0;
      bool ok = true;
      auto slot_free = [&] {
        ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(RFREE + n % kRing), ((n / kRing) & 1) ^ 1, ctl, &abort_flag));
        return ok;
      };
      auto segment_free = [&] {
        ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(GFREE + ord % kSegs), ((ord / kSegs) & 1) ^ 1, ctl, &abort_flag));
        return ok;
      };
      for (; ok && walk.template next<BM>(c, b, a, sg); ++ord) {
        if (!segment_free()) break;
        const int* table = b.table + static_cast<int64_t>(sg.seq) * b.max_pages;
        const int end = min(sg.sq.len, sg.b.maxpos + 1);
        bool hole = false;
        const int first = (sg.b.t0 + sg.begin) * BN, past = min(end, (sg.b.t0 + sg.end) * BN);
        for (int p = first / c.page_tokens + lane; p * static_cast<long long>(c.page_tokens) < past; p += 32) {
          const int page = __ldg(table + p);
          hole |= page < 0 || page >= c.pages;
        }
        sg.holes = __any_sync(0xFFFFFFFFu, hole);
        if (lane == 0) {
          segs[ord % kSegs] = sg;
          mbar_arrive(bar(GFULL + ord % kSegs));
        }
        __syncwarp();
        for (int i = sg.begin; i < sg.end; ++i, ++n) {
          const int t = sg.b.t0 + i, pos = t * BN + (lane & 7) * kGranule;
          const bool there = pos < end;
          const int page = there ? __ldg(table + pos / c.page_tokens) : -1;
          const bool paged = page >= 0 && page < c.pages;
          if (there && !paged) report_index(ctl.status);
          // A granule without a page of its own loads page 0's: its scores are hidden, so
          // its keys do not matter, and its values only have to be finite (cleaned).
          const long long off = granule_offset(c, paged ? page : 0, 0, sg.head, pos, GB);
          const uint32_t valid_bits = __ballot_sync(0xFFFFFFFFu, paged || !there) & 0xFFu;
          // tokens from_j .. to_j - 1 of the granule lie where some row may see them
          const int to_j = max(0, min(kGranule, end - pos));
          const int from_j = a.window ? max(0, min(kGranule, max(0, sg.b.minpos - a.window + 1) - pos)) : 0;
          const uint32_t seen = paged ? ((1u << to_j) - 1) & ~((1u << from_j) - 1) : 0u;
          if (!slot_free()) break;
          TileInfo& x = ring[n % kRing];
          if (lane < 8) {
            x.off[lane] = off;
            x.seen[lane] = static_cast<uint16_t>(seen);
          }
          if (lane == 0) {
            x.ord = ord;
            x.valid = static_cast<int>(valid_bits);
            x.flags = tile_masked(sg.b, a.window, t) || valid_bits != 0xFFu ? kClean : 0;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(RFULL + n % kRing));
        }
      }
      if (ok && slot_free()) {
        if (lane < 8) ring[n % kRing].off[lane] = 0;
        if (lane == 0) {
          ring[n % kRing].flags = kEnd;
          mbar_arrive(bar(RFULL + n % kRing));
        }
        if (segment_free() && lane == 0) {
          segs[ord % kSegs].begin = -1;
          mbar_arrive(bar(GFULL + ord % kSegs));
        }
      }
      __syncwarp();
    }
    if (warp == kMmaWarp && rank == 0) {
      // ---------------- the matrix instructions ----------------
      // (the whole warp waits, so that operands stay warp-uniform; one lane issues.  One
      // warp for both streams: their products alternate, so that one stream's softmax
      // runs while the other has the tensor core; a warp a stream fell into step and was
      // slower)
      constexpr uint32_t idS = idesc_f16(BF, 256, BN, false, false);
      constexpr uint32_t idO = idesc_f16(BF, 256, D, false, false);
      const uint64_t dQ = sdesc_sw128(sQ, 16, 1024), dK = sdesc_sw128(sK, 16, 1024), dV = sdesc_sw128(sV, 16, 1024);
      const uint32_t one = elect_one();
      const uint32_t tm = uniform(tmem);
      uint32_t n = 0, n1 = 0, q0 = 0, q1 = 0;  // tiles; stream 1's tiles; segments of each
      bool ok = true;
      auto wait = [&](int i, uint32_t parity) {
        ok = ok && __all_sync(0xFFFFFFFFu, wait_bar(bar(i), parity, ctl, &abort_flag));
        return ok;
      };
      // (one stream: h is the score tile's turn)
      auto scores = [&](int h, uint32_t slot) {
        const uint64_t q = dQ + (NS == 2 ? h : 0) * (C::Q >> 4), k = dK + slot * (C::KV >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tm + h * 128, q + (((i >> 2) * C::CHUNK + (i & 3) * 32) >> 4),
                 k + (((i >> 2) * C::KCHUNK + (i & 3) * 32) >> 4), idS, i != 0, one);
        commit_one(bar(SFULL + h), one);
      };
      auto product = [&](int h, uint32_t slot, bool first) {
        const uint64_t v = dV + slot * (C::KV >> 4);
#pragma unroll
        for (int i = 0; i < BN / 16; ++i)
          mma_ts(tm + kColO + (NS == 2 ? h : 0) * 128, tm + h * 128 + 8 * i, v + (((i >> 2) * C::VCHUNK + (i & 3) * 32) >> 4), idO,
                 i != 0 || !first, one);
      };
      // (FREE's event e: the scores of tile e and the products of tile e - 1 are done)
      int ord = 0;
      bool first_pair = true;
      while (wait(GFULL + ord % kSegs, (ord / kSegs) & 1)) {
        const Segment& sg = segs[ord % kSegs];
        const int count = uniform(sg.end - sg.begin);
        const bool two = uniform(sg.b.rows) > 256;
        if (uniform(sg.begin) < 0) break;
        if (first_pair && !wait(FULL, 0)) break;
        first_pair = false;
        if (!wait(QFULL, q0++ & 1)) break;
        tc_fence_after();
        if constexpr (NS == 1) {
          // scores a tile ahead of the products, so that a softmax runs beside them
          scores(n & 1, n & 1);
          commit_one(bar(FREE + (n & 1)), one);
          for (int i = 0; i < count; ++i, ++n) {
            const uint32_t slot = n & 1, next = (n + 1) & 1;
            const bool more = i + 1 < count;
            if (!wait(FULL + next, ((n + 1) >> 1) & 1)) break;
            tc_fence_after();
            if (more) scores(next, next);
            if (!wait(PFULL + slot, (n >> 1) & 1)) break;
            tc_fence_after();
            product(slot, slot, i == 0);
            // (a barrier for every other product: the softmax may be a product behind)
            commit_one(bar(ODONE + slot), one);
            if (more) commit_one(bar(FREE + next), one);
          }
        } else {
          scores(0, n & 1);
          if (two) {
            if (!wait(QFULL + 1, q1++ & 1)) break;
            tc_fence_after();
            scores(1, n & 1);
          }
          commit_one(bar(FREE + (n & 1)), one);
          for (int i = 0; i < count; ++i, ++n) {
            const uint32_t slot = n & 1, next = (n + 1) & 1;
            const bool more = i + 1 < count;
            if (!wait(FULL + next, ((n + 1) >> 1) & 1)) break;
            if (!wait(PFULL, n & 1)) break;
            tc_fence_after();
            product(0, slot, i == 0);
            if (more)
              scores(0, next);
            else
              commit_one(bar(ODONE), one);
            if (two) {
              if (!wait(PFULL + 1, n1++ & 1)) break;
              tc_fence_after();
              product(1, slot, i == 0);
              if (more)
                scores(1, next);
              else
                commit_one(bar(ODONE + 1), one);
            }
            if (more) commit_one(bar(FREE + next), one);
          }
        }
        if (!ok) break;
        if (one) mbar_arrive(bar(GFREE + ord % kSegs));
        ++ord;
      }
      if (!ok) {  // every product issued ends before tensor memory is freed
        commit_one(bar(DRAIN), one);
        volatile int no_abort = 0;
        (void)mbar_wait(bar(DRAIN), 0, ctl, &no_abort);
      }
      __syncwarp();
    }
  } else if (tid == 0 && rank == 0) {
    desc[pair].last = -1;
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // nothing of the pair's is in flight: each result waited for its products
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

template <int TYPE, int D>
cudaError_t go(const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev, cudaStream_t stream) {
  auto kern = attend_tiles_kernel<TYPE, D>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  // pairs of CTAs that can be on the device at once (an SM without a partner in its
  // cluster takes none), asked once per kernel and device
  static std::atomic<int> cached[64];
  const int pairs = std::min(dev.num_sms / 2, resident(cached[dev.device & 63], dev.num_sms / 2, [&](int* n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(dev.num_sms / 2 * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, kern, &cfg);
  }));
  Desc* desc = static_cast<Desc*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) + (sizeof(Desc) * dev.num_sms + 255) / 256 * 256);
  kern<<<2 * pairs, kThreads, Cfg<D>::SMEM, stream>>>(c, b, a, desc, parts, WaitCtl{dev.status, dev.wait_limit_ns});
  if ((e = counted(cudaGetLastError())) != cudaSuccess) return e;
  return launch_join(a, desc, parts, Cfg<D>::BM, D, pairs, stream);
}

template <int TYPE>
cudaError_t go_dim(const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev, cudaStream_t s) {
  return c.dim == 64    ? go<TYPE, 64>(c, b, a, ws, dev, s)
         : c.dim == 128 ? go<TYPE, 128>(c, b, a, ws, dev, s)
                        : go<TYPE, 256>(c, b, a, ws, dev, s);
}

}  // namespace

size_t tiles_workspace(const Cache& c, const DevInfo& dev) {
  return (sizeof(Desc) * dev.num_sms + 255) / 256 * 256 +
         (static_cast<size_t>(dev.num_sms / 2) * 2 * part_floats(c.dim == 256 ? Cfg<256>::BM : Cfg<128>::BM, c.dim) * 4 + 255) / 256 * 256;
}

cudaError_t launch_tiles(int type, const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev,
                         cudaStream_t stream) {
  switch (type) {
    case RG_F16: return go_dim<RG_F16>(c, b, a, ws, dev, stream);
    case RG_BF16: return go_dim<RG_BF16>(c, b, a, ws, dev, stream);
    case RG_Q8_0: return go_dim<RG_Q8_0>(c, b, a, ws, dev, stream);
    default: return go_dim<RG_Q4_0>(c, b, a, ws, dev, stream);
  }
}

}  // namespace kv
}  // namespace rg
