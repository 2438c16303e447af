// rg_kv_tiles.cu - attention of many rows a sequence over the paged cache:
// prompts and chunks of prompts, on the 5th-generation tensor cores.
//
// An item is 256 rows (new tokens x the query heads of one kv head) of a
// sequence, two streams of 128, against its 128-token key tiles:
//   S = Q K^T           tcgen05.mma, both operands in shared memory, S in TMEM
//   P = 2^(S c - m)     one thread a row, TMEM -> registers -> TMEM (16 bits, over S)
//   O += P V            tcgen05.mma, P read from TMEM, V^T from shared memory
// While one stream's softmax runs, the tensor core works for the other.  Warps:
//   0 - 7    softmax, a warpgroup a stream; they also load Q and write the result
//   8 - 15   decoders: a granule (16 tokens) of each tile a warp, global memory ->
//            registers -> operand tiles (128-byte swizzle), a tile ahead
//   16       the thread that issues the matrix instructions
// The running maximum is a reference that moves only when a score passes it by
// 2^8 (as in rg_kv_rows.cu), so O is rescaled, which needs the tensor core's
// previous product finished, a few times an item.
// All items' key tiles form one line that is cut into equal shares, one a CTA:
// causal items of different lengths and ragged sequences balance, and a short
// prompt over a long cache uses every SM.  An item cut by a border leaves F32
// parts that a second kernel joins in a fixed order.
#include "rg_kv_attend.cuh"

namespace rg {
namespace kv {
namespace {

constexpr int BN = 128;          // tokens of a key tile
constexpr int BM = 256;          // rows of an item
constexpr int kSoftWarps = 8, kDecWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + kDecWarps + 1);
constexpr uint32_t kTmemCols = 512, kColO = 256;

template <int D>
struct Cfg {
  static constexpr int Q = 128 * D * 2;      // one stream's queries
  static constexpr int KV = 128 * D * 2;     // one tile's keys, or values
  static constexpr int SMEM = 2 * Q + 4 * KV + 1024;
  static constexpr int CHUNK = 128 * 128;    // 128 rows x 64 values
  static constexpr int VCHUNK = D * 128;     // D rows x 64 tokens
};

// --- the line of key tiles ----------------------------------------------------

struct Block {
  int t0, nt;          // first tile, tiles
  int minpos, maxpos;  // positions of the block's first and last row
  int rows;
};
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
__device__ __forceinline__ int blocks_of(const Seq& q, int group, int max_rows) {
  return q.n * group > max_rows ? (q.n * group + BM - 1) / BM : 0;
}

// A CTA's part of an item: tiles begin .. end - 1 of nt.
struct Segment {
  Seq sq;
  Block b;
  int seq, head, rb, begin, end;
  long long last;  // the line's index of the item's last tile
};
// Walks a CTA's share; every role walks it for itself.
struct Walk {
  long long at, hi;
  int seq, head, rb, tile, nrb;
  Seq sq;
  __device__ __forceinline__ bool next(const Cache& c, const Batch& b, const Attend& a, Segment& s) {
    if (at >= hi) return false;
    while (nrb == 0) {  // a new sequence
      if (++seq >= b.seqs) return false;
      sq = load_seq(b, c.page_tokens, seq, nullptr);
      nrb = blocks_of(sq, a.group, a.rows_limit);
    }
    s.sq = sq;
    s.seq = seq;
    s.head = head;
    s.rb = rb;
    s.b = block_of(sq, a.group, a.window, rb);
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

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tiles_kernel(Cache c, Batch b, Attend a, Desc* desc, float* parts, WaitCtl ctl) {
  using C = Cfg<D>;
  constexpr bool BF = TYPE == RG_BF16;
  constexpr int BLK = D / 32, GB = granule_bytes(TYPE, D);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[17];
  __shared__ __align__(8) uint8_t valid[8][kDecWarps];  // by tile ordinal: the granule's page exists
  __shared__ int poison[4];                             // by segment ordinal: values left out of the product
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ Walk sh_walk;
  __shared__ long long sh_sum[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, sK = base + 2 * C::Q, sV = sK + 2 * C::KV;
  auto bar = [&](int i) { return smem_addr(&bars[i]); };
  // barriers: two of each kind
  constexpr int KFULL = 0, KFREE = 2, VFULL = 4, VFREE = 6, SFULL = 8, PFULL = 10, ODONE = 12, QFULL = 14, DRAIN = 16;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(KFULL + i), kDecWarps);
      mbar_init(bar(KFREE + i), 1);
      mbar_init(bar(VFULL + i), kDecWarps);
      mbar_init(bar(VFREE + i), 1);
      mbar_init(bar(SFULL + i), 1);
      mbar_init(bar(PFULL + i), 4);
      mbar_init(bar(ODONE + i), 1);
      mbar_init(bar(QFULL + i), 4);
    }
    mbar_init(bar(DRAIN), 1);
    abort_flag = 0;
    for (int i = 0; i < 4; ++i) poison[i] = -1;
    fence_mbar_init();
  }
  if (warp == kSoftWarps + kDecWarps) {
    tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }

  // this CTA's share of the line
  auto tiles_of = [&](int s, int* status) -> long long {
    const Seq q = load_seq(b, c.page_tokens, s, status);
    const int nrb = blocks_of(q, a.group, a.rows_limit);
    long long n = 0;
    for (int rb = 0; rb < nrb; ++rb) n += block_of(q, a.group, a.window, rb).nt;
    return n * c.kv_heads;
  };
  long long sum = 0;
  for (int s = tid; s < b.seqs; s += kThreads) sum += tiles_of(s, ctl.status);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) sh_sum[warp] = sum;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  long long total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += sh_sum[w];
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long lo = per * blockIdx.x, hi = min(total, lo + per);
  if (warp == 0 && lo < hi) {  // where it begins
    long long acc = 0;
    for (int s0 = 0;; s0 += 32) {
      const long long v = s0 + lane < b.seqs ? tiles_of(s0 + lane, nullptr) : 0;
      long long inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, acc + inc > lo);
      if (past || s0 + 32 >= b.seqs) {
        const int l = past ? __ffs(past) - 1 : 31;
        const long long before = acc + __shfl_sync(0xFFFFFFFFu, inc - v, l);
        if (lane == 0) {
          Walk w;
          w.at = lo;
          w.hi = past ? hi : lo;
          w.seq = s0 + l;
          w.sq = load_seq(b, c.page_tokens, min(w.seq, b.seqs - 1), nullptr);
          w.nrb = blocks_of(w.sq, a.group, a.rows_limit);
          long long one = 0;
          for (int rb = 0; rb < w.nrb; ++rb) one += block_of(w.sq, a.group, a.window, rb).nt;
          long long rel = lo - before;
          w.head = one ? static_cast<int>(rel / one) : 0;
          rel -= w.head * one;
          w.rb = 0;
          for (; w.rb < w.nrb - 1; ++w.rb) {
            const int nt = block_of(w.sq, a.group, a.window, w.rb).nt;
            if (rel < nt) break;
            rel -= nt;
          }
          w.tile = static_cast<int>(rel);
          sh_walk = w;
        }
        break;
      }
      acc += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
  }
  __syncthreads();

  if (lo < hi) {
    Walk walk = sh_walk;
    Segment sg;
    if (warp < kSoftWarps) {
      // ---------------- softmax: a row a thread ----------------
      const int h = warp >> 2, r = (warp & 3) * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + lanes + h * 128, tO = tmem + lanes + kColO + h * 128;
      // (a scale of zero stands for a tiny one: hidden scores are -inf, and -inf x 0 is NaN)
      const float cz = fmaxf(fabsf(a.scale_log2), 1e-37f);
      const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
      uint32_t n_s = 0;      // tiles this stream has had
      uint32_t tile_no = 0;  // tiles of the CTA
      bool ok = true, headed = false;
      for (int ord = 0; ok && walk.next(c, b, a, sg); ++ord) {
        const int row = h * 128 + r;
        if (h == 1 && sg.b.rows <= 128) {
          tile_no += sg.end - sg.begin;
          continue;
        }
        const bool real = row < sg.b.rows;
        const int grow = sg.rb * BM + row;
        const int pos = real ? sg.sq.len - sg.sq.n + grow / a.group : -1;
        const int tok = sg.sq.start + grow / a.group, hd = sg.head * a.group + grow % a.group;
        {
          const uint32_t to = sQ + h * C::Q + r * 128;
#pragma unroll 4
          for (int k = 0; k < D / 8; ++k) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (real) v = query8<BF>(a, tok, hd, 8 * k, ctl.status);
            sts128(to + (k >> 3) * C::CHUNK + (((k & 7) ^ (r & 7)) << 4), v.x ^ flip, v.y ^ flip, v.z ^ flip,
                   v.w ^ flip);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(QFULL + h));
        }
        float m_ref = kNone, l = 0.0f;
        for (int i = sg.begin; i < sg.end; ++i, ++tile_no, ++n_s) {
          const int t = sg.b.t0 + i;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(SFULL + h), n_s & 1, ctl, &abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint64_t granules = *reinterpret_cast<const volatile uint64_t*>(valid[tile_no & 7]);
          const bool masked = tile_masked(sg.b, a.window, t) || granules != 0x0101010101010101ull;
          // columns (lim_lo, lim_hi] of the tile are visible to this row
          const int lim_hi = pos - t * BN, lim_lo = a.window ? pos - a.window - t * BN : -1;
          auto hide = [&](uint32_t (&s)[32], int c0) {
            const bool g0 = (granules >> (c0 / 16 * 8)) & 1, g1 = (granules >> (c0 / 16 * 8 + 8)) & 1;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (c0 + k > lim_hi || c0 + k <= lim_lo || !(k < 16 ? g0 : g1)) s[k] = 0xFF800000u;
          };
          float top = kNone;
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(tS + 32 * k4, s);
            if (masked) hide(s, 32 * k4);
#pragma unroll
            for (int k = 0; k < 32; ++k) top = fmaxf(top, __uint_as_float(s[k]));
          }
          top = top <= kNone ? kNone : top * cz;
          if (i == sg.begin) {
            m_ref = fmaxf(top, kNone);
          } else if (__any_sync(0xFFFFFFFFu, top > m_ref + kSlack)) {
            // rescale what has been accumulated, once the last product is in
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(ODONE + h), (n_s - 1) & 1, ctl, &abort_flag));
            if (!ok) break;
            tc_fence_after();
            const float v = fmaxf(top, m_ref), f = ex2(m_ref - v);
            m_ref = v;
            l *= f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(tO + 32 * k, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(tO + 32 * k, o);
            }
          }
          const float off = kHead - m_ref;
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            uint32_t s[32], p[16];
            tmem_ld_32x32b_x32(tS + 32 * k4, s);
            if (masked) hide(s, 32 * k4);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float e0 = ex2(fmaf(__uint_as_float(s[2 * k]), cz, off));
              const float e1 = ex2(fmaf(__uint_as_float(s[2 * k + 1]), cz, off));
              l += e0 + e1;
              p[k] = pack16<BF>(e0, e1);
            }
            tmem_st16(tS + 16 * k4, p);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PFULL + h));
        }
        if (!ok) break;
        // the result, or this CTA's part of it
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(ODONE + h), (n_s - 1) & 1, ctl, &abort_flag));
        if (!ok) break;
        tc_fence_after();
        const bool starts = sg.begin == 0, ends = sg.end == sg.b.nt;
        const bool left_out = *reinterpret_cast<volatile int*>(&poison[ord & 3]) == ord;
        float* part = parts + (static_cast<int64_t>(blockIdx.x) * 2 + (starts ? 1 : 0)) * part_floats(BM, D);
        const float inv = starts && ends ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
        if (!(starts && ends) && real) {
          part[row] = m_ref;
          part[BM + row] = l;
        }
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + 32 * k, o);
          if (left_out && real) {
            // values that are not finite, to the rows that see them
            const int* table = b.table + static_cast<int64_t>(sg.seq) * b.max_pages;
            for (int i = sg.begin; i < sg.end; ++i) {
              const int t = sg.b.t0 + i;
              if (!tile_masked(sg.b, a.window, t)) continue;
              for (int j = t * BN; j < t * BN + BN && j <= pos; ++j) {
                if (a.window && j <= pos - a.window) continue;
                const int page = table[j / c.page_tokens];
                if (page < 0 || page >= c.pages) continue;
                const uint8_t* src = c.data + granule_offset(c, page, 1, sg.head, j, GB);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) +
                                         value_not_finite<TYPE, D>(src, j % kGranule, 32 * k + e));
              }
            }
          }
          if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float v[4] = {__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                  __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv};
              if (starts && ends)
                store_out(a, tok, hd, 32 * k + e, v);
              else
                *reinterpret_cast<float4*>(part + 2 * BM + row * D + 32 * k + e) = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
        if (tid == 0 && starts && !ends) {
          headed = true;
          desc[blockIdx.x] = Desc{static_cast<int>(sg.last / per), sg.b.rows, sg.sq.start + sg.rb * BM / a.group,
                                  sg.rb * BM % a.group, sg.head};
        }
      }
      if (tid == 0 && !headed) desc[blockIdx.x].last = -1;
    } else if (warp < kSoftWarps + kDecWarps) {
      // ---------------- decoders: a granule of each tile a warp ----------------
      const int w = warp - kSoftWarps, g = lane >> 2, t4 = lane & 3;
      const int key0 = 4 * (g >> 1) + (g & 1);
      struct Tile {
        int page, pos, head, ord;
        bool there, masked;   // inside the sequence; hidden from some row
      };
      // the tile after the one before, its page number on the way
      bool more = walk.next(c, b, a, sg);
      int ord = 0, i = more ? sg.begin : 0;
      auto next_tile = [&](Tile& x) {
        if (!more) return false;
        const int t = sg.b.t0 + i;
        x.pos = t * BN + w * kGranule;
        x.head = sg.head;
        x.ord = ord;
        x.there = x.pos < min(sg.sq.len, sg.b.maxpos + 1);
        x.masked = tile_masked(sg.b, a.window, t);
        x.page = x.there ? __ldg(b.table + static_cast<int64_t>(sg.seq) * b.max_pages + x.pos / c.page_tokens) : -1;
        if (++i == sg.end) {
          more = walk.next(c, b, a, sg);
          ++ord;
          i = sg.begin;
        }
        return true;
      };
      KeyWords<TYPE> kw[BLK];
      ValueWords<TYPE> vw[BLK];
      auto load_keys = [&](const Tile& x) {
        if (x.page >= 0 && x.page < c.pages) {
          const uint8_t* src = c.data + granule_offset(c, x.page, 0, x.head, x.pos, GB);
#pragma unroll
          for (int k = 0; k < BLK; ++k) load_words<TYPE, D>(kw[k], src, k, lane);
        } else {
#pragma unroll
          for (int k = 0; k < BLK; ++k) kw[k] = KeyWords<TYPE>{};
        }
      };
      auto load_values = [&](const Tile& x) {
        if (x.page >= 0 && x.page < c.pages) {
          const uint8_t* src = c.data + granule_offset(c, x.page, 1, x.head, x.pos, GB);
#pragma unroll
          for (int k = 0; k < BLK; ++k) load_words<TYPE, D>(vw[k], src, k, lane);
        } else {
#pragma unroll
          for (int k = 0; k < BLK; ++k) vw[k] = ValueWords<TYPE>{};
        }
      };
      Tile cur, nxt;
      bool have = next_tile(cur);
      if (have) {
        load_keys(cur);
        load_values(cur);
      }
      for (uint32_t n = 0; have; ++n) {
        const bool have_next = next_tile(nxt);
        const uint32_t slot = n & 1, ph = (n >> 1) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar(KFREE + slot), ph ^ 1, ctl, &abort_flag))) break;
        {
          const uint32_t to = sK + slot * C::KV;
#pragma unroll
          for (int k = 0; k < BLK; ++k) {
            uint32_t kb[2][4];
            key_operand(kw[k], kb);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int row = 16 * w + key0 + 2 * q, chunk = (k & 1) * 4 + t4;
              sts128(to + (k >> 1) * C::CHUNK + row * 128 + ((chunk ^ (row & 7)) << 4), kb[q][0], kb[q][1], kb[q][2],
                     kb[q][3]);
            }
          }
          if (lane == 0) {
            const bool ok = !cur.there || (cur.page >= 0 && cur.page < c.pages);
            *reinterpret_cast<volatile uint8_t*>(&valid[n & 7][w]) = ok;
            if (!ok) report_index(ctl.status);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(KFULL + slot));
        }
        if (have_next) load_keys(nxt);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar(VFREE + slot), ph ^ 1, ctl, &abort_flag))) break;
        {
          const uint32_t to = sV + slot * C::KV + (w >> 2) * C::VCHUNK + (t4 & 1) * 8;
          const int chunk = (w & 3) * 2 + (t4 >> 1);
          bool bad = false;
#pragma unroll
          for (int k = 0; k < BLK; ++k) {
            uint32_t vb[4][2];
            if (cur.masked)
              value_operand<TYPE, true>(vw[k], vb, &bad);
            else
              value_operand<TYPE, false>(vw[k], vb, &bad);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row = 32 * k + 8 * q + g;
              sts64(to + row * 128 + ((chunk ^ (row & 7)) << 4), vb[q][0], vb[q][1]);
            }
          }
          if (bad) *reinterpret_cast<volatile int*>(&poison[cur.ord & 3]) = cur.ord;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(VFULL + slot));
        }
        if (have_next) load_values(nxt);
        cur = nxt;
        have = have_next;
      }
    } else if (lane == 0) {
      // ---------------- the matrix instructions ----------------
      constexpr uint32_t idS = idesc_f16(BF, 128, BN, false, false);
      constexpr uint32_t idO = idesc_f16(BF, 128, D, false, false);
      uint32_t n = 0, ns[2] = {0, 0}, nq[2] = {0, 0};
      bool ok = true;
      auto wait = [&](int i, uint32_t parity) {
        if (ok) ok = mbar_wait(bar(i), parity, ctl, &abort_flag);
        if (ok) tc_fence_after();
        return ok;
      };
      auto scores = [&](int h, uint32_t slot) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_f16(tmem + h * 128, sdesc_sw128(sQ + h * C::Q + (k >> 2) * C::CHUNK + (k & 3) * 32, 16, 1024),
                     sdesc_sw128(sK + slot * C::KV + (k >> 2) * C::CHUNK + (k & 3) * 32, 16, 1024), idS, k != 0);
        tc_commit(bar(SFULL + h));
      };
      while (ok && walk.next(c, b, a, sg)) {
        const int streams = sg.b.rows > 128 ? 2 : 1, count = sg.end - sg.begin;
        for (int h = 0; h < streams; ++h) wait(QFULL + h, nq[h]++ & 1);
        if (!wait(KFULL + (n & 1), (n >> 1) & 1)) break;
        for (int h = 0; h < streams; ++h) scores(h, n & 1);
        tc_commit(bar(KFREE + (n & 1)));
        for (int i = 0; i < count && ok; ++i, ++n) {
          const uint32_t slot = n & 1, next = (n + 1) & 1;
          if (!wait(VFULL + slot, (n >> 1) & 1)) break;
          for (int h = 0; h < streams; ++h) {
            if (!wait(PFULL + h, ns[h] & 1)) break;
            ++ns[h];
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_ts(tmem + kColO + h * 128, tmem + h * 128 + 8 * k,
                     sdesc_sw128(sV + slot * C::KV + (k >> 2) * C::VCHUNK + (k & 3) * 32, 16, 1024), idO,
                     i != 0 || k != 0);
            tc_commit(bar(ODONE + h));
            if (h == streams - 1) tc_commit(bar(VFREE + slot));
            if (i + 1 < count) {
              if (h == 0 && !wait(KFULL + next, ((n + 1) >> 1) & 1)) break;
              scores(h, next);
              if (h == streams - 1) tc_commit(bar(KFREE + next));
            }
          }
        }
      }
      if (!ok) {  // every product issued ends before tensor memory is freed
        tc_commit(bar(DRAIN));
        volatile int no_abort = 0;
        (void)mbar_wait(bar(DRAIN), 0, ctl, &no_abort);
      }
    }
    __syncwarp();
  } else if (tid == 0) {
    desc[blockIdx.x].last = -1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kDecWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  pdl_launch_dependents();
}

template <int TYPE, int D>
cudaError_t go(const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev, cudaStream_t stream) {
  auto kern = attend_tiles_kernel<TYPE, D>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  Desc* desc = static_cast<Desc*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) + (sizeof(Desc) * dev.num_sms + 255) / 256 * 256);
  kern<<<dev.num_sms, kThreads, Cfg<D>::SMEM, stream>>>(c, b, a, desc, parts, WaitCtl{dev.status, dev.wait_limit_ns});
  if ((e = counted(cudaGetLastError())) != cudaSuccess) return e;
  return launch_join(a, desc, parts, BM, D, dev.num_sms, stream);
}

template <int TYPE>
cudaError_t go_dim(const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev, cudaStream_t s) {
  return c.dim == 64 ? go<TYPE, 64>(c, b, a, ws, dev, s) : go<TYPE, 128>(c, b, a, ws, dev, s);
}

}  // namespace

bool tiles_have(int dim) { return dim <= 128; }

size_t tiles_workspace(const Cache& c, const DevInfo& dev) {
  return (sizeof(Desc) * dev.num_sms + 255) / 256 * 256 +
         (static_cast<size_t>(dev.num_sms) * 2 * part_floats(BM, c.dim) * 4 + 255) / 256 * 256;
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
