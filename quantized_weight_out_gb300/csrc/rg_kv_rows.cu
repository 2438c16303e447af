// rg_kv_rows.cu - attention of few rows a sequence over the paged cache: single
// tokens, drafted tokens, short chunks.
//
// The rows of a kv head (new tokens x the query heads that share it) are the N
// side of m16n8k16 products, 8, 16 or 32 at a time, and the cache is the M side
// (S^T = K Q^T, O^T = V^T P^T: few rows fill their side, and accumulators take
// D / 4 registers a lane for 8 rows); it is read once and decoded in registers.  With one running maximum and sum a row
// (out = sum_j 2^(z_j - m) v_j / sum_j 2^(z_j - m), z = score * scale * log2 e)
// keys can be taken in any order and in parts that are joined later by
// 2^(m_part - m), so the cache's length is the axis that work is split along:
//   - all (sequence, kv head, row block) items' 64-token tiles form one line, cut
//     into equal shares, one a CTA, whatever the sequences' lengths;
//   - inside a CTA every warp takes each fourth granule, with a ring of its own
//     that one lane fills by bulk copies (no barrier between warps);
//   - the warps' results are joined in shared memory; an item cut by a share's
//     border leaves partial sums that a second kernel joins, in a fixed order.
// The maximum is a reference that only moves when a score passes it by 2^8:
// probabilities are at most 2^15, the range fp16 has to spare, and the
// accumulators are rescaled a few times a row instead of at every granule.
// What bounds it: Q8_0 at G = 4, 64 ragged contexts of 300 to 15,000 tokens (1.15 GB),
// 200 us, 5.8 TB/s, 0.85 of the copy bandwidth; fewer bytes a value leave the decode's
// instructions in front: Q4_0 at 131,072 tokens 65 us, 2.3 TB/s (550 warp instructions a
// granule, issued in 62 % of the cycles of a kernel of 58 us; the rest is the join).  Rows on the M side, as first built, took 250 us for the
// ragged batch: 16 rows where 4 exist, twice the accumulators and matrix instructions.
// Scores, statistics and accumulators are F32; queries (of another type), decoded
// values and probabilities are rounded once to fp16 (a BF16 cache: bf16), since the
// matrix instructions take 16-bit operands, both of one type.
#include "rg_kv_launch.h"
#include "rg_kv_attend.cuh"

namespace rg {
namespace kv {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 64;            // tokens: a granule a warp
template <int TYPE, int D, int NT>
struct Cfg {
  static constexpr int BM = 8 * NT;
  static constexpr int OREGS = NT * D / 4;                 // accumulator registers a lane
  // granules a step: two where decoding is the work, so that the softmax's bookkeeping
  // and the queries' loads count once for 32 tokens (ragged Q8_0 batch: 220 us against
  // 238); one where there is no decoding, or no registers for two
  static constexpr int NG = has_scales(TYPE) && OREGS <= 64 ? 2 : 1;
  static constexpr bool QREG = NT * D <= 128;              // queries in registers (16 words a lane)
  static constexpr int GB = granule_bytes(TYPE, D);
  static constexpr int STAGE = 2 * GB;
  static constexpr int QBYTES = QREG ? 0 : NT * (D / 32) * 512;
  // CTAs a SM: as the registers allow, and with a ring of two stages at least
  static constexpr int fit(int ctas) { return ((227 * 1024) / ctas - 2048 - QBYTES) / (kWarps * STAGE); }
  static constexpr int most(int ctas) { return ctas > 1 && fit(ctas) < 2 ? most(ctas - 1) : ctas; }
  static constexpr int MINB = most(OREGS <= 32 ? 4 : OREGS <= 64 ? 3 : 2);
  static constexpr int MERGE_LD = D + 4;
  static constexpr int MERGE = kWarps * BM * MERGE_LD * 4;
  static constexpr int STAGES = fit(MINB) > 6 ? 6 : fit(MINB);
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int SMEM = (RING > MERGE ? RING : MERGE) + QBYTES;
  static_assert(STAGES >= 2, "a ring needs two stages");
};

struct Shape {
  int rb, t0, nt;  // row blocks; first tile; tiles
};
__device__ __forceinline__ Shape shape_of(const Seq& q, int group, int bm, int window, int max_rows) {
  Shape s{0, 0, 0};
  if (q.n == 0 || q.n * group > max_rows) return s;  // (the tile kernel's)
  s.rb = (q.n * group + bm - 1) / bm;
  const int first = max(q.len - q.n, 0);
  s.t0 = window ? max(0, first - window + 1) / kTile : 0;
  // a sequence that sees nothing still has its rows to write: one tile
  s.nt = max(1, (q.len + kTile - 1) / kTile - s.t0);
  return s;
}

// a / b for a >= 0, b > 0: 32-bit division where that is enough (it mostly is).
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a >> 32 == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, Cfg<TYPE, D, NT>::MINB)
    attend_rows_kernel(Cache c, Batch b, Attend a, Desc* desc, float* parts, WaitCtl ctl) {
  using C = Cfg<TYPE, D, NT>;
  constexpr bool BF = TYPE == RG_BF16;
  constexpr int BLK = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kWarps][C::STAGES];
  __shared__ float sm_m[kWarps][C::BM], sm_l[kWarps][C::BM];
  __shared__ long long sh_sum[kWarps];
  __shared__ int sh_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int G = a.group;

  if (lane < C::STAGES) mbar_init(smem_addr(&full[warp][lane]), 1);
  if (tid == 0) sh_abort = 0;
  fence_mbar_init();
  pdl_launch_dependents();  // (the joining kernel waits for this one's end before it reads)

  // this CTA's share [lo, hi) of the line of tiles
  auto tiles_of = [&](int s) -> long long {
    const Seq q = load_seq(b, c.page_tokens, s, ctl.status);
    const Shape sh = shape_of(q, G, C::BM, a.window, a.rows_limit);
    return static_cast<long long>(sh.rb) * sh.nt * c.kv_heads;
  };
  // tiles of 32 sequences by lane, and with those before
  auto scan = [&](int s0, long long* inc) {
    const long long v = s0 + lane < b.seqs ? tiles_of(s0 + lane) : 0;
    *inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, *inc, o);
      if (lane >= o) *inc += u;
    }
    return v;
  };
  long long inc0, total;
  const long long v0 = scan(0, &inc0);
  if (b.seqs <= 32) {  // every warp for itself
    total = __shfl_sync(0xFFFFFFFFu, inc0, 31);
  } else {
    long long sum = 0;
    for (int s = tid; s < b.seqs; s += 32 * kWarps) sum += tiles_of(s);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) sh_sum[warp] = sum;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sh_sum[w];
  }
  const long long per = quotient(total + gridDim.x - 1, gridDim.x);
  const long long lo = per * blockIdx.x, hi = min(total, lo + per);
  if (lo >= hi) {
    if (tid == 0) desc[blockIdx.x].last = -1;
    return;
  }
  // the sequence that tile lo belongs to
  int seq = 0;
  long long acc = 0;
  for (int s0 = 0;; s0 += 32) {
    long long inc = inc0, v = v0;
    if (s0) v = scan(s0, &inc);
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, acc + inc > lo);
    if (past || s0 + 32 >= b.seqs) {
      const int l = past ? __ffs(past) - 1 : 31;
      seq = s0 + l;
      acc += __shfl_sync(0xFFFFFFFFu, inc - v, l);
      break;
    }
    acc += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  __syncthreads();
  long long at = lo;
  bool headed = false;
  uint32_t it = 0;  // granules this warp has taken from its ring
  const uint32_t ring = smem_addr(smem) + C::QBYTES + warp * C::STAGES * C::STAGE;
  const uint32_t qbase = smem_addr(smem);
  float* merge = reinterpret_cast<float*>(smem + C::QBYTES);

  while (at < hi && seq < b.seqs) {
    const Seq sq = load_seq(b, c.page_tokens, seq, ctl.status);
    const Shape sh = shape_of(sq, G, C::BM, a.window, a.rows_limit);
    const long long tot = static_cast<long long>(sh.rb) * sh.nt * c.kv_heads;
    if (at >= acc + tot) {
      acc += tot;
      ++seq;
      continue;
    }
    const int item = static_cast<int>(quotient(at - acc, sh.nt));
    const int tile = static_cast<int>(at - acc - static_cast<long long>(item) * sh.nt);
    const int tend = static_cast<int>(min(static_cast<long long>(sh.nt), tile + (hi - at)));
    const int head = item / sh.rb, rb = item % sh.rb;
    const int row0 = rb * C::BM, nrows = sq.n * G, first = sq.len - sq.n;
    const int rows = min(C::BM, nrows - row0);
    const int minpos = first + row0 / G, maxpos = first + (row0 + rows - 1) / G;

    // positions of this lane's rows 8m + 2t + r (below every token: a row that does not exist)
    int pos[NT][2];
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 8 * m + 2 * t + r;
        pos[m][r] = row < rows ? first + (row0 + row) / G : -1;
      }

    // o[m][i]: dimensions 16i + g (words 0, 1: rows 2t, 2t + 1) and 16i + 8 + g (2, 3)
    float o[NT][D / 16][4], m_ref[NT][2], l_sum[NT][2];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][d][i] = 0.0f;
      m_ref[m][0] = m_ref[m][1] = kNone;
      l_sum[m][0] = l_sum[m][1] = 0.0f;
    }

    // this warp's granules: g0 + 4 k, k < count
    const int gend = min(4 * (sh.t0 + tend), (min(sq.len, maxpos + 1) + kGranule - 1) / kGranule);
    const int g0 = 4 * (sh.t0 + tile) + warp;
    const int count = g0 < gend ? (gend - g0 + kWarps - 1) / kWarps : 0;
    const int* table = b.table + static_cast<int64_t>(seq) * b.max_pages;
    // byte offsets of the keys of 32 of this warp's granules, one a lane (-1: no such page)
    auto load_offsets = [&](int k) -> long long {
      if (k + lane >= count) return -1;
      const int pos = (g0 + kWarps * (k + lane)) * kGranule;
      const int page = table[pos / c.page_tokens];
      if (page >= 0 && page < c.pages) return granule_offset(c, page, 0, head, pos, C::GB);
      report_index(ctl.status);
      return -1;
    };
    long long offs = load_offsets(0), offs_next = load_offsets(32);
    const long long to_values = c.kv_heads * c.slab_bytes;
    uint32_t st_in = it % C::STAGES, usable = 0;  // the next stage to fill; stages that hold something
    // granule k into its stage of the ring (the whole warp)
    auto issue = [&](int k) {
      if (k && (k & 31) == 0) {
        offs = offs_next;
        offs_next = load_offsets(k + 32);
      }
      const long long off = __shfl_sync(0xFFFFFFFFu, offs, k & 31);
      usable = off >= 0 ? usable | (1u << st_in) : usable & ~(1u << st_in);
      if (lane == 0) {
        const uint32_t bar = smem_addr(&full[warp][st_in]), to = ring + st_in * C::STAGE;
        if (off >= 0) {
          mbar_arrive_expect_tx(bar, C::STAGE);
          bulk_load(to, c.data + off, C::GB, bar);
          bulk_load(to + C::GB, c.data + off + to_values, C::GB, bar);
        } else {
          mbar_arrive(bar);
        }
      }
      st_in = st_in + 1 == C::STAGES ? 0 : st_in + 1;
    };

    const int first_batch = min(count, C::STAGES);
    for (int k = 0; k < first_batch; ++k) issue(k);

    // queries as B operands: row 8m + g, dimensions 32k + 8t .. + 7
    uint4 qreg[C::QREG ? NT : 1][C::QREG ? BLK : 1];
    auto query = [&](int m, int k) {
      const int row = row0 + 8 * m + g;
      return row < row0 + rows ? query8<BF>(a, (sq.start + row / G) * a.q_t + (head * G + row % G) * a.q_h + 32 * k + 8 * t,
                                            ctl.status)
                               : make_uint4(0, 0, 0, 0);
    };
    if constexpr (C::QREG) {
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int k = 0; k < BLK; ++k) qreg[m][k] = query(m, k);
    } else {
      for (int u = warp; u < NT * BLK; u += kWarps) reinterpret_cast<uint4*>(smem)[u * 32 + lane] = query(u / BLK, u % BLK);
      __syncthreads();
    }

    // N granules gran, gran + kWarps, ... in stages at kb[]: scores, probabilities, products
    // with the values.  have: bit u, granule u's page exists (MASKED only)
    auto step = [&](auto masked_c, auto n_c, int gran, const uint32_t* kb, uint32_t have) {
      constexpr bool MASKED = decltype(masked_c)::value;
      constexpr int N = decltype(n_c)::value;
      // s[m][u]: words 0, 1: token 4(g / 2) + g % 2 for rows 2t, 2t + 1; 2, 3: the token two on
      float s[NT][N][4];
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[m][u][i] = 0.0f;
#pragma unroll
      for (int k = 0; k < BLK; ++k) {
        uint4 x[NT];
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          if constexpr (C::QREG)
            x[m] = qreg[m][k];
          else
            x[m] = lds128(qbase + ((m * BLK + k) * 32 + lane) * 16);
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
          KeyWords<TYPE> kw;
          load_words<TYPE, D>(kw, kb[u], k, lane);
          uint32_t op[2][4];
          key_operand(kw, op);
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            mma16<BF>(s[m][u], op[0][0], op[1][0], op[0][1], op[1][1], x[m].x, x[m].y);
            mma16<BF>(s[m][u], op[0][2], op[1][2], op[0][3], op[1][3], x[m].z, x[m].w);
          }
        }
      }
      uint32_t p[NT][2 * N];
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        float top[2] = {kNone, kNone};
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float z = s[m][u][i] * a.scale_log2;
            if constexpr (MASKED) {
              const int j = (gran + kWarps * u) * kGranule + 4 * (g >> 1) + 2 * (i >> 1) + (g & 1), ps = pos[m][i & 1];
              if (j > ps || (a.window && j <= ps - a.window) || !((have >> u) & 1)) z = -INFINITY;
            }
            s[m][u][i] = z;
            top[i & 1] = fmaxf(top[i & 1], z);
          }
        if (__any_sync(0xFFFFFFFFu, top[0] > m_ref[m][0] + kSlack || top[1] > m_ref[m][1] + kSlack)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float v = fmaxf(top[r], m_ref[m][r]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
            const float f = ex2(m_ref[m][r] - v);
            m_ref[m][r] = v;
            l_sum[m][r] *= f;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              o[m][d][r] *= f;
              o[m][d][2 + r] *= f;
            }
          }
        }
        const float base0 = m_ref[m][0] - kHead, base1 = m_ref[m][1] - kHead;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const float e0 = ex2(s[m][u][0] - base0), e1 = ex2(s[m][u][1] - base1);
          const float e2 = ex2(s[m][u][2] - base0), e3 = ex2(s[m][u][3] - base1);
          l_sum[m][0] += e0 + e2;
          l_sum[m][1] += e1 + e3;
          // [token][row] -> [row][token]: tokens 4t, 4t + 1 and 4t + 2, 4t + 3 of row g
          p[m][2 * u] = transpose8x8(pack16<BF>(e0, e1));
          p[m][2 * u + 1] = transpose8x8(pack16<BF>(e2, e3));
        }
      }
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const uint32_t vbase = kb[u] + C::GB;
        bool bad = false;
        uint32_t seen[2] = {0, 0};  // the lane's tokens that some row may see (others hold anything)
        if constexpr (MASKED) {
          const int j = (gran + kWarps * u) * kGranule + 4 * t;
          const int from = a.window ? minpos - a.window + 1 : 0, to = (have >> u) & 1 ? maxpos : -1;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j + i >= from && j + i <= to) seen[i >> 1] |= i & 1 ? 0xFFFF0000u : 0xFFFFu;
        }
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
          ValueWords<TYPE> vw;
          load_words<TYPE, D>(vw, vbase, k, lane);
          uint32_t vb[4][2];
          value_operand(vw, vb);
          if constexpr (MASKED) bad |= clean_operand<TYPE>(vb, seen);
#pragma unroll
          for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int q = 0; q < 4; q += 2)
              mma16<BF>(o[m][2 * k + q / 2], vb[q][0], vb[q + 1][0], vb[q][1], vb[q + 1][1], p[m][2 * u], p[m][2 * u + 1]);
        }
        if constexpr (MASKED) {
          // values that are not finite were left out of the product (0 x inf would
          // reach rows that may not see them): add them to the rows that do
          if (__any_sync(0xFFFFFFFFu, bad)) {
            for (int jj = 0; jj < kGranule; ++jj) {
              const int j = (gran + kWarps * u) * kGranule + jj;
#pragma unroll
              for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float v = value_not_finite<TYPE, D>(vbase, jj, 16 * d + 8 * e + g);
#pragma unroll
                  for (int m = 0; m < NT; ++m)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                      if (j <= pos[m][r] && !(a.window && j <= pos[m][r] - a.window)) o[m][d][2 * e + r] += v;
                }
            }
          }
        }
      }
    };

    bool gave_up = false;
    uint32_t st = it % C::STAGES, phase = it / C::STAGES & 1;  // of the next granule to use
    for (int k = 0; k < count;) {
      // as many as a step takes, if they are there
      const int n = C::NG == 2 && k + 1 < count ? 2 : 1;
      uint32_t kb[2], have = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u >= n) break;
        if (!gave_up && !wait_bar(smem_addr(&full[warp][st]), phase, ctl, &sh_abort)) gave_up = true;
        kb[u] = ring + st * C::STAGE;
        have |= (usable >> st & 1) << u;
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1;
        }
      }
      gave_up = __any_sync(0xFFFFFFFFu, gave_up);
      if (gave_up) {
        // copies already under way must land before the CTA's shared memory is given up
        const uint64_t t0 = globaltimer_ns();
        for (int u = k; u < min(count, k + C::STAGES); ++u)
          while (!mbar_try_wait(smem_addr(&full[warp][(it + u) % C::STAGES]), (it + u) / C::STAGES & 1) &&
                 globaltimer_ns() - t0 < ctl.limit_ns) {
          }
        break;
      }
      const int gran = g0 + kWarps * k, j0 = gran * kGranule, j1 = (gran + kWarps * (n - 1)) * kGranule;
      const bool whole = have == (1u << n) - 1 && j1 + kGranule - 1 <= minpos && !(a.window && j0 <= maxpos - a.window);
      if (n == 2) {
        if constexpr (C::NG == 2) {
          if (whole)
            step(std::false_type{}, std::integral_constant<int, 2>{}, gran, kb, have);
          else {
            uint32_t at = kb[0];
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
              step(std::true_type{}, std::integral_constant<int, 1>{}, gran + kWarps * u, &at, have >> u);
              at = kb[1];
            }
          }
        }
      } else if (C::NG == 1 && whole) {
        step(std::false_type{}, std::integral_constant<int, 1>{}, gran, kb, have);
      } else {
        step(std::true_type{}, std::integral_constant<int, 1>{}, gran, kb, have);
      }
      __syncwarp();
#pragma unroll 1
      for (int u = 0; u < n; ++u)
        if (k + u + C::STAGES < count) issue(k + u + C::STAGES);
      k += n;
    }
    if (__syncthreads_or(gave_up)) {
      if (tid == 0 && !headed) desc[blockIdx.x].last = -1;
      return;
    }
    it += count;

    // join the four warps
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = l_sum[m][r];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        const int row = 8 * m + 2 * t + r;
        if (g == 0) {
          sm_m[warp][row] = m_ref[m][r];
          sm_l[warp][row] = l;
        }
        if (row < rows) {
          float* to = merge + (warp * C::BM + row) * C::MERGE_LD + g;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            to[16 * d] = o[m][d][r];
            to[16 * d + 8] = o[m][d][2 + r];
          }
        }
      }
    __syncthreads();
    const bool starts = tile == 0, ends = tend == sh.nt;
    float* part = parts + (static_cast<int64_t>(blockIdx.x) * 2 + (starts ? 1 : 0)) * part_floats(C::BM, D);
    for (int u = tid; u < rows * (D / 4); u += 32 * kWarps) {
      const int row = u / (D / 4), d = u % (D / 4) * 4;
      float top = sm_m[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][row]);
      float v[4] = {0, 0, 0, 0}, l = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(sm_m[w][row] - top);
        const float4 x = *reinterpret_cast<const float4*>(merge + (w * C::BM + row) * C::MERGE_LD + d);
        l += f * sm_l[w][row];
        v[0] += f * x.x; v[1] += f * x.y; v[2] += f * x.z; v[3] += f * x.w;
      }
      if (top == kNone && sees_any(c, table, a.window, first + (row0 + row) / G, (sh.t0 + tile) * kTile,
                                   (sh.t0 + tend) * kTile))
        top = kMinusInf;
      if (starts && ends) {
        const float inv = row_factor(top, l);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= inv;
        store_out(a, sq.start + (row0 + row) / G, head * G + (row0 + row) % G, d, v);
      } else {
        *reinterpret_cast<float4*>(part + 2 * C::BM + row * D + d) = make_float4(v[0], v[1], v[2], v[3]);
        if (d == 0) {
          part[row] = top;
          part[C::BM + row] = l;
        }
      }
    }
    if (starts && !ends) {
      headed = true;
      if (tid == 0) {
        const long long end = acc + static_cast<long long>(item + 1) * sh.nt - 1;
        desc[blockIdx.x] =
            Desc{static_cast<int>(per >> 31 == 0 ? quotient(end, static_cast<int>(per)) : end / per), rows, sq.start + row0 / G, row0 % G, head};
      }
    }
    at += tend - tile;
    fence_proxy_async_smem();  // the ring is refilled over what was just read and written
    __syncthreads();
  }
  if (tid == 0 && !headed) desc[blockIdx.x].last = -1;
}

// Joins the parts of items that several CTAs share: block (i, y) has `stretch`
// rows of the item whose first part CTA i has.  A warp a row first finds the
// row's reference and sum; then threads take (row, 4 dimensions), and where there
// are more threads than that, several share the parts, added in a fixed order.
// Each part's loads stand alone, so that many are in flight.
constexpr int kJoin = 512;
__global__ void __launch_bounds__(kJoin) attend_join_kernel(Attend a, const Desc* desc, const float* parts, int bm,
                                                            int dim, int stretch) {
  __shared__ float sm_top[32], sm_inv[32];
  __shared__ __align__(16) float sm_v[kJoin * 4];
  pdl_wait();
  const Desc ds = desc[blockIdx.x];
  const int first = blockIdx.y * stretch, rows = min(stretch, ds.rows - first);
  if (ds.last < 0 || rows <= 0) return;
  const int tid = threadIdx.x, lane = tid & 31;
  const int n = ds.last - static_cast<int>(blockIdx.x) + 1;
  const int64_t size = part_floats(bm, dim);
  const float* head = parts + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * size;
  const float* rest = parts + static_cast<int64_t>(blockIdx.x) * 2 * size;  // part i >= 1: rest + 2 i size
  auto part = [&](int i) { return i == 0 ? head : rest + 2 * i * size; };
  for (int r = tid >> 5; r < rows; r += kJoin / 32) {
    const int row = first + r;
    float top = kNone, l = 0.0f;
    for (int i0 = 0; i0 < n; i0 += 128) {  // 128 parts at a time, their loads together
      float m[4], s[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 32 * u + lane;
        m[u] = i < n ? part(i)[row] : kNone;
        s[u] = i < n ? part(i)[bm + row] : 0.0f;
      }
      float v = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
#pragma unroll
      for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
      v = fmaxf(v, top);
      l *= ex2(top - v);
      top = v;
#pragma unroll
      for (int u = 0; u < 4; ++u) l += s[u] * ex2(m[u] - top);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    if (lane == 0) {
      sm_top[r] = top;
      sm_inv[r] = row_factor(top, l);
    }
  }
  __syncthreads();
  const int quads = dim / 4, items = rows * quads;
  const int groups = items < kJoin ? kJoin / items : 1;
  for (int u0 = 0; u0 < items; u0 += kJoin) {
    const int u = groups > 1 ? tid % items : u0 + tid, grp = groups > 1 ? tid / items : 0;
    const bool mine = u < items && grp < groups;
    const int r = mine ? u / quads : 0, row = first + r, d = mine ? u % quads * 4 : 0;
    float v[4] = {0, 0, 0, 0};
    if (mine) {
      const float top = sm_top[r];
      for (int i0 = grp; i0 < n; i0 += 8 * groups) {  // eight parts at a time
        float m[8];
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float* p = part(min(i0 + k * groups, n - 1));
          // (past the last part: nothing, by way of its loads; 0 x an infinity would be NaN)
          const bool there = i0 + k * groups < n;
          m[k] = there ? p[row] : -INFINITY;
          x[k] = *reinterpret_cast<const float4*>(p + 2 * bm + row * dim + d);
          if (!there) x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float f = ex2(m[k] - top);
          v[0] += f * x[k].x; v[1] += f * x[k].y; v[2] += f * x[k].z; v[3] += f * x[k].w;
        }
      }
    }
    if (groups > 1) {
      *reinterpret_cast<float4*>(sm_v + 4 * tid) = make_float4(v[0], v[1], v[2], v[3]);
      __syncthreads();
      if (mine && grp == 0)
        for (int k = 1; k < groups; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(sm_v + 4 * (tid + k * items));
          v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        }
    }
    if (mine && grp == 0) {
      const float inv = sm_inv[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= inv;
      store_out(a, ds.token + (ds.lead + row) / a.group, ds.head * a.group + (ds.lead + row) % a.group, d, v);
    }
  }
}

constexpr int kMaxCtasPerSm = 4;

// Rows of eight side by side: as many as the longest sequence has, up to 32 (16 of
// 256 dimensions: the accumulators' registers).
int rows_nt(const Batch& b, int group, int dim) {
  const int64_t rows = static_cast<int64_t>(b.max_new) * group;
  return rows <= 8 ? 1 : rows <= 16 || dim == 256 ? 2 : 4;
}

template <int TYPE, int D, int NT>
cudaError_t go(const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev, cudaStream_t stream) {
  using K = Cfg<TYPE, D, NT>;
  auto kern = attend_rows_kernel<TYPE, D, NT>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), K::SMEM);
  if (e != cudaSuccess) return e;
  // no more CTAs than tiles there can be
  const int64_t blocks = (static_cast<int64_t>(b.tokens) * a.group + K::BM - 1) / K::BM + b.seqs;
  const int64_t tiles = static_cast<int64_t>(b.max_pages) * c.page_tokens / kTile + 1;
  const int64_t most = blocks > kMaxCtasPerSm * 1024 / c.kv_heads ? kMaxCtasPerSm * 1024 : blocks * c.kv_heads * tiles;
  const int grid = static_cast<int>(std::min<int64_t>(most, static_cast<int64_t>(dev.num_sms) * K::MINB));
  Desc* desc = static_cast<Desc*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                          (sizeof(Desc) * kMaxCtasPerSm * dev.num_sms + 255) / 256 * 256);
  kern<<<grid, 32 * kWarps, K::SMEM, stream>>>(c, b, a, desc, parts, WaitCtl{dev.status, dev.wait_limit_ns});
  if ((e = counted(cudaGetLastError())) != cudaSuccess) return e;
  return launch_join(a, desc, parts, K::BM, D, grid, stream);
}

template <int TYPE>
cudaError_t go_dim(const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev, cudaStream_t s) {
  const int nt = rows_nt(b, a.group, c.dim);
  if (c.dim == 64)
    return nt == 4   ? go<TYPE, 64, 4>(c, b, a, ws, dev, s)
           : nt == 2 ? go<TYPE, 64, 2>(c, b, a, ws, dev, s)
                     : go<TYPE, 64, 1>(c, b, a, ws, dev, s);
  if (c.dim == 128)
    return nt == 4   ? go<TYPE, 128, 4>(c, b, a, ws, dev, s)
           : nt == 2 ? go<TYPE, 128, 2>(c, b, a, ws, dev, s)
                     : go<TYPE, 128, 1>(c, b, a, ws, dev, s);
  return nt == 2 ? go<TYPE, 256, 2>(c, b, a, ws, dev, s) : go<TYPE, 256, 1>(c, b, a, ws, dev, s);
}

}  // namespace

cudaError_t launch_join(const Attend& a, const Desc* desc, const float* parts, int bm, int dim, int ctas,
                        cudaStream_t stream) {
  const int stretch = std::min(bm, std::min(32, kJoin * 4 / dim));  // rows a block: one (row, 4 dimensions) a thread
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, (bm + stretch - 1) / stretch);
  cfg.blockDim = dim3(kJoin);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted(cudaLaunchKernelEx(&cfg, attend_join_kernel, a, desc, parts, bm, dim, stretch));
}

size_t rows_workspace(const Cache& c, const Batch& b, int group, const DevInfo& dev) {
  const int bm = 8 * rows_nt(b, group, c.dim);
  const int64_t ctas = static_cast<int64_t>(kMaxCtasPerSm) * dev.num_sms;
  return static_cast<size_t>((ctas * sizeof(Desc) + 255) / 256 * 256 + ctas * 2 * part_floats(bm, c.dim) * 4);
}

cudaError_t launch_rows(int type, const Cache& c, const Batch& b, const Attend& a, void* ws, const DevInfo& dev,
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
