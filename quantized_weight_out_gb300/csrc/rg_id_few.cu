// rg_id_few.cu - the forward by slot where each expert has a few slots (a
// decoding batch): the chosen experts' rows are streamed once.
//
// The bytes of W bound it.  A work item is a chunk of up to ns slots of one
// expert and a strip of 16 wr rows of its W: y[rows x ns] = W x^T as warp-level
// MMAs (m16n8k16, W the row operand), 16 rows to a group of wk warps that share
// the contraction (wr wk = 8).  Blocks are persistent and take equal runs of
// the items, an expert's strips of rows one after another: a producer warp
// copies boxes of row pieces into a ring of stages ahead of the consumers, so the
// stream does not pause between items (by TMA boxes: a bulk copy for each row's
// piece costs about 30 ns an SM); the chunk's rows of X lie in shared memory as
// 16-bit operands, scaled by a power of two a row as the tile route's copies
// are, and change once an expert.
// The operands of the common types are the weights' integers (or E2M1 codes)
// themselves, exact in fp16, and a block's scale multiplies the MMA's F32 sums
// of its 16 or 32 values: fewer instructions a weight than scaling the operand,
// and no rounding of W.  (Every value decoded to F32 and rounded to fp16 took 61
// us for 66 MB of Q4_K, bound by its 180 instructions for 512 values.)  The
// contraction's order inside an MMA is free: X is stored in the order in which
// a lane finds its eight weights of a block, one 16-byte read.  The warps' sums
// of an item meet in shared memory in a fixed order.
#include <algorithm>

#include "rg_act.cuh"
#include "rg_id_launch.h"
#include "rg_raw.cuh"

namespace rg {
namespace id {

namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;  // consumers; one more warp copies

struct Few {
  Batch b;
  const void* W;
  int64_t N, rb;
  int K;
  const void* in;
  int64_t in_row;
  int in_tokens, atype;
  int ns, cap, stages, xstride;  // slots a chunk, chunks at most, ring stages, bytes of a row of X
  int wk, wr;                    // warps along the contraction and groups of 16 rows: wk wr = 8
  int pv, rs;                    // values of a row in a stage, bytes from row to row there
  const float* weights;
  void* out;
  int64_t out_row;
  int otype;
  float beta;
  uint8_t* live;
  WaitCtl ctl;
};

struct Chunk {
  int expert, first, rows;
};

// All consumer warps; the `threads` of group `id`.
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); }
__device__ __forceinline__ void bar_group(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(2 + id), "r"(threads) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void load_row8(const void* row, int atype, int at, float (&v)[8]) {
  if (atype == RG_F32) load_act8<RG_F32>(row, at, v);
  else if (atype == RG_BF16) load_act8<RG_BF16>(row, at, v);
  else load_act8<RG_F16>(row, at, v);
}

// How a 32-value block of X lies in shared memory: lane t of a quad has 16 bytes, four values for the first MMA of 16,
// then four for the second.  SPLIT: they are values 4t .. and 16 + 4t .. (types whose nibbles or scales go by halves of
// 16), else 8t .. 8t + 7.  CROSS: of four values the pairs are (0, 2) and (1, 3) (nibbles masked out of a word in
// place), else (0, 1) and (2, 3).
template <int WT>
constexpr bool x_split() { return WT == RG_Q4_0 || WT == RG_MXFP4 || WT == RG_Q6_K; }
template <int WT>
constexpr bool x_cross() { return WT == RG_Q4_0 || WT == RG_Q4_K; }
// Types whose nibbles are used in place, as the fp16 subnormals q 2^-24: their sums are 2^-24 of the values', and with
// them the sums of X's blocks of 32 that join them (for a minimum, or q - 8); the row's sum is multiplied by 2^24.
template <int WT>
constexpr bool x_sums() { return WT == RG_Q4_0 || WT == RG_Q4_K; }

__device__ __forceinline__ uint32_t h2sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The bytes u0, u1 (u2, u3) of x as fp16 pairs 1024 + u (0x6400: 1024, whose last place is 1), less `bias`.
__device__ __forceinline__ void bytes_to_h2(uint32_t x, uint32_t bias, uint32_t& lo, uint32_t& hi) {
  lo = h2sub(__byte_perm(x, 0x64646464u, 0x5140), bias);
  hi = h2sub(__byte_perm(x, 0x64646464u, 0x7362), bias);
}
// Four E2M1 codes in the low nibbles of x's bytes as fp16 pairs, exactly: their high bytes by a lookup.
__device__ __forceinline__ void e2m1_to_h2(uint32_t x, uint32_t& lo, uint32_t& hi) {
  const uint32_t m = x & 0x07070707u, u = m | (m >> 4);
  const uint32_t sel = (u & 0xFFu) | ((u >> 8) & 0xFF00u);
  const uint32_t hb = __byte_perm(0x3E3C3800u, 0x46444240u, sel) | ((x & 0x08080808u) << 4);
  lo = __byte_perm(hb, 0u, 0x1404);
  hi = __byte_perm(hb, 0u, 0x3424);
}
// The word at byte `at` of p, which is aligned to 4: 4, 2 or 1 byte steps by aligned loads.
__device__ __forceinline__ uint32_t word_at(const uint8_t* p, int at) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p + (at & ~3));
  return (at & 3) == 0 ? w[0] : __funnelshift_r(w[0], w[1], 8 * (at & 3));
}
__device__ __forceinline__ uint32_t word_2(const uint8_t* p) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
  return h[0] | static_cast<uint32_t>(h[1]) << 16;
}

// One lane's view of the chunk's X: its row (column of the MMA) of each group of eight slots.
template <int NT>
struct XView {
  const uint8_t* row[NT];
  const float* sums;  // [block of 32][8 NT], at this lane's two columns
  __device__ __forceinline__ uint4 at(int j, int k) const { return *reinterpret_cast<const uint4*>(row[j] + 2 * k); }
  __device__ __forceinline__ float2 sum(int j, int k) const {
    return *reinterpret_cast<const float2*>(sums + (k >> 5) * (8 * NT) + 8 * j);
  }
};

// acc (rows g and g + 8, two columns) += the granule's 128 values: r0 and r1 point at the 256-value tile of the two
// rows, h says which half; k is the granule's first value in the row, `values` how many the row still has.
template <int WT, int NT>
__device__ __forceinline__ void granule(float (&acc)[NT][4], const uint8_t* r0, const uint8_t* r1, int h, int t, int k,
                                        int values, const XView<NT>& x) {
  __builtin_assume(__isShared(r0));
  __builtin_assume(__isShared(r1));
  __builtin_assume(__isShared(x.sums));
#pragma unroll
  for (int j = 0; j < NT; ++j) __builtin_assume(__isShared(x.row[j]));
  const uint8_t* const r[2] = {r0, r1};
  // acc += s[0], s[1] times the sums of one 32-value block (two MMAs), its operands a[row][word]
  auto block = [&](const uint32_t (&a)[2][4], const float (&s)[2], int kb) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint4 b = x.at(j, kb);
      float d[4] = {0, 0, 0, 0};
      mma<false>(d, a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
      mma<false>(d, a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(s[i >> 1], d[i], acc[j][i]);
    }
  };
  if constexpr (WT == RG_F16 || WT == RG_BF16) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int v0 = 32 * u;
      if (v0 >= values) break;
      uint32_t a[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (v0 + 8 * t < values) q = *reinterpret_cast<const uint4*>(r[i] + 256 * h + 2 * (v0 + 8 * t));
        a[i][0] = q.x; a[i][1] = q.y; a[i][2] = q.z; a[i][3] = q.w;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 b = x.at(j, k + v0);
        mma<WT == RG_BF16>(acc[j], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
        mma<WT == RG_BF16>(acc[j], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
      }
    }
  } else if constexpr (WT == RG_Q8_0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t a[2][4];
      float s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* p = r[i] + 136 * h;
        s[i] = f16_to_f32(ld_u16(p + 34 * u));
        bytes_to_h2(word_at(p + 8 * t, 34 * u + 2) ^ 0x80808080u, 0x64806480u, a[i][0], a[i][1]);
        bytes_to_h2(word_at(p + 8 * t, 34 * u + 6) ^ 0x80808080u, 0x64806480u, a[i][2], a[i][3]);
      }
      block(a, s, k + 32 * u);
    }
  } else if constexpr (WT == RG_MXFP4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t a[2][4];
      float s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* p = r[i] + 68 * h;
        s[i] = e8m0_f32(p[17 * u]);
        const uint32_t q = word_at(p + 4 * t, 17 * u + 1);
        e2m1_to_h2(q & 0x0F0F0F0Fu, a[i][0], a[i][1]);
        e2m1_to_h2((q >> 4) & 0x0F0F0F0Fu, a[i][2], a[i][3]);
      }
      block(a, s, k + 32 * u);
    }
  } else if constexpr (WT == RG_Q4_0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t a[2][4];
      float s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* p = r[i] + 72 * h + 18 * u;
        s[i] = f16_to_f32(ld_u16(p));
        const uint32_t q = word_2(p + 2 + 4 * t);
        a[i][0] = q & 0x000F000Fu;
        a[i][1] = (q >> 8) & 0x000F000Fu;
        a[i][2] = (q >> 4) & 0x000F000Fu;
        a[i][3] = (q >> 12) & 0x000F000Fu;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 b = x.at(j, k + 32 * u);
        const float2 sx = x.sum(j, k + 32 * u);
        constexpr float C = -8.0f;  // q - 8
        float d[4] = {C * sx.x, C * sx.y, C * sx.x, C * sx.y};
        mma<false>(d, a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
        mma<false>(d, a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(s[i >> 1], d[i], acc[j][i]);
      }
    }
  } else if constexpr (WT == RG_Q4_K) {
    // lane t of a quad: the 6-bit scale and minimum of the granule's sub-block t, of both rows, as an fp16 pair
    uint32_t scm[2];
    float d[2], dmin[2];
    uint2 q[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 hd = *reinterpret_cast<const uint4*>(r[i]);
      const uint32_t ab = __byte_perm(hd.y, hd.z, t | (4 + t) << 4);  // bytes t and 4 + t of the twelve
      const uint32_t c = hd.w >> (8 * t);
      const uint32_t six = h == 0 ? ab & 0x3F3Fu : (c & 0x0Fu) | ((c << 4) & 0x0F00u) | ((ab >> 2) & 0x3030u);
      scm[i] = h2sub(__byte_perm(six, 0x64646464u, 0x4140), 0x64006400u);
      d[i] = f16_to_f32(static_cast<uint16_t>(hd.x & 0xFFFFu));
      dmin[i] = -f16_to_f32(static_cast<uint16_t>(hd.x >> 16));
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2)
        q[i][c2] = *reinterpret_cast<const uint2*>(r[i] + 16 + 64 * h + 32 * c2 + 8 * t);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t a[2][4];
      float s[2], n[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t p = __shfl_sync(0xffffffffu, scm[i], u, 4);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
        s[i] = (u & 1 ? d[i] * 0.0625f : d[i]) * f.x;
        n[i] = dmin[i] * f.y;
        // (high nibbles where they are: 16 times as large)
        const uint2 w = q[i][u >> 1];
        const uint32_t m = u & 1 ? 0x00F000F0u : 0x000F000Fu;
        a[i][0] = w.x & m;
        a[i][1] = (w.x >> 8) & m;
        a[i][2] = w.y & m;
        a[i][3] = (w.y >> 8) & m;
      }
      block(a, s, k + 32 * u);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float2 sx = x.sum(j, k + 32 * u);
        acc[j][0] = fmaf(n[0], sx.x, acc[j][0]);
        acc[j][1] = fmaf(n[0], sx.y, acc[j][1]);
        acc[j][2] = fmaf(n[1], sx.x, acc[j][2]);
        acc[j][3] = fmaf(n[1], sx.y, acc[j][3]);
      }
    }
  } else if constexpr (WT == RG_Q6_K) {
    // value 32 i + l of the half: the low (i < 2) or high nibble of ql[32 (i % 2) + l], two bits of qh[l]; a scale for
    // each 16 values, so the two MMAs of a block are scaled apart
    uint32_t ql[2][2][2], qh[2][2];
    float d[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      d[i] = f16_to_f32(ld_u16(r[i] + 208));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qh[i][e] = word_2(r[i] + 128 + 32 * h + 16 * e + 4 * t);
#pragma unroll
        for (int f = 0; f < 2; ++f) ql[i][f][e] = word_2(r[i] + 64 * h + 32 * f + 16 * e + 4 * t);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t a[2][2];
        float s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[i] = d[i] * static_cast<float>(static_cast<int8_t>(r[i][192 + 8 * h + 2 * u + e]));
          const uint32_t v = ((ql[i][u & 1][e] >> (4 * (u >> 1))) & 0x0F0F0F0Fu) | (((qh[i][e] >> (2 * u)) & 0x03030303u) << 4);
          bytes_to_h2(v, 0x64206420u, a[i][0], a[i][1]);  // 1024 + 32
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint2 b = *reinterpret_cast<const uint2*>(x.row[j] + 2 * (k + 32 * u) + 8 * e);
          float p[4] = {0, 0, 0, 0};
          mma<false>(p, a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(s[i >> 1], p[i], acc[j][i]);
        }
      }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t a[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        smt::Raw<WT> raw;
        smt::load_raw_smem<WT>(r[i], 16 * h + 4 * u + t, raw);
        float f[8];
        smt::decode_raw<WT>(raw, 16 * h + 4 * u + t, f);
#pragma unroll
        for (int w = 0; w < 4; ++w) a[i][w] = pack16<false>(f[2 * w], f[2 * w + 1]);
      }
      const float one[2] = {1.0f, 1.0f};
      block(a, one, k + 32 * u);
    }
  }
}

template <int WT, int NT>
__global__ void __launch_bounds__(THREADS + 32, 2) few_kernel(const __grid_constant__ CUtensorMap map, Few f) {
  constexpr bool BF16 = WT == RG_BF16;
  constexpr int COLS = 8 * NT, RED = COLS * 17;
  const int PV = f.pv, RS = f.rs, strip = 16 * f.wr, SB = strip * RS;
  const int piece_bytes = PV / 256 * smt::tile_bytes<WT>();
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* ring = sm;
  const uint32_t box = static_cast<uint32_t>(SB);
  uint8_t* xs = ring + f.stages * SB;
  float* red = reinterpret_cast<float*>(xs + f.ns * f.xstride);        // [2][warp][column][row], 17 apart
  float* sums = red + 2 * WARPS * RED;                                     // [block of 32][column]
  Chunk* chunks = reinterpret_cast<Chunk*>(sums + (x_sums<WT>() ? (f.K + 31) / 32 * COLS : 0));  // [cap]
  __shared__ uint64_t bars[16];                                         // full, empty: up to eight stages
  __shared__ int s_warp[WARPS + 1], s_base, s_abort, s_slot[COLS], s_top[COLS];
  __shared__ float s_mul[COLS], s_weight[COLS];  // what undoes a row's power of two; the slot's weight
  __shared__ const char* s_from[COLS];
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (8 + s); };
  if (tid == 0) {
    for (int s = 0; s < f.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), WARPS);
    }
    s_abort = 0;
    s_base = 0;
    fence_mbar_init();
    tma_prefetch_map(&map);
  }
  // (every entry of order is looked at by some block; the load is under way while start is read)
  int at_order = static_cast<int>(blockIdx.x) * (THREADS + 32) + tid;
  int named = at_order < f.b.slots ? __ldg(f.b.order + at_order) : 0;
  // the chunks: a running sum of the experts'
  __syncthreads();
  for (int e0 = 0; e0 < f.b.experts; e0 += THREADS + 32) {
    const int e = e0 + tid;
    int first = 0, rows = 0;
    if (e < f.b.experts) {
      const int lo = __ldg(f.b.start + e), hi = __ldg(f.b.start + e + 1);
      if (lo < 0 || hi < lo || hi > f.b.slots) report_index(f.ctl.status);
      else first = lo, rows = hi - lo;
    }
    const int mine = (rows + f.ns - 1) / f.ns;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int at = s_base + upto - mine;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    if (at + mine > f.cap) report_index(f.ctl.status);  // (ranges that overlap)
    for (int i = 0; i < mine && at + i < f.cap; ++i)
      chunks[at + i] = Chunk{e, first + i * f.ns, min(f.ns, rows - i * f.ns)};
    __syncthreads();
    if (tid == THREADS + 31) s_base = at + mine;
    __syncthreads();
  }
  while (at_order < f.b.slots) {
    if (static_cast<unsigned>(named) >= static_cast<unsigned>(f.b.slots)) report_index(f.ctl.status);
    at_order += static_cast<int>(gridDim.x) * (THREADS + 32);
    named = at_order < f.b.slots ? __ldg(f.b.order + at_order) : 0;
  }
  const int n_chunks = min(f.cap, s_base);
  const int N = static_cast<int>(f.N), strips = (N + strip - 1) / strip, pieces = (f.K + PV - 1) / PV;
  const int64_t items = static_cast<int64_t>(n_chunks) * strips;
  const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
  // the items one after another: chunk c, the strip from row n on
  int c = static_cast<int>(i0 / max(1, strips)), n = static_cast<int>(i0 - static_cast<int64_t>(c) * strips) * strip;
  auto advance = [&] {
    n += strip;
    if (n >= N) {
      n = 0;
      ++c;
    }
  };
  if (blockIdx.x == 0 && f.live != nullptr) {
    // the slots of the chunks, and no others: rows of slots outside them are not written
    for (int i = tid; i < f.b.slots; i += THREADS + 32) f.live[i] = 0;
    __syncthreads();
    for (int i = tid; i < n_chunks * f.ns; i += THREADS + 32) {
      const Chunk ch = chunks[i / f.ns];
      const int r = i % f.ns;
      if (r >= ch.rows) continue;
      const int s = __ldg(f.b.order + ch.first + r);
      if (static_cast<unsigned>(s) < static_cast<unsigned>(f.b.slots)) f.live[s] = 1;
    }
  }

  if (warp == WARPS) {
    // ---------------- the copies ----------------
    if (lane != 0) return;
    int s = 0;
    uint32_t ph = 0, pend = 0, pend_ph = 0;
    bool ok = true;
    for (int left = static_cast<int>(i1 - i0); ok && left > 0; --left, advance()) {
      const int expert = chunks[c].expert;
      for (int p = 0; p < pieces; ++p) {
        ok = mbar_wait(empty(s), ph ^ 1u, f.ctl, abort_flag);
        if (!ok) break;
        mbar_arrive_expect_tx(full(s), box);
        // from the 16-byte grain that the piece begins in
        tma_load_3d(smem_addr(ring + s * SB), &map, full(s), ((p * piece_bytes) & ~15) / 4, n, expert);
        pend |= 1u << s;
        pend_ph = (pend_ph & ~(1u << s)) | (ph << s);
        if (++s == f.stages) { s = 0; ph ^= 1u; }
      }
    }
    // every copy started lands before the block leaves
    volatile int no_abort = 0;
    for (int st = 0; st < f.stages; ++st)
      if (pend & (1u << st)) (void)mbar_wait(full(st), (pend_ph >> st) & 1u, f.ctl, &no_abort);
    return;
  }

  // ---------------- the consumers ----------------
  // (a wait that gave up is reported; the warp then goes on without waiting, for the barriers' sake)
  const int g = lane >> 2, t = lane & 3, wk = warp % f.wk, wr = warp / f.wk;
  int s = 0, at_chunk = -1, count = 0, par = 0;
  uint32_t ph = 0;
  bool ok = true;
  XView<NT> x;
  x.sums = sums + 2 * t;
  for (int left = static_cast<int>(i1 - i0); left > 0; --left, par ^= 1, advance()) {
    const int n0 = n + 16 * wr;
    if (c != at_chunk) {
      // the chunk's rows of X, once no warp reads the old ones any more: 256 values a warp and step,
      // first for each row's largest magnitude, then (from the L1 cache) to be stored
      if (at_chunk >= 0) bar_consumers();
      const Chunk ch = chunks[c];
      at_chunk = c;
      count = ch.rows;
      if (tid < count) {
        int slot = __ldg(f.b.order + ch.first + tid);
        if (static_cast<unsigned>(slot) >= static_cast<unsigned>(f.b.slots)) slot = -1;
        s_slot[tid] = slot;
        slot = max(slot, 0);
        s_from[tid] = static_cast<const char*>(f.in) +
                      static_cast<int64_t>(f.in_tokens ? slot / f.b.per_token : slot) * f.in_row * act_bytes(f.atype);
        s_mul[tid] = 1.0f;
        s_weight[tid] = f.weights != nullptr ? __ldg(f.weights + slot) : 1.0f;
        s_top[tid] = 0;
      }
      bar_consumers();
      const int segs = (f.K + 255) / 256;
      // U steps' loads in flight; what a warp's lanes hold of step o: row r, values k .. k + 7
      constexpr int U = 2;
      const int steps = count * segs;
      float v[U][8];
      auto fetch = [&](int o0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int o = min(o0 + u * WARPS, steps - 1), r = o / segs, k = 256 * (o - r * segs) + 8 * lane;
          load_row8(s_from[r], f.atype, min(k, f.K - 8), v[u]);
        }
      };
      if constexpr (!BF16) {
        for (int o0 = warp; o0 < steps; o0 += U * WARPS) {
          fetch(o0);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int o = o0 + u * WARPS;
            float top = 0.0f;  // (lanes past the row's end hold its last values again)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[u][j]));
            const int most = __reduce_max_sync(0xffffffffu, __float_as_int(top));  // (not negative: ordered as an integer)
            if (lane == 0 && o < steps) atomicMax(&s_top[o / segs], most);
          }
        }
        bar_consumers();
      }
      for (int o0 = warp; o0 < steps; o0 += U * WARPS) {
        fetch(o0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int o = o0 + u * WARPS;
          if (o >= steps) break;
          const int r = o / segs, k = 256 * (o - r * segs) + 8 * lane;
          if (!x_sums<WT>() && k >= (f.K + 31) / 32 * 32) continue;
          float w8[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w8[j] = k < f.K ? v[u][j] : 0.0f;
          if constexpr (!BF16) {
            const int shift = row_shift(__int_as_float(s_top[r]));
            const float mul = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j) w8[j] *= mul;
            if (k == 0) s_mul[r] = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
          }
          uint8_t* to = xs + r * f.xstride;
          // two groups of four values of the block: group q goes to its lane's first or second eight bytes
          const int l = (k >> 3) & 3;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int q = 2 * l + e, at = x_split<WT>() ? 16 * (q & 3) + 8 * (q >> 2) : 8 * q;
            const float* w = w8 + 4 * e;
            const uint2 two = x_cross<WT>() ? make_uint2(pack16<BF16>(w[0], w[2]), pack16<BF16>(w[1], w[3]))
                                            : make_uint2(pack16<BF16>(w[0], w[1]), pack16<BF16>(w[2], w[3]));
            *reinterpret_cast<uint2*>(to + 2 * (k & ~31) + at) = two;
          }
          if constexpr (x_sums<WT>()) {
            // the block's sum, of the values as they are rounded (K is a multiple of 256: whole warps)
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += __half2float(__float2half_rn(w8[j]));
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (l == 0) sums[(k >> 5) * COLS + r] = sum * 0x1p-24f;
          }
        }
      }
      bar_consumers();
      // (columns past the chunk's slots repeat its last row, and are not stored)
#pragma unroll
      for (int j = 0; j < NT; ++j) x.row[j] = xs + min(8 * j + g, count - 1) * f.xstride + 16 * t;
    }
    float acc[NT][4] = {};
    for (int p = 0; p < pieces; ++p) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(full(s), ph, f.ctl, abort_flag));
      const int values = min(PV, f.K - p * PV);
      const uint8_t* stage = ring + s * SB + (16 * wr + g) * RS + ((p * piece_bytes) & 15);
      for (int v1 = 128 * wk; ok && v1 < values; v1 += 128 * f.wk) {
        const uint8_t* tile = stage + (v1 >> 8) * smt::tile_bytes<WT>();
        granule<WT, NT>(acc, tile, tile + 8 * RS, (v1 >> 7) & 1, t, p * PV + v1, values - v1, x);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
      if (++s == f.stages) { s = 0; ph ^= 1u; }
    }
    // the warps' sums: rows g and g + 8, columns 2t and 2t + 1 of each group of eight slots
    // (two buffers: a warp fills the next one when its group has met for this one)
    float* mine = red + (par * WARPS + warp) * RED;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* q = mine + (8 * j + 2 * t) * 17 + g;
      q[0] = acc[j][0];
      q[17] = acc[j][1];
      q[8] = acc[j][2];
      q[25] = acc[j][3];
    }
    if (f.wk > 1) bar_group(wr, 32 * f.wk);
    else __syncwarp();
    const float* first = red + (par * WARPS + wr * f.wk) * RED;
    for (int o = 32 * wk + lane; o < 16 * count; o += 32 * f.wk) {
      const int row = o & 15, col = o >> 4, slot = s_slot[col];
      if (slot < 0 || n0 + row >= N) continue;
      float v = 0.0f;
      for (int w = 0; w < f.wk; ++w) v += first[w * RED + col * 17 + row];
      // (one after another: the factors' product can pass F32's range where the result does not)
      if (x_sums<WT>()) v *= 0x1p24f;
      v = v * s_mul[col] * s_weight[col];
      char* to = static_cast<char*>(f.out) + static_cast<int64_t>(slot) * f.out_row * act_bytes(f.otype);
      if (f.beta != 0.0f) v = fmaf(f.beta, load_act(to, f.otype, n0 + row), v);
      store_act(to, f.otype, n0 + row, v);
    }
    if (f.wk == 1) __syncwarp();
  }
}

// Bytes of a row of X in shared memory: 64 off a multiple of 128 apart, so that two rows' 16-byte reads of a quarter
// warp fall on different banks.
int64_t x_stride(int64_t K) { return (K * 2 + 127) / 128 * 128 + 64; }

template <int WT, int NT>
cudaError_t launch_few_t(Few f, const DevInfo& dev, cudaStream_t stream) {
  const int fixed = f.ns * f.xstride + 2 * WARPS * 8 * NT * 17 * 4 + f.cap * static_cast<int>(sizeof(Chunk)) +
                    (x_sums<WT>() ? (f.K + 31) / 32 * 8 * NT * 4 : 0);
  const int half = 108 * 1024, whole = 220 * 1024;
  // A stage's rows lie an odd multiple of 32 bytes apart: four rows' eight-byte reads fall on
  // different banks.  (A piece may begin inside a 16-byte grain.)
  const int tile = smt::tile_bytes<WT>();
  auto stride = [&](int tiles) {
    const int bytes = tiles * tile;
    return (bytes + (bytes % 16 ? 14 : 0) + 31) / 64 * 64 + 32;
  };
  // A strip's rows: the warps along the contraction (and the meetings of an item) halve while the
  // items stay two for each of the two blocks an SM and a stage of one tile a row is no more
  // than 28 KB.
  const int64_t chunks = std::min<int64_t>(f.cap, std::max<int64_t>(1, f.b.slots / f.ns));
  f.wr = 1;
  while (f.wr < WARPS && 32 * f.wr * stride(1) <= 28 * 1024 &&
         chunks * ((f.N + 32 * f.wr - 1) / (32 * f.wr)) >= 4 * dev.num_sms)
    f.wr *= 2;
  f.wk = WARPS / f.wr;
  // tiles of a row in a stage: up to four, a box's row at most 1024 bytes, a stage of about 20 KB
  int tiles = std::min(4, (f.K + 255) / 256);
  while (tiles > 1 && (stride(tiles) > 1024 || 16 * f.wr * stride(tiles) > 24 * 1024)) --tiles;
  f.pv = 256 * tiles;
  f.rs = stride(tiles);
  const int stage = 16 * f.wr * f.rs;
  // two blocks an SM where both get three stages, else one; as many stages as fit, at most eight
  const bool two = fixed + 3 * stage <= half;
  f.stages = std::min(8, ((two ? half : whole) - fixed) / stage);
  if (f.stages < 2) return cudaErrorInvalidValue;
  auto kern = few_kernel<WT, NT>;
  const int smem = fixed + f.stages * stage;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), whole);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (encode_tiled(&map, CU_TENSOR_MAP_DATA_TYPE_UINT32, f.W, static_cast<uint64_t>(f.rb / 4),
                   static_cast<uint64_t>(f.N), static_cast<uint64_t>(f.rb), static_cast<uint32_t>(f.rs / 4),
                   static_cast<uint32_t>(16 * f.wr), CU_TENSOR_MAP_SWIZZLE_NONE,
                   static_cast<uint64_t>(f.b.experts), static_cast<uint64_t>(f.N * f.rb)) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  kern<<<dev.num_sms * (two ? 2 : 1), THREADS + 32, smem, stream>>>(map, f);
  return counted(cudaGetLastError());
}

}  // namespace

constexpr int64_t X_ROOM = 96 * 1024;  // what a chunk's rows of X take at most

int few_rows(int64_t K) { return static_cast<int>(std::min<int64_t>(8, X_ROOM / x_stride(K))); }

// Whether a type has chunks of two MMAs' columns: those that stream more than five slots an expert.
constexpr bool two_mmas(int wtype) { return wtype == RG_Q6_K || wtype == RG_Q3_K; }

// Slots a chunk: one MMA's eight, or two's where an expert has more than five on average (40 tokens,
// 5 slots an expert of 64: 50 us with eight, 59 with sixteen), no more than there are tokens, while
// the rows of X fit.
int few_slots(const Batch& b, const Product& p) {
  const int64_t avg = (b.slots + std::min(b.experts, b.slots) - 1) / std::min(b.experts, b.slots);
  const int64_t want = std::min<int64_t>(avg > 5 && two_mmas(p.wtype) ? 16 : 8, b.slots / b.per_token);
  return static_cast<int>(std::min<int64_t>(want, X_ROOM / x_stride(p.K)));
}

bool few_fits(const Batch& b, const Product& p) {
  const int ns = few_slots(b, p);
  return p.fwd && ns >= 1 && p.N <= (1 << 30) && max_tiles(b.slots, b.experts, ns) <= 1024;
}

cudaError_t launch_few(const Product& p, const Batch& b, const Slots& s, const DevInfo& dev, cudaStream_t stream) {
  Few f{};
  f.b = b;
  f.W = p.W;
  f.N = p.N;
  f.K = static_cast<int>(p.K);
  f.rb = padded_row_bytes(p.wtype, p.K);
  f.in = p.in;
  f.in_row = p.in_row;
  f.in_tokens = p.in_tokens ? 1 : 0;
  f.atype = p.atype;
  f.ns = few_slots(b, p);
  f.cap = static_cast<int>(max_tiles(b.slots, b.experts, f.ns));
  f.xstride = static_cast<int>(x_stride(p.K));
  f.weights = s.weights;
  f.out = s.out;
  f.out_row = s.out_row;
  f.otype = s.otype;
  f.beta = s.beta;
  f.live = s.live;
  f.ctl = WaitCtl{dev.status, dev.wait_limit_ns};
  return with_wtype(p.wtype, cudaErrorInvalidValue, [&](auto wt) {
    constexpr int WT = decltype(wt)::value;
    if constexpr (WT == RG_F32) {
      return cudaErrorInvalidValue;
    } else {
      if constexpr (two_mmas(WT))
        if (f.ns > 8) return launch_few_t<WT, 2>(f, dev, stream);
      return launch_few_t<WT, 1>(f, dev, stream);
    }
  });
}

}  // namespace id
}  // namespace rg
