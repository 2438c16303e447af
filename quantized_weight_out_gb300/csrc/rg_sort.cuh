// rg_sort.cuh - a stable sort of indices into groups, by one block or a
// cluster of them: slots by expert, a batch's tokens by table row.
//
// Least significant digit first, at most 10 bits a pass (experts: one pass over
// whole keys).  Each warp of the cluster owns a part of the input; a walk counts
// its digits, the sums over (digit, block, warp) turn the counts into places,
// and each id goes to its digit's place and its rank there (kept from the walk
// where a warp has at most 256 ids, else found by a second walk): the result
// depends on the ids alone.  Lanes of equal digit are found by a ballot for each bit of
// it (a match instruction takes as many steps as there are different values:
// 65536 slots of 128 experts took 154 us with it and one block), so there are
// no atomics.  Blocks of a cluster read each other's counts in shared memory.
#pragma once

#include "rg_act.cuh"
#include "rg_id_launch.h"

namespace rg {
namespace id {

constexpr int SORT_MAX_WARPS = 32, SORT_THREADS = 32 * SORT_MAX_WARPS;
constexpr int SORT_BATCH = 8;  // loads in flight a lane

struct Sort {
  const int32_t* ids;
  uint2* buf[2];  // (key, position) pairs between the passes
  int32_t *order, *sorted, *start;  // start and sorted may be NULL
  int64_t n;
  int groups, passes, bits, bins;   // of a pass; one pass: bins = groups + 1
};

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The bytes of shared memory that sort_block needs: each warp's counts (rows of an odd length, so that the warps' of one
// digit lie on different banks), the block's, and the digits' places.
__host__ __device__ constexpr int sort_smem(int bins, int warps) { return (warps + 2) * (bins | 1) * 4; }
constexpr int SORT_MAX_BLOCKS = 16;

// By every thread of every block of the cluster (whole warps, a power of two of them, at most 32).  ids are read past any
// caching that a kernel before this one could have left behind (or lie in shared memory).
// Returns whether this thread saw an id of `groups` or more.
template <bool SHARED>
__device__ bool sort_block(const Sort& p, int* hist) {
  __shared__ int warp_sum[SORT_MAX_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  const int stride = p.bins | 1;
  int *tot = hist + warps * stride, *base = tot + stride;
  const int blocks = static_cast<int>(cluster_nctarank()), block = static_cast<int>(cluster_ctarank());
  // this warp's part, whole steps of 32
  const int64_t steps = (p.n + 31) / 32, per = (steps + blocks * warps - 1) / (blocks * warps);
  const int64_t lo = min(steps, per * (block * warps + warp)), hi = min(steps, lo + per);
  const unsigned below = (1u << lane) - 1u;
  int* mine = hist + warp * stride;
  bool bad = false;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const bool whole = p.passes == 1;
    const uint2* from = p.buf[(pass + 1) & 1];
    for (int i = tid; i < stride * warps; i += threads) hist[i] = 0;
    __syncthreads();
    auto digit = [&](uint2 kv) { return whole ? kv.x : (kv.x >> shift) & static_cast<uint32_t>(p.bins - 1); };
    // a batch of steps: its pairs, and of each pair the count of its digit in `mine` before it, which counts on
    auto batch = [&](int64_t s0, uint2 (&kv)[SORT_BATCH], int (&place)[SORT_BATCH]) {
#pragma unroll
      for (int u = 0; u < SORT_BATCH; ++u) {
        const int64_t i = (s0 + u) * 32 + lane;
        kv[u] = make_uint2(0u, 0u);
        if (s0 + u < hi && i < p.n) {
          if (pass == 0) {
            const int id = SHARED ? p.ids[i] : __ldcg(p.ids + i);
            bad |= id >= p.groups;
            kv[u] = make_uint2(static_cast<unsigned>(id) < static_cast<unsigned>(p.groups) ? id : p.groups,
                               static_cast<uint32_t>(i));
          } else {
            kv[u] = __ldcg(from + i);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < SORT_BATCH; ++u) {
        place[u] = -1;
        if (s0 + u >= hi) continue;
        const bool in = (s0 + u) * 32 + lane < p.n;
        const uint32_t d = digit(kv[u]);
        unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll 4
        for (int b = 0; b < p.bits; ++b) {
          const unsigned set = __ballot_sync(0xffffffffu, d >> b & 1u);
          same &= d >> b & 1u ? set : ~set;
        }
        int at = 0;
        if (in) at = mine[d];
        __syncwarp();
        // the last of the lanes of this digit counts them all
        if (in && (same >> lane) == 1u) mine[d] = at + __popc(same);
        __syncwarp();
        if (in) place[u] = at + __popc(same & below);
      }
    };
    uint2 kv[SORT_BATCH];
    int place[SORT_BATCH];
    for (int64_t s0 = lo; s0 < hi; s0 += SORT_BATCH) batch(s0, kv, place);
    __syncthreads();
    // a digit's counts of the warps: what is before a warp's, and the block's (few warps: a thread a
    // digit; many: a lane a warp, four digits at a time)
    if (warps <= 8) {
      for (int d = tid; d < p.bins; d += threads) {
        int sum = 0;
        for (int w = 0; w < warps; ++w) {
          const int c = hist[w * stride + d];
          hist[w * stride + d] = sum;
          sum += c;
        }
        tot[d] = sum;
      }
    } else {
      constexpr int U = 4;
      for (int d0 = U * warp; d0 < p.bins; d0 += U * warps) {
        int c[U], upto[U];
#pragma unroll
        for (int u = 0; u < U; ++u) upto[u] = c[u] = d0 + u < p.bins && lane < warps ? hist[lane * stride + d0 + u] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int x = __shfl_up_sync(0xffffffffu, upto[u], o);
            if (lane >= o) upto[u] += x;
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (d0 + u < p.bins) {
            if (lane < warps) hist[lane * stride + d0 + u] = upto[u] - c[u];
            if (lane == 31) tot[d0 + u] = upto[u];
          }
      }
    }
    cluster_sync();
    // places: digit by digit, block by block
    int before_all = 0;
    for (int d0 = 0; d0 < p.bins; d0 += threads) {
      const int d = d0 + tid;
      int all = 0, before = 0;
      if (d < p.bins) {
        const uint32_t at = smem_addr(tot + d);
#pragma unroll
        for (int c = 0; c < SORT_MAX_BLOCKS; ++c)
          if (c < blocks) {
            const int x = ld_cluster(mapa_shared(at, c));
            if (c < block) before += x;
            all += x;
          }
      }
      int upto = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      const int ws = lane < warps ? warp_sum[lane] : 0;
      int wu = ws;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, wu, o);
        if (lane >= o) wu += x;
      }
      const int at = before_all + upto - all + __shfl_sync(0xffffffffu, wu - ws, warp);
      before_all += __shfl_sync(0xffffffffu, wu, 31);
      if (d < p.bins) {
        if (p.start != nullptr && block == 0 && d <= p.groups) p.start[d] = at;
        base[d] = at + before;
      }
      __syncthreads();
    }
    const bool last = pass + 1 == p.passes;
    uint2* to = p.buf[pass & 1];
    auto put = [&](uint2 x, int at) {
      if (!last) {
        __stcg(to + at, x);
      } else {
        p.order[at] = static_cast<int32_t>(x.y);
        if (p.sorted != nullptr) p.sorted[at] = static_cast<int32_t>(x.x);
      }
    };
    if (hi - lo <= SORT_BATCH) {
      // one batch: its places within the warp's are at hand (registers)
#pragma unroll
      for (int u = 0; u < SORT_BATCH; ++u)
        if (lo + u < hi && place[u] >= 0) put(kv[u], base[digit(kv[u])] + mine[digit(kv[u])] + place[u]);
    } else {
      for (int64_t s0 = lo; s0 < hi; s0 += SORT_BATCH) {
        batch(s0, kv, place);
#pragma unroll
        for (int u = 0; u < SORT_BATCH; ++u)
          if (place[u] >= 0) put(kv[u], base[digit(kv[u])] + place[u]);
      }
    }
    if (!last) __threadfence();
    cluster_sync();  // the pairs are written; no block's counts are read any more
  }
  return bad;
}

// Keys are 0 .. groups: the bits of a key, passes and bits a pass.
inline void sort_plan(int64_t groups, bool start, Sort* p) {
  int b = 1;
  while ((groups >> b) != 0) ++b;
  p->passes = start || b <= 10 ? 1 : (b + 9) / 10;
  p->bits = (b + p->passes - 1) / p->passes;
  p->bins = p->passes == 1 ? static_cast<int>(groups) + 1 : 1 << p->bits;
}
constexpr int kSortMostSmem = sort_smem(kMaxExperts + 1, SORT_MAX_WARPS);

}  // namespace id
}  // namespace rg
