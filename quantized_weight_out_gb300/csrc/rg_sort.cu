// rg_sort.cu - a stable sort of indices into groups: slots by expert, a
// batch's tokens by table row.
//
// One block, least significant digit first, at most 10 bits a pass (one pass
// for experts).  Warp w owns the w-th part of the input; a first walk counts
// its digits (lanes of equal digit found by a match, so no atomics), a sum over
// (digit, warp) turns the counts into places, and a second walk hands the
// places out in order: the result depends on the ids alone.
//
// The bound is latency: the walks' loads (eight in flight a lane) and the
// match chains.
#include <algorithm>

#include "rg_act.cuh"
#include "rg_id_launch.h"

namespace rg {
namespace id {

namespace {

constexpr int WARPS = 32, THREADS = 32 * WARPS;
constexpr int MAX_BINS = 1 << 10;
constexpr int BATCH = 8;

struct Pass {
  const int32_t* ids;   // the first pass: key of i is ids[i]
  const uint2* from;    // later ones: (key, position) pairs
  uint2* to;            // every one but the last
  int32_t *order, *sorted, *start;  // the last (start: the only) one; sorted and start may be NULL
  int n, groups, shift, bins;
};

__global__ void __launch_bounds__(THREADS, 1) sort_pass_kernel(Pass p, int* status) {
  extern __shared__ int hist[];  // [WARPS][bins]
  __shared__ int warp_sum[WARPS];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < p.bins * WARPS; i += THREADS) hist[i] = 0;
  __syncthreads();
  // this warp's part, whole steps of 32
  const int64_t steps = (p.n + 31ll) / 32, per = (steps + WARPS - 1) / WARPS;
  const int64_t lo = min(steps, per * warp), hi = min(steps, lo + per);
  const unsigned below = (1u << lane) - 1u;
  bool bad = false;
  auto walk = [&](auto&& each) {
    for (int64_t s0 = lo; s0 < hi; s0 += BATCH) {
      uint2 kv[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int64_t i = (s0 + u) * 32 + lane;
        kv[u] = make_uint2(0u, 0u);
        if (s0 + u < hi && i < p.n) {
          if (p.ids != nullptr) {
            const int id = __ldcg(p.ids + i);
            bad |= id >= p.groups;
            kv[u] = make_uint2(static_cast<unsigned>(id) < static_cast<unsigned>(p.groups) ? id : p.groups,
                               static_cast<uint32_t>(i));
          } else {
            kv[u] = p.from[i];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u)
        if (s0 + u < hi) {
          const bool in = (s0 + u) * 32 + lane < p.n;
          const int d = in ? static_cast<int>((kv[u].x >> p.shift) & static_cast<uint32_t>(p.bins - 1)) : -1;
          each(kv[u], p.start != nullptr && in ? static_cast<int>(kv[u].x) : d, in);
        }
    }
  };
  walk([&](uint2, int d, bool in) {
    const unsigned same = __match_any_sync(0xffffffffu, d);
    if (in && (same & below) == 0) hist[warp * p.bins + d] += __popc(same);
    __syncwarp();
  });
  __syncthreads();
  // places: digit by digit, warp by warp
  int base = 0;
  for (int d0 = 0; d0 < p.bins; d0 += THREADS) {
    const int d = d0 + tid;
    int mine = 0;
    if (d < p.bins)
      for (int w = 0; w < WARPS; ++w) mine += hist[w * p.bins + d];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int at = base + upto - mine, all = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) at += warp_sum[w];
      all += warp_sum[w];
    }
    if (d < p.bins) {
      if (p.start != nullptr && d <= p.groups) p.start[d] = at;
      for (int w = 0; w < WARPS; ++w) {
        const int c = hist[w * p.bins + d];
        hist[w * p.bins + d] = at;
        at += c;
      }
    }
    base += all;
    __syncthreads();
  }
  walk([&](uint2 kv, int d, bool in) {
    const unsigned same = __match_any_sync(0xffffffffu, d);
    int at = 0;
    if (in) at = hist[warp * p.bins + d] + __popc(same & below);
    __syncwarp();
    if (in && (same & below) == 0) hist[warp * p.bins + d] = at + __popc(same);
    __syncwarp();
    if (in) {
      if (p.to != nullptr) {
        p.to[at] = kv;
      } else {
        p.order[at] = static_cast<int32_t>(kv.y);
        if (p.sorted != nullptr) p.sorted[at] = static_cast<int32_t>(kv.x);
      }
    }
  });
  if (bad) report_index(status);
}

// Keys are 0 .. groups: bits, passes and bits a pass.
int passes_of(int64_t groups, int* bits) {
  int b = 1;
  while ((groups >> b) != 0) ++b;
  const int n = (b + 9) / 10;
  *bits = (b + n - 1) / n;
  return n;
}

}  // namespace

size_t sort_workspace(int64_t n, int64_t groups) {
  int bits;
  const int passes = groups <= kMaxExperts ? 1 : passes_of(groups, &bits);
  return static_cast<size_t>(passes > 2 ? 2 : passes - 1) * static_cast<size_t>(up256(n * 8));
}

cudaError_t launch_sort(const int32_t* ids, int64_t n, int64_t groups, int32_t* start, int32_t* order,
                        int32_t* sorted, void* ws, const DevInfo& dev, cudaStream_t stream) {
  int bits = 0;
  const int passes = groups <= kMaxExperts ? 1 : passes_of(groups, &bits);
  uint2* buf[2] = {static_cast<uint2*>(ws), reinterpret_cast<uint2*>(static_cast<char*>(ws) + up256(n * 8))};
  for (int i = 0; i < passes; ++i) {
    Pass p{};
    p.n = static_cast<int>(n);
    p.groups = static_cast<int>(groups);
    p.ids = i == 0 ? ids : nullptr;
    p.from = i == 0 ? nullptr : buf[(i - 1) & 1];
    p.to = i == passes - 1 ? nullptr : buf[i & 1];
    p.order = order;
    p.sorted = sorted;
    p.shift = passes == 1 ? 0 : i * bits;
    p.start = start;
    if (passes == 1) {
      // one pass over whole keys (0 .. groups): as many bins, a power of two or not
      p.bins = start != nullptr ? static_cast<int>(groups) + 1 : 1;
      while (start == nullptr && p.bins <= groups) p.bins *= 2;
    } else {
      p.bins = 1 << bits;
    }
    const int smem = p.bins * WARPS * 4;
    constexpr int kMost = (std::max(MAX_BINS, kMaxExperts) + 1) * WARPS * 4;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(sort_pass_kernel), kMost);
    if (e != cudaSuccess) return e;
    e = counted(launch_after_prev_smem(static_cast<size_t>(smem), sort_pass_kernel, dim3(1), dim3(THREADS), stream, p,
                                       dev.status));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace id
}  // namespace rg
