// rg_route.cu - the router of a mixture of experts: each token's experts by
// its logits, their weights, and the gradient through the weights.
//
// A warp per token, lane l with the logits of experts l, l + 32, ...; the k
// largest one after another by warp-wide maxima of an integer that orders as
// the logit does.
#include "rg_act.cuh"
#include "rg_id_launch.h"
#include "rg_sort.cuh"

namespace rg {
namespace id {

namespace {

constexpr int THREADS = 256;

// An unsigned integer that orders as the finite or infinite v does, 0 for a
// logit that is never chosen (-inf, NaN).  (-0 counts as 0.)
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
  return v > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One token by one warp: lane j's j-th choice and its weight.
template <int PER>
__device__ __forceinline__ void route_token(const float* __restrict__ row, int experts, int top, int mode, float scale,
                                            int lane, int& my_id, float& weight) {
  uint32_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 32 * j;
    key[j] = e < experts ? order_key(__ldg(row + e)) : 0u;
  }
  float part = 0.0f;  // of the sum over all experts
  float most = 0.0f, my_exp = 0.0f;
  my_id = -1;
  for (int c = 0; c < top; ++c) {
    uint32_t k = 0;
    int e = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (key[j] > k) {  // (of equals the first: the lowest expert of this lane)
        k = key[j];
        e = lane + 32 * j;
      }
    const uint32_t best = __reduce_max_sync(0xffffffffu, k);
    if (best == 0) break;  // nothing left to choose
    const int id = static_cast<int>(__reduce_min_sync(0xffffffffu, k == best ? static_cast<unsigned>(e) : 0x7fffffffu));
    const float v = key_value(best);
    if (c == 0) {
      most = v;
      if (mode == RG_ROUTE_ALL) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (key[j] != 0) part += expf(key_value(key[j]) - most);
      }
    }
    if (lane == c) {
      my_id = id;
      my_exp = expf(v - most);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (lane + 32 * j == id) key[j] = 0;
  }
  const float total = warp_sum(mode == RG_ROUTE_ALL ? part : my_exp);
  weight = my_id < 0 ? 0.0f : scale * (my_exp / total);
}

template <int PER>
__global__ void __launch_bounds__(THREADS) route_kernel(const float* __restrict__ logits, int64_t l_row, int64_t T,
                                                        int experts, int top, int mode, float scale,
                                                        int32_t* __restrict__ ids, float* __restrict__ weights) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
  for (int64_t t = blockIdx.x * static_cast<int64_t>(THREADS / 32) + (threadIdx.x >> 5); t < T; t += step) {
    int id;
    float w;
    route_token<PER>(logits + t * l_row, experts, top, mode, scale, lane, id, w);
    if (lane < top) {
      ids[t * top + lane] = id;
      weights[t * top + lane] = w;
    }
  }
}

// A decoding batch: the router and the sort of its slots by one block, in one
// launch (as two, one token's took 11.5 us).
constexpr int ONE_TOKENS = 64, ONE_SLOTS = 1024;
template <int PER>
__global__ void __launch_bounds__(SORT_THREADS, 1) route_one_kernel(const float* __restrict__ logits, int64_t l_row,
                                                                    int T, int experts, int top, int mode, float scale,
                                                                    int32_t* __restrict__ ids,
                                                                    float* __restrict__ weights, Sort p) {
  extern __shared__ int hist[];
  __shared__ int32_t s_ids[ONE_SLOTS];
  const int lane = threadIdx.x & 31;
  for (int t = threadIdx.x >> 5; t < T; t += static_cast<int>(blockDim.x >> 5)) {
    int id;
    float w;
    route_token<PER>(logits + t * l_row, experts, top, mode, scale, lane, id, w);
    if (lane < top) {
      s_ids[t * top + lane] = id;
      ids[t * top + lane] = id;
      weights[t * top + lane] = w;
    }
  }
  __syncthreads();
  p.ids = s_ids;
  (void)sort_block<true>(p, hist);
}

template <int PER>
__global__ void __launch_bounds__(THREADS) route_back_kernel(const float* __restrict__ logits, int64_t l_row, int64_t T,
                                                             int experts, int top, int mode, float scale,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ dweights,
                                                             float* __restrict__ dlogits, int64_t dl_row, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
  for (int64_t t = blockIdx.x * static_cast<int64_t>(THREADS / 32) + (threadIdx.x >> 5); t < T; t += step) {
    const float* row = logits + t * l_row;
    int id = -1;
    float dw = 0.0f;
    if (lane < top) {
      id = __ldg(ids + t * top + lane);
      dw = __ldg(dweights + t * top + lane);
      if (id >= experts) {
        report_index(status);
        id = -1;
      }
      if (id < 0) dw = 0.0f;
    }
    float l[PER], up[PER];
    uint32_t chosen = 0;  // bit j: this lane's j-th expert is one of the token's
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + 32 * j;
      l[j] = e < experts ? __ldg(row + e) : -INFINITY;
      if (!(l[j] > -INFINITY)) l[j] = -INFINITY;  // NaN: as one that is never chosen
      up[j] = 0.0f;
    }
    for (int c = 0; c < top; ++c) {
      const int e = __shfl_sync(0xffffffffu, id, c);
      const float d = __shfl_sync(0xffffffffu, dw, c);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (lane + 32 * j == e) {
          chosen |= 1u << j;
          up[j] += d;
        }
    }
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (mode != RG_ROUTE_ALL && !(chosen >> j & 1u)) l[j] = -INFINITY;
      most = fmaxf(most, l[j]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    float part = 0.0f;
    uint32_t in = 0;  // bit j: this lane's j-th expert takes part
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (l[j] > -INFINITY) in |= 1u << j;
      l[j] = l[j] > -INFINITY ? expf(l[j] - most) : 0.0f;
      part += l[j];
    }
    const float total = warp_sum(part);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      l[j] = in >> j & 1u ? l[j] / total : 0.0f;  // (a logit of +inf: NaN for all that take part, as in the weights)
      if (chosen >> j & 1u) dot = fmaf(l[j], up[j], dot);
    }
    dot = warp_sum(dot);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + 32 * j;
      if (e < experts) dlogits[t * dl_row + e] = in >> j & 1u ? scale * (l[j] * (up[j] - dot)) : 0.0f;
    }
  }
}

// f(std::integral_constant<int, PER>{}) for the logits a lane holds.
template <class F>
cudaError_t with_per(int experts, F&& f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>{});
  if (experts <= 64) return f(std::integral_constant<int, 2>{});
  if (experts <= 128) return f(std::integral_constant<int, 4>{});
  if (experts <= 256) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route(const float* logits, int64_t l_row, int64_t T, int experts, int top, int mode, float scale,
                         int32_t* ids, float* weights, int32_t* start, int32_t* order, const DevInfo& dev,
                         cudaStream_t stream) {
  if (start != nullptr && T <= ONE_TOKENS && T * top <= ONE_SLOTS) {
    Sort p{};
    sort_plan(experts, true, &p);
    p.order = order;
    p.start = start;
    p.n = T * top;
    p.groups = experts;
    return with_per(experts, [&](auto per) {
      auto kern = route_one_kernel<decltype(per)::value>;
      const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kSortMostSmem);
      if (e != cudaSuccess) return e;
      const int threads = T <= 8 ? 256 : SORT_THREADS;
      kern<<<1, threads, sort_smem(p.bins, threads / 32), stream>>>(logits, l_row, static_cast<int>(T), experts, top,
                                                                    mode, scale, ids, weights, p);
      return counted(cudaGetLastError());
    });
  }
  const cudaError_t e = with_per(experts, [&](auto per) {
    route_kernel<decltype(per)::value><<<grid_for(T * 32, THREADS, dev), THREADS, 0, stream>>>(
        logits, l_row, T, experts, top, mode, scale, ids, weights);
    return counted(cudaGetLastError());
  });
  if (e != cudaSuccess || start == nullptr) return e;
  return launch_sort(ids, T * top, experts, start, order, nullptr, nullptr, dev, stream);
}

cudaError_t launch_route_back(const float* logits, int64_t l_row, int64_t T, int experts, int top, int mode,
                              float scale, const int32_t* ids, const float* dweights, float* dlogits, int64_t dl_row,
                              const DevInfo& dev, cudaStream_t stream) {
  return with_per(experts, [&](auto per) {
    route_back_kernel<decltype(per)::value><<<grid_for(T * 32, THREADS, dev), THREADS, 0, stream>>>(
        logits, l_row, T, experts, top, mode, scale, ids, dweights, dlogits, dl_row, dev.status);
    return counted(cudaGetLastError());
  });
}

}  // namespace id
}  // namespace rg
