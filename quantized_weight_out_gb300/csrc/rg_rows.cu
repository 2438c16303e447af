// rg_rows.cu - rows of a resident table by token, scaled, and the gradient of
// a trained table: dY's rows added to the table's rows by token.
#include <algorithm>

#include "rg_act.cuh"
#include "rg_id_launch.h"

namespace rg {
namespace id {

namespace {

constexpr int THREADS = 256;

// One thread per 8 values.  A row of zeros for an id below 0, and for one past
// the table, which is reported.
template <int WT, int AT>
__global__ void __launch_bounds__(THREADS) get_rows_kernel(const uint8_t* __restrict__ W, int64_t N, int64_t rb,
                                                           const int32_t* __restrict__ ids, int64_t total,
                                                           int64_t groups, float scale, void* __restrict__ out,
                                                           int64_t out_row, int* status) {
  for (int64_t g = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; g < total;
       g += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int64_t i = g / groups;
    const int k0 = static_cast<int>(g - i * groups) * 8;
    const int64_t id = __ldg(ids + i);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (id >= 0 && id < N) {
      decode8_f32<WT>(W + id * rb, k0, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= scale;
    } else if (id >= N) {
      report_index(status);
    }
    store_act8<AT>(static_cast<char*>(out) + i * out_row * act_bytes(AT), k0, v);
  }
}

// --- the gradient -----------------------------------------------------------
// dY's rows, sorted by id, are cut into windows of WIN.  A row of the table has
// one run of sorted positions; the thread that owns (row, 8 columns) adds the
// positions of the run's first window itself, and of each later window the sum
// that the first kernel made of the run's part in it: runs of any length are
// added in an order that the ids alone decide, without atomics.
constexpr int WIN = 64;

// (What the kernel before this one wrote is read by __ldcg after pdl_wait: a load that counts as constant for the
// kernel's life may be moved before the wait.)
template <int AT>
__device__ __forceinline__ void add_run(float (&sum)[8], const void* dY, int64_t dy_row, const int32_t* order,
                                        const int32_t* sorted, int64_t from, int64_t to, int id, int64_t c) {
  for (int64_t p = from; p < to && __ldcg(sorted + p) == id; ++p) {
    float v[8];
    load_act8<AT>(static_cast<const char*>(dY) + static_cast<int64_t>(__ldcg(order + p)) * dy_row * act_bytes(AT), c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += v[i];
  }
}

// The first position of each run into first[id] (entries of rows without one
// are never written, and recognised by what they point at); the sum of each
// window's part of a run that began before it into part[window].
template <int AT>
__global__ void __launch_bounds__(THREADS) rows_back_parts_kernel(const void* __restrict__ dY, int64_t dy_row,
                                                                  const int32_t* order,
                                                                  const int32_t* sorted, int64_t n,
                                                                  int64_t N, int64_t K, int32_t* first,
                                                                  float* part) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t w = blockIdx.x, p0 = w * WIN;
  for (int64_t p = p0 + threadIdx.x; p < min(n, p0 + WIN); p += THREADS) {
    const int id = __ldcg(sorted + p);
    if (id < N && (p == 0 || __ldcg(sorted + p - 1) != id)) first[id] = static_cast<int32_t>(p);
  }
  const int id = __ldcg(sorted + p0);
  if (p0 == 0 || id >= N || __ldcg(sorted + p0 - 1) != id) return;
  for (int64_t c = 8 * threadIdx.x; c < K; c += 8 * THREADS) {
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    add_run<AT>(sum, dY, dy_row, order, sorted, p0, min(n, p0 + WIN), id, c);
    store_act8<RG_F32>(part + w * K, c, sum);
  }
}

template <int AT>
__global__ void __launch_bounds__(THREADS) rows_back_kernel(const void* __restrict__ dY, int64_t dy_row,
                                                            const int32_t* order,
                                                            const int32_t* sorted, int64_t n, int64_t total,
                                                            int64_t groups, const int32_t* first,
                                                            const float* part, float scale,
                                                            float* __restrict__ G, int64_t g_row, float beta) {
  pdl_wait();
  const int64_t K = groups * 8;
  for (int64_t g = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; g < total;
       g += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int64_t r = g / groups, c = (g - r * groups) * 8;
    const int id = static_cast<int>(r);
    const int64_t p = __ldcg(first + r);
    const bool has = p >= 0 && p < n && __ldcg(sorted + p) == id && (p == 0 || __ldcg(sorted + p - 1) != id);
    if (!has && beta == 1.0f) continue;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (has) {
      const int64_t w = p / WIN;
      add_run<AT>(sum, dY, dy_row, order, sorted, p, min(n, (w + 1) * WIN), id, c);
      for (int64_t x = w + 1; x * WIN < n && __ldcg(sorted + x * WIN) == id; ++x) {
        const float4* q = reinterpret_cast<const float4*>(part + x * K + c);
        const float4 a = __ldcg(q), b = __ldcg(q + 1);
        sum[0] += a.x; sum[1] += a.y; sum[2] += a.z; sum[3] += a.w;
        sum[4] += b.x; sum[5] += b.y; sum[6] += b.z; sum[7] += b.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] *= scale;
    }
    float* to = G + r * g_row + c;
    if (beta != 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(beta, to[i], sum[i]);
    }
    store_act8<RG_F32>(to, 0, sum);
  }
}

}  // namespace

cudaError_t launch_get_rows(int wtype, const void* W, int64_t N, int64_t K, const int32_t* ids, int64_t n,
                            float scale, int atype, void* out, int64_t out_row, const DevInfo& dev,
                            cudaStream_t stream) {
  const int64_t rb = K / block_values(wtype) * block_bytes(wtype), total = n * (K / 8);
  return with_wtype(wtype, cudaErrorInvalidValue, [&](auto wt) {
    constexpr int WT = decltype(wt)::value;
    auto kern = atype == RG_F32   ? get_rows_kernel<WT, RG_F32>
                : atype == RG_F16 ? get_rows_kernel<WT, RG_F16>
                                  : get_rows_kernel<WT, RG_BF16>;
    kern<<<grid_for(total, THREADS, dev), THREADS, 0, stream>>>(static_cast<const uint8_t*>(W), N, rb, ids, total, K / 8,
                                                                scale, out, out_row, dev.status);
    return counted(cudaGetLastError());
  });
}

// order, sorted, first and the windows' sums, then the sort's own.
size_t rows_back_workspace(int64_t n, int64_t N, int64_t K) {
  const int64_t windows = (n + WIN - 1) / WIN;
  return static_cast<size_t>(2 * up256(n * 4) + up256(N * 4) + up256(windows * K * 4)) + sort_workspace(n, N);
}

cudaError_t launch_rows_back(int atype, const void* dY, int64_t dy_row, const int32_t* ids, int64_t n, float scale,
                             float* G, int64_t g_row, int64_t N, int64_t K, float beta, void* ws, const DevInfo& dev,
                             cudaStream_t stream) {
  char* at = static_cast<char*>(ws);
  auto take = [&](int64_t bytes) {
    char* p = at;
    at += up256(bytes);
    return p;
  };
  const int64_t windows = (n + WIN - 1) / WIN;
  int32_t* order = reinterpret_cast<int32_t*>(take(n * 4));
  int32_t* sorted = reinterpret_cast<int32_t*>(take(n * 4));
  int32_t* first = reinterpret_cast<int32_t*>(take(N * 4));
  float* part = reinterpret_cast<float*>(take(windows * K * 4));
  cudaError_t e = launch_sort(ids, n, N, nullptr, order, sorted, at, dev, stream);
  if (e != cudaSuccess) return e;
  const int64_t total = N * (K / 8);
  auto go = [&](auto t) {
    constexpr int AT = decltype(t)::value;
    cudaError_t r = counted(launch_after_prev(rows_back_parts_kernel<AT>, dim3(static_cast<unsigned>(windows)),
                                              dim3(THREADS), stream, dY, dy_row, order, sorted, n, N, K, first, part));
    if (r != cudaSuccess) return r;
    return counted(launch_after_prev(rows_back_kernel<AT>, dim3(static_cast<unsigned>(grid_for(total, THREADS, dev))),
                                     dim3(THREADS), stream, dY, dy_row, order, sorted, n, total, K / 8, first, part,
                                     scale, G, g_row, beta));
  };
  return atype == RG_F32   ? go(std::integral_constant<int, RG_F32>{})
         : atype == RG_F16 ? go(std::integral_constant<int, RG_F16>{})
                           : go(std::integral_constant<int, RG_BF16>{});
}

}  // namespace id
}  // namespace rg
