// rg_rows.cu - rows of a resident table by token, scaled, and the gradient of
// a trained table: dY's rows added to the table's rows by token.
#include <algorithm>

#include "rg_act.cuh"
#include "rg_id_launch.h"
#include "rg_raw.cuh"

namespace rg {
namespace id {

namespace {

constexpr int THREADS = 256;

// One thread per 8 values, a warp's 32 threads one 256-value tile of a row: the
// bytes of a type by the wide loads of its layout (8 of single bytes a thread
// took 30.8 us for 8191 rows of 4096 Q6_K values).  A row of zeros for an id
// below 0, and for one past the table, which is reported.  What is written
// bounds it (that case: 67 of 95 MB).
template <int WT, int AT, int U>
__global__ void __launch_bounds__(THREADS) get_rows_kernel(const uint8_t* __restrict__ W, int64_t N, int64_t rb,
                                                           const int32_t* __restrict__ ids, int64_t n, int K,
                                                           float scale, void* __restrict__ out, int64_t out_row,
                                                           int* status) {
  const int lane = threadIdx.x & 31, units = (K + 256 * U - 1) / (256 * U);  // U tiles of a row at a time
  const int64_t total = n * units, step = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
  for (int64_t g = blockIdx.x * static_cast<int64_t>(THREADS / 32) + (threadIdx.x >> 5); g < total; g += step) {
    const int64_t i = g / units;
    const int kt = static_cast<int>(g - i * units) * U, k0 = 256 * kt + 8 * lane;
    const int64_t id = __ldg(ids + i);
    const bool real = id >= 0 && id < N;
    if (id >= N) report_index(status);
    smt::Raw<WT> raw[U];
    const uint8_t* tile = W + id * rb + static_cast<int64_t>(kt) * smt::tile_bytes<WT>();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (real && k0 + 256 * u < K) smt::load_raw_smem<WT>(tile + u * smt::tile_bytes<WT>(), lane, raw[u]);
    char* to = static_cast<char*>(out) + i * out_row * act_bytes(AT);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + 256 * u >= K) break;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (real) {
        smt::decode_raw<WT>(raw[u], lane, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= scale;
      }
      store_act8<AT>(to, k0 + 256 * u, v);
    }
  }
}

// --- the gradient -----------------------------------------------------------
// Four launches.  The sort of the ids; while its few blocks run, the table's
// old values times beta (zeros for beta 0, nothing for beta 1) by the others;
// then dY's rows in sorted order, cut into windows of WIN, each summed by
// itself: a run of one id that lies in one window is added to its row at once,
// the pieces of one that crosses windows are kept; the last launch adds these
// up, in order, for the window that the run begins in.  Runs of any length cost
// the same a row of dY, and the order of a sum is decided by the ids alone:
// there are no atomics.  (A thread per row and column that looked its run up and
// walked it took 187 us beside 128 us of partial sums for 16381 rows of 4096
// into a table of 32000: the walks' loads wait for one another.)
// (What the kernel before this one wrote is read by __ldcg after pdl_wait: a
// load that counts as constant for the kernel's life may be moved before it.)
constexpr int WIN = 32;
constexpr int COLS = 4 * THREADS;  // columns of a block at most (blockIdx.y: which)

// G's rows times beta.  Starts beside the sort, which started after everything
// before it had ended, and ends after it: the kernel behind this one may count
// on both.
__global__ void __launch_bounds__(THREADS) rows_scale_kernel(float* __restrict__ G, int64_t g_row, int64_t total,
                                                             int64_t quads, float beta) {
  pdl_launch_dependents();
  for (int64_t g = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; g < total;
       g += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int64_t r = quads * 4 == g_row ? 0 : g / quads;
    float4* to = reinterpret_cast<float4*>(G + r * g_row + 4 * (g - r * quads));
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (beta != 0.0f) {
      v = *to;
      v.x *= beta; v.y *= beta; v.z *= beta; v.w *= beta;
    }
    *to = v;
  }
  pdl_wait();
}

// Windows of the sorted rows: `lanes` threads (a power of two) a window, four
// columns a thread.  head[w] receives the last run's piece where the run goes
// on behind the window, cont[w] the first run's where it began before it (the
// whole window's, where that run fills it).
template <int AT>
__global__ void __launch_bounds__(THREADS) rows_window_kernel(const void* __restrict__ dY, int64_t dy_row,
                                                              const int32_t* order, const int32_t* sorted, int64_t n,
                                                              int64_t N, int64_t K, int lanes, float scale, float* G,
                                                              int64_t g_row, bool fresh, float* head, float* cont) {
  constexpr int U = 16;  // rows in flight
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, group = tid / lanes, lane = tid & (lanes - 1), groups = THREADS / lanes;
  const int64_t w0 = blockIdx.x * static_cast<int64_t>(groups), p0 = w0 * WIN;
  extern __shared__ int32_t s_win[];  // [groups * WIN] order, [groups * WIN + 2] ids from p0 - 1 on
  int32_t* so = s_win;
  int32_t* si = s_win + groups * WIN;
  for (int i = tid; i < groups * WIN + 2; i += THREADS) {
    const int64_t p = p0 - 1 + i;
    si[i] = p >= 0 && p < n ? __ldcg(sorted + p) : -1;
    if (i < groups * WIN && p0 + i < n) so[i] = __ldcg(order + p0 + i);
  }
  __syncthreads();
  const int64_t w = w0 + group, c = blockIdx.y * static_cast<int64_t>(COLS) + 4 * lane;
  if (w * WIN >= n || c >= K) return;
  const int here = static_cast<int>(min(static_cast<int64_t>(WIN), n - w * WIN));
  const int32_t* id = si + group * WIN + 1;
  const int32_t* ord = so + group * WIN;
  float sum[4] = {0, 0, 0, 0};
  bool began = id[-1] != id[0];  // this run began in this window
  for (int q = 0; q < here; q += U) {
    float v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)  // (every load without a condition, past the end the last row again: all in flight)
      load_act4<AT>(static_cast<const char*>(dY) +
                        static_cast<int64_t>(ord[min(q + u, here - 1)]) * dy_row * act_bytes(AT), c, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = q + u;
      if (p >= here || id[p] >= N) break;  // (ids of no row are the last)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += v[u][i];
      const bool ends = id[p + 1] != id[p];
      if (!ends && p + 1 < here) continue;
      const float4 s = make_float4(sum[0], sum[1], sum[2], sum[3]);
      if (ends && began) {
        float4* to = reinterpret_cast<float4*>(G + static_cast<int64_t>(id[p]) * g_row + c);
        float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!fresh) old = *to;
        *to = make_float4(fmaf(scale, s.x, old.x), fmaf(scale, s.y, old.y), fmaf(scale, s.z, old.z),
                          fmaf(scale, s.w, old.w));
      } else {
        __stcg(reinterpret_cast<float4*>((began ? head : cont) + w * K + c), s);
      }
      sum[0] = sum[1] = sum[2] = sum[3] = 0.0f;
      began = true;
    }
  }
}

// The runs that cross windows: a block of the window that one begins in.
__global__ void __launch_bounds__(THREADS) rows_cross_kernel(const int32_t* sorted, int64_t n, int64_t N, int64_t K,
                                                             float scale, float* G, int64_t g_row, bool fresh,
                                                             const float* head, const float* cont) {
  constexpr int U = 8;
  pdl_wait();
  const int64_t w = blockIdx.x, end = (w + 1) * WIN;
  if (end >= n) return;
  const int id = __ldcg(sorted + end - 1);
  // the run goes on behind the window, and did not begin before it
  if (id >= N || __ldcg(sorted + end) != id || (w > 0 && __ldcg(sorted + w * WIN - 1) == id)) return;
  const int64_t c = blockIdx.y * static_cast<int64_t>(COLS) + 4 * threadIdx.x;
  if (c >= K) return;
  float4 s = __ldcg(reinterpret_cast<const float4*>(head + w * K + c));
  for (int64_t x = w + 1; x * WIN < n; x += U) {
    bool on[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // (loads without a condition, past the end of the last window)
      const int64_t y = min(x + u, (n - 1) / WIN);
      on[u] = y == x + u && __ldcg(sorted + y * WIN) == id;
      v[u] = __ldcg(reinterpret_cast<const float4*>(cont + y * K + c));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (on[u]) {
        s.x += v[u].x; s.y += v[u].y; s.z += v[u].z; s.w += v[u].w;
      }
    if (!on[U - 1]) break;
  }
  float4* to = reinterpret_cast<float4*>(G + static_cast<int64_t>(id) * g_row + c);
  float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (!fresh) old = *to;
  *to = make_float4(fmaf(scale, s.x, old.x), fmaf(scale, s.y, old.y), fmaf(scale, s.z, old.z), fmaf(scale, s.w, old.w));
}

}  // namespace

cudaError_t launch_get_rows(int wtype, const void* W, int64_t N, int64_t K, const int32_t* ids, int64_t n,
                            float scale, int atype, void* out, int64_t out_row, const DevInfo& dev,
                            cudaStream_t stream) {
  const int64_t rb = K / block_values(wtype) * block_bytes(wtype), tiles = (K + 255) / 256;
  // more tiles than the GPU holds warps: four in flight a warp (8191 rows of 4096: 25.8 us with one)
  const bool many = n * tiles > static_cast<int64_t>(dev.num_sms) * 64;
  const int64_t threads = n * (many ? (tiles + 3) / 4 : tiles) * 32;
  return with_wtype(wtype, cudaErrorInvalidValue, [&](auto wt) {
    constexpr int WT = decltype(wt)::value;
    auto kern = atype == RG_F32   ? (many ? get_rows_kernel<WT, RG_F32, 4> : get_rows_kernel<WT, RG_F32, 1>)
                : atype == RG_F16 ? (many ? get_rows_kernel<WT, RG_F16, 4> : get_rows_kernel<WT, RG_F16, 1>)
                                  : (many ? get_rows_kernel<WT, RG_BF16, 4> : get_rows_kernel<WT, RG_BF16, 1>);
    kern<<<grid_for(threads, THREADS, dev), THREADS, 0, stream>>>(static_cast<const uint8_t*>(W), N, rb, ids, n,
                                                                  static_cast<int>(K), scale, out, out_row, dev.status);
    return counted(cudaGetLastError());
  });
}

// order, the sorted ids and the windows' pieces, then the sort's own.
size_t rows_back_workspace(int64_t n, int64_t N, int64_t K) {
  const int64_t windows = (n + WIN - 1) / WIN;
  return static_cast<size_t>(2 * up256(n * 4) + 2 * up256(windows * K * 4)) + sort_workspace(n, N);
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
  const int64_t windows = (n + WIN - 1) / WIN, chunks = (K + COLS - 1) / COLS;  // (chunks: at most 65535)
  int32_t* order = reinterpret_cast<int32_t*>(take(n * 4));
  int32_t* sorted = reinterpret_cast<int32_t*>(take(n * 4));
  float* head = reinterpret_cast<float*>(take(windows * K * 4));
  float* cont = reinterpret_cast<float*>(take(windows * K * 4));
  cudaError_t e = launch_sort(ids, n, N, nullptr, order, sorted, at, dev, stream, /*after_prev=*/beta == 1.0f);
  if (e != cudaSuccess) return e;
  if (beta != 1.0f) {
    const int64_t total = N * (K / 4);
    e = counted(launch_after_prev(rows_scale_kernel, dim3(static_cast<unsigned>(grid_for(total, THREADS, dev))),
                                  dim3(THREADS), stream, G, g_row, total, K / 4, beta));
    if (e != cudaSuccess) return e;
  }
  const bool fresh = beta == 0.0f;
  int lanes = 2;  // threads a window
  while (lanes < THREADS && 4 * lanes < K) lanes *= 2;
  const int groups = THREADS / lanes;
  const dim3 grid(static_cast<unsigned>((windows + groups - 1) / groups), static_cast<unsigned>(chunks));
  const size_t smem = static_cast<size_t>(2 * groups * WIN + 2) * 4;
  auto window = [&](auto t) {
    return counted(launch_after_prev_smem(smem, rows_window_kernel<decltype(t)::value>, grid, dim3(THREADS), stream, dY,
                                          dy_row, order, sorted, n, N, K, lanes, scale, G, g_row, fresh, head, cont));
  };
  e = atype == RG_F32   ? window(std::integral_constant<int, RG_F32>{})
      : atype == RG_F16 ? window(std::integral_constant<int, RG_F16>{})
                        : window(std::integral_constant<int, RG_BF16>{});
  if (e != cudaSuccess || windows == 1) return e;
  return counted(launch_after_prev(rows_cross_kernel, dim3(static_cast<unsigned>(windows), static_cast<unsigned>(chunks)),
                                   dim3(THREADS), stream, sorted, n, N, K, scale, G, g_row, fresh, head, cont));
}

}  // namespace id
}  // namespace rg
