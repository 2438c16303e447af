// rg_id.cu - products by slot around the tensor-core kernel: the table of
// tiles and the input's copy in sorted order, the sum over a token's slots, the
// copy of W whose rows TMA cannot address as they lie, and the product in F32 by
// plain threads for F32 weights.
#include <algorithm>

#include "rg_act.cuh"
#include "rg_id_launch.h"

namespace rg {
namespace id {

namespace {

constexpr int THREADS = 256;

// The table of tiles, by one block: a running sum of the experts' tiles.  An
// expert whose range is not one (reported) has no slots; one whose tiles would
// pass the table's end (ranges that overlap) is reported, and empty tiles stand
// where its would.  Returns whether a range was refused.
__device__ bool build_tiles(const Batch& b, int bt, Tile* tiles, int* n_tiles, int cap, int* status) {
  __shared__ int64_t warp_sum[THREADS / 32];
  __shared__ int64_t base_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool refused = false;
  if (threadIdx.x == 0) base_s = 0;
  __syncthreads();
  for (int e0 = 0; e0 < b.experts; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    int first = 0, rows = 0;
    if (e < b.experts) {
      const int lo = __ldg(b.start + e), hi = __ldg(b.start + e + 1);
      if (lo < 0 || hi < lo || hi > b.slots) refused = true;
      else first = lo, rows = hi - lo;
    }
    const int64_t mine = rows / bt + (rows % bt != 0);
    int64_t upto = mine;  // tiles of this warp's experts up to and with this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int64_t at = base_s + upto - mine;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    const bool fits = at + mine <= cap;
    if (!fits) report_index(status);
    for (int64_t i = at; i < at + mine && i < cap; ++i)
      tiles[i] = fits ? Tile{e, first, rows, static_cast<int>(at)} : Tile{0, 0, 0, static_cast<int>(i)};
    __syncthreads();
    if (threadIdx.x == THREADS - 1) base_s = at + mine;
    __syncthreads();
  }
  if (threadIdx.x == 0) *n_tiles = static_cast<int>(base_s < cap ? base_s : cap);
  if (refused) report_index(status);
  return __syncthreads_or(refused);
}

// Block 0 builds the table; the other blocks' groups of LANES threads (a warp,
// or for rows over 4096 values the block: so many rows of warps would be under
// way that their second reading misses the L2, 103 us for 8186 rows of 14336)
// take the sorted slots in turn, and report those that are none.  Where start
// ascends, the ranges that the table takes lie between its ends, and those are
// the rows copied; where a range is refused, the others may lie anywhere, and
// block 0 copies the rest (a look at all of start by every block took 1 us).
// A row of an fp16 copy is multiplied by the power of two that brings
// its largest magnitude to 2^14 .. 2^15, so that gradients of any size keep
// fp16's 11 bits (values down to 2^-28 of the row's largest are not subnormal)
// and none overflows; the product's rows are multiplied by the inverse, which
// is exact, in F32.  Where they are multiplied by weights too, that is by one
// factor; one that F32 does not hold is reported here (a second multiplication
// in the tensor-core kernel's epilogue cost calls without weights 1 to 10 %).
template <int AT, bool BF16, int LANES>
__global__ void __launch_bounds__(THREADS) gather_kernel(Batch b, int bt, Tile* tiles, int* n_tiles, int cap,
                                                         const void* __restrict__ in, int64_t in_row, int in_tokens,
                                                         const float* __restrict__ weights, int wide,
                                                         uint16_t* __restrict__ x16, int64_t ld,
                                                         float* __restrict__ unscale, uint8_t* __restrict__ live,
                                                         int* status) {
  pdl_launch_dependents();
  // (unsigned: within a step of 2^31 slots the next place passes 31 bits)
  unsigned step = (gridDim.x - 1) * (THREADS / LANES), block = blockIdx.x - 1;
  const bool rest = blockIdx.x == 0;
  if (rest) {
    if (!build_tiles(b, bt, tiles, n_tiles, cap, status)) return;
    step = THREADS / LANES;
    block = 0;
  }
  __shared__ float s_top[THREADS / 32];
  const int lane = threadIdx.x % LANES;
  const unsigned slots = static_cast<unsigned>(b.slots);
  const unsigned begin = __ldg(b.start), end = __ldg(b.start + b.experts);
  for (unsigned i = block * (THREADS / LANES) + threadIdx.x / LANES; i < slots; i += step) {
    const int s = __ldg(b.order + i);
    const bool ok = static_cast<unsigned>(s) < slots;
    if (lane == 0) {
      if (!ok) report_index(status);
      if (live != nullptr) live[i] = 0;
    }
    if (x16 == nullptr || (i >= begin && i < end) == rest) continue;
    uint16_t* to = x16 + i * ld;
    const int64_t row = ok ? (in_tokens ? s / b.per_token : s) : 0;
    const char* from = static_cast<const char*>(in) + row * in_row * act_bytes(AT);
    constexpr int U = 4;  // steps in flight
    float v[U][8];
    auto fetch = [&](int c0) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_act8<AT>(from, min(c0 + 8 * LANES * u, wide - 8), v[u]);
    };
    float mul = 1.0f;
    if constexpr (!BF16) {
      float top = 0.0f;
      for (int c0 = 8 * lane; c0 < wide; c0 += 8 * LANES * U) {
        fetch(c0);  // (past the row's end its last values again)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[u][j]));
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if constexpr (LANES > 32) {
        __syncthreads();  // (the last row's reads)
        if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, s_top[w]);
      }
      const int shift = row_shift(top);
      mul = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
      if (lane == 0) {
        const float back = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
        unscale[i] = back;
        const float weight = weights != nullptr && ok ? __ldg(weights + s) : 0.0f;
        if (top < INFINITY && fabsf(weight) < INFINITY && fabsf(weight * back) == INFINITY) report_range(status);
      }
    }
    for (int c0 = 8 * lane; c0 < wide; c0 += 8 * LANES * U) {
      fetch(c0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + 8 * LANES * u;
        if (c >= wide) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] = ok ? v[u][j] * mul : 0.0f;
        store_act8<BF16 ? RG_BF16 : RG_F16>(to, c, v[u]);
      }
    }
  }
}

template <int AT>
__global__ void __launch_bounds__(THREADS) join_kernel(const float* rows, int64_t groups, int64_t total,
                                                       const uint8_t* live, int per_token,
                                                       const float* __restrict__ weights, void* __restrict__ out,
                                                       int64_t out_row, float beta) {
  pdl_wait();  // the rows come from the kernel before this one
  const int64_t width = groups * 8;
  for (int64_t g = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; g < total;
       g += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int64_t t = g / groups, c = (g - t * groups) * 8;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    constexpr int U = 4;  // slots in flight (rows of slots without an expert are read, and not used)
    for (int j0 = 0; j0 < per_token; j0 += U) {
      float4 v[U][2];
      float w[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t s = t * per_token + min(j0 + u, per_token - 1);
        const float4* p = reinterpret_cast<const float4*>(rows + s * width + c);
        v[u][0] = __ldcg(p);
        v[u][1] = __ldcg(p + 1);
        on[u] = j0 + u < per_token && __ldcg(live + s);
        w[u] = weights != nullptr ? __ldg(weights + s) : 1.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on[u]) {
          const float4 a = v[u][0], b = v[u][1];
          sum[0] = fmaf(w[u], a.x, sum[0]); sum[1] = fmaf(w[u], a.y, sum[1]);
          sum[2] = fmaf(w[u], a.z, sum[2]); sum[3] = fmaf(w[u], a.w, sum[3]);
          sum[4] = fmaf(w[u], b.x, sum[4]); sum[5] = fmaf(w[u], b.y, sum[5]);
          sum[6] = fmaf(w[u], b.z, sum[6]); sum[7] = fmaf(w[u], b.w, sum[7]);
        }
    }
    char* to = static_cast<char*>(out) + t * out_row * act_bytes(AT);
    if (beta != 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(beta, load_act(to, AT, c + i), sum[i]);
    }
    store_act8<AT>(to, c, sum);
  }
}

// A tile of 64 slots by 64 outputs; 32 contraction values a step, each thread
// 4 x 4 sums.  F32 weights, products and sums.
template <bool FWD>
__global__ void __launch_bounds__(THREADS) simt_kernel(Slots g, const uint8_t* __restrict__ W, int64_t N, int64_t K,
                                                       int64_t rb, const void* __restrict__ in, int64_t in_row,
                                                       int in_tokens, int atype) {
  __shared__ float sx[32][kSimtTile + 4];  // [contraction][slot]
  __shared__ float sw[32][kSimtTile + 4];  // [contraction][output]
  __shared__ int s_slot[kSimtTile];
  pdl_wait();  // the table comes from the kernel before this one
  if (static_cast<int>(blockIdx.x) >= __ldcg(g.n_tiles)) return;
  const int4 tile = __ldcg(reinterpret_cast<const int4*>(g.tiles) + blockIdx.x);
  const int pos = tile.y + (static_cast<int>(blockIdx.x) - tile.w) * kSimtTile;
  const int rows = min(kSimtTile, tile.y + tile.z - pos);
  const int64_t out_w = FWD ? N : K, wide = FWD ? K : N;
  const int64_t o0 = static_cast<int64_t>(blockIdx.y) * kSimtTile;
  const uint8_t* we = W + tile.x * N * rb;
  const int tid = threadIdx.x;
  if (tid < kSimtTile) {
    int s = tid < rows ? __ldg(g.order + pos + tid) : -1;
    if (static_cast<unsigned>(s) >= static_cast<unsigned>(g.slots)) s = -1;
    s_slot[tid] = s;
    if (g.live != nullptr && blockIdx.y == 0 && s >= 0) g.live[s] = 1;
  }
  __syncthreads();
  float acc[4][4] = {};
  const int tx = tid & 15, ty = tid >> 4;  // outputs 4 tx .., slots 4 ty ..
  for (int64_t c0 = 0; c0 < wide; c0 += 32) {
    {
      // eight values of one slot's row
      const int r = tid >> 2, cc = 8 * (tid & 3);
      const int s = s_slot[r];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = 0.0f;
        if (s >= 0 && c0 + cc + i < wide)
          v = load_act(static_cast<const char*>(in) + static_cast<int64_t>(in_tokens ? s / g.per_token : s) * in_row *
                                                          act_bytes(atype),
                       atype, c0 + cc + i);
        sx[cc + i][r] = v;
      }
    }
    {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if constexpr (FWD) {
        const int n = tid >> 2, cc = 8 * (tid & 3);
        if (o0 + n < N && c0 + cc < K) decode8_f32<RG_F32>(we + (o0 + n) * rb, static_cast<int>(c0) + cc, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sw[cc + i][n] = v[i];
      } else {
        const int n = tid >> 3, kk = 8 * (tid & 7);
        if (c0 + n < N && o0 + kk < K) decode8_f32<RG_F32>(we + (c0 + n) * rb, static_cast<int>(o0) + kk, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sw[n][kk + i] = v[i];
      }
    }
    __syncthreads();
#pragma unroll 8
    for (int c = 0; c < 32; ++c) {
      float x[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sx[c][4 * ty + i], w[i] = sw[c][4 * tx + i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], w[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = s_slot[4 * ty + i];
    if (s < 0) continue;
    const float m = g.weights != nullptr ? __ldg(g.weights + s) : 1.0f;
    char* to = static_cast<char*>(g.out) + static_cast<int64_t>(s) * g.out_row * act_bytes(g.otype);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t o = o0 + 4 * tx + j;
      if (o >= out_w) continue;
      float v = acc[i][j] * m;
      if (g.beta != 0.0f) v = fmaf(g.beta, load_act(to, g.otype, o), v);
      store_act(to, g.otype, o, v);
    }
  }
}

// Rows of `rb` bytes (a multiple of 2) copied to rows of `grains` 16-byte
// grains, zeros behind their end: what TMA needs of the types whose rows are not
// multiples of 16 bytes (Q6_K, Q3_K, Q2_K, MXFP4 at some K).  A warp a row; an
// expert without slots is skipped.  Whole products with the copy, against plain
// threads that read the rows as they lie: 64 Q6_K experts of 2048 x 1536, 2 / 16 /
// 256 slots an expert, 122 / 187 / 270 us against 745 / 916 / 4449; 128 MXFP4
// experts of 2048 x 768, 107 / 151 / 282 against 713 / 840 / 4115.
constexpr int PAD_ROWS = 32;

__global__ void __launch_bounds__(THREADS) pad_kernel(const uint8_t* __restrict__ W, int64_t N, int64_t rb,
                                                      const int32_t* __restrict__ start, uint4* __restrict__ to,
                                                      int64_t grains) {
  const int e = blockIdx.y;
  if (__ldg(start + e + 1) <= __ldg(start + e)) return;
  const int lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * PAD_ROWS;
  for (int64_t n = first + (threadIdx.x >> 5); n < min(N, first + PAD_ROWS); n += THREADS / 32) {
    const int64_t row = e * N + n;
    const uint8_t* from = W + row * rb;
    const int shift = (row * rb & 2) ? 16 : 0;  // (W is 16-byte aligned)
    const uint32_t* words = reinterpret_cast<const uint32_t*>(from - (shift >> 3));
    for (int64_t j = lane; j < grains; j += 32) {
      uint32_t w[5], v[4];
#pragma unroll
      for (int i = 0; i < 5; ++i)  // words that hold bytes of the row
        w[i] = 16 * j + 4 * i < rb + (shift >> 3) ? __ldg(words + 4 * j + i) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __funnelshift_r(w[i], w[i + 1], shift);
        const int64_t left = rb - 16 * j - 4 * i;
        v[i] = left <= 0 ? 0 : left < 4 ? v[i] & 0xFFFFu : v[i];
      }
      to[row * grains + j] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

template <class F>
cudaError_t with_atype(int atype, F&& f) {
  switch (atype) {
    case RG_F32: return f(std::integral_constant<int, RG_F32>{});
    case RG_F16: return f(std::integral_constant<int, RG_F16>{});
    default: return f(std::integral_constant<int, RG_BF16>{});
  }
}

}  // namespace

cudaError_t launch_gather(const Batch& b, int bt, Tile* tiles, int* n_tiles, int cap, const Product& p, bool bf16,
                          uint16_t* x16, int64_t ld, float* unscale, uint8_t* live, const DevInfo& dev,
                          cudaStream_t stream) {
  const bool wide = x16 != nullptr && p.wide() > 4096;
  const int64_t a_block = wide ? 1 : THREADS / 32;
  const int64_t blocks = std::min<int64_t>((b.slots + a_block - 1) / a_block, dev.num_sms * 8);
  return with_atype(p.atype, [&](auto at) {
    constexpr int AT = decltype(at)::value;
    auto kern = bf16 ? (wide ? gather_kernel<AT, true, THREADS> : gather_kernel<AT, true, 32>)
                     : (wide ? gather_kernel<AT, false, THREADS> : gather_kernel<AT, false, 32>);
    kern<<<static_cast<unsigned>(1 + blocks), THREADS, 0, stream>>>(
        b, bt, tiles, n_tiles, cap, p.in, p.in_row, p.in_tokens ? 1 : 0, p.out_tokens ? nullptr : p.weights,
        static_cast<int>(p.wide()), x16, ld, unscale, live, dev.status);
    return counted(cudaGetLastError());
  });
}

cudaError_t launch_join(const float* rows, int64_t width, const uint8_t* live, const Batch& b, const Product& p,
                        const DevInfo& dev, cudaStream_t stream) {
  const int64_t groups = width / 8, total = static_cast<int64_t>(b.slots / b.per_token) * groups;
  return with_atype(p.atype, [&](auto at) {
    constexpr int AT = decltype(at)::value;
    return counted(launch_after_prev(join_kernel<AT>, dim3(static_cast<unsigned>(grid_for(total, THREADS, dev))),
                                     dim3(THREADS), stream, rows, groups, total, live, b.per_token, p.weights, p.out,
                                     p.out_row, p.beta));
  });
}

cudaError_t launch_simt(const Product& p, const Slots& s, int cap, cudaStream_t stream) {
  const int64_t rb = row_bytes(p.wtype, p.K);
  const int64_t gy = (p.out_w() + kSimtTile - 1) / kSimtTile;  // (at most 65535)
  auto kern = p.fwd ? simt_kernel<true> : simt_kernel<false>;
  return counted(launch_after_prev(kern, dim3(static_cast<unsigned>(cap), static_cast<unsigned>(gy)), dim3(THREADS),
                                   stream, s, static_cast<const uint8_t*>(p.W), p.N, p.K, rb, p.in, p.in_row,
                                   p.in_tokens ? 1 : 0, p.atype));
}

cudaError_t launch_pad(const Product& p, const Batch& b, void* to, cudaStream_t stream) {
  const unsigned gx = static_cast<unsigned>((p.N + PAD_ROWS - 1) / PAD_ROWS);
  pad_kernel<<<dim3(gx, static_cast<unsigned>(b.experts)), THREADS, 0, stream>>>(
      static_cast<const uint8_t*>(p.W), p.N, row_bytes(p.wtype, p.K), b.start, static_cast<uint4*>(to),
      padded_row_bytes(p.wtype, p.K) / 16);
  return counted(cudaGetLastError());
}

}  // namespace id
}  // namespace rg
