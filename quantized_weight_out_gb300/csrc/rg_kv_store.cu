// rg_kv_store.cu - rg_kv_write and rg_kv_read: new tokens' keys and values into
// the paged cache in its storage type, and stored tokens back out.
//
// A warp handles one granule (16 tokens) of one head and kind, as far as the
// new tokens cover it, 32 dimensions at a time: lane (g, t) loads 8 consecutive
// dimensions of two tokens, so four lanes hold a token's block and two shuffles
// give its largest magnitude.  Keys leave in that arrangement; values are
// transposed through 1 KB of shared memory a warp when the granule is whole, and
// go out byte by byte when it is not (a byte belongs to one token).  Bound by
// memory for prompts, by latency for single tokens.
#include "rg_kv.cuh"
#include "rg_kv_launch.h"

namespace rg {
namespace kv {
namespace {

constexpr int kWarps = 8;

// Codes of 8 values of a row whose 32-value block lies in lanes t = 0..3 of
// the same g: codes[e] (int8 as 0..255, or 0..15) and the block's fp16 scale.
template <int TYPE>
__device__ __forceinline__ uint16_t quantise8(const float (&x)[8], int t, int (&code)[8], int* status) {
  // the largest magnitude as an integer: infinities and NaN are larger than every finite value
  uint32_t m = 0;
  int at = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    if (b > m) { m = b; at = e; }
  }
  uint32_t big = m;
  big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
  big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
  float top = __uint_as_float(big);
  if constexpr (TYPE == RG_Q4_0) {
    // sign of the first value of that magnitude: the smallest index that has it
    int first = m == big ? 2 * (8 * t + at) + (x[at] < 0.0f) : 1 << 16;
    first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 1));
    first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 2));
    if (first & 1) top = -top;
  }
  constexpr float kSteps = TYPE == RG_Q8_0 ? 127.0f : -8.0f;
  __half d = __float2half_rn(top / kSteps);
  float inv = kSteps / top;
  if (big >= 0x7F800000u) {  // a value that is not finite: the block reads back as NaN
    d = __ushort_as_half(0x7E00);
    inv = 0.0f;
  } else {
    if (big > 0x477FE000u) report_range(status);  // 65504: past the fp16 operands of the attention
    if ((__half_as_ushort(d) & 0x7FFFu) == 0) inv = 0.0f;  // rounds to zero: zero codes
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // inv 0 gives the zero code, also for values that are not finite (their product is NaN or 0)
    const float r = inv == 0.0f ? 0.0f : rintf(x[e] * inv);
    if constexpr (TYPE == RG_Q8_0)
      code[e] = static_cast<int>(r) & 255;
    else
      code[e] = min(max(static_cast<int>(r) + 8, 0), 15);
  }
  return __half_as_ushort(d);
}

__device__ __forceinline__ uint32_t bytes4(int a, int b, int c, int d) {
  return static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 8) | (static_cast<uint32_t>(c) << 16) |
         (static_cast<uint32_t>(d) << 24);
}

// A granule's share of the batch's new tokens.
struct Piece {
  int j0, cnt;   // tokens j0 .. j0 + cnt - 1 of the granule
  int token;     // packed token of j0
  int64_t off;   // byte offset of the granule of (kind 0, head 0)
  bool ok;
};

// The piece that starts at packed token i, if one does: i is the first new
// token of its sequence, or the first token of its granule.
__device__ __forceinline__ bool piece_at(const Cache& c, const Batch& b, int i, int gran_bytes, int* status,
                                         Piece* out) {
  const int s = find_seq(b, i);
  const Seq q = load_seq(b, c.page_tokens, s, status);
  if (i < q.start || i >= q.start + q.n) return false;
  const int first = q.len - q.n;              // position of the first new token (negative: before the cache)
  const int pos = first + (i - q.start);
  const bool starts = pos < 0 || pos % kGranule == 0 || i == q.start;
  if (!starts) return false;
  if (pos < 0) {  // one token with no place
    *out = Piece{0, 1, i, 0, false};
    return true;
  }
  const int j0 = pos % kGranule;
  const int page = b.table[static_cast<int64_t>(s) * b.max_pages + pos / c.page_tokens];
  *out = Piece{j0, min(kGranule - j0, q.start + q.n - i), i, 0, page >= 0 && page < c.pages};
  if (out->ok)
    out->off = granule_offset(c, page, 0, 0, pos, gran_bytes);
  else
    report_index(status);
  return true;
}

struct Rows {
  const void* p[2];        // keys, values (NULL: left out)
  int64_t t[2], h[2];      // element strides of tokens and heads
};
struct OutRows {
  void* p[2];
  int64_t t[2], h[2];
};

// grid (windows of `window` packed tokens, groups of kWarps (head, kind) pairs)
template <int TYPE, int AT>
__global__ void __launch_bounds__(32 * kWarps) kv_write_kernel(Cache c, Batch b, Rows in, int window, int* status) {
  __shared__ __align__(16) uint8_t stage[kWarps][1024];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.y * kWarps + warp;
  if (unit >= 2 * c.kv_heads) return;
  const int kind = unit / c.kv_heads, head = unit % c.kv_heads;
  const void* src = in.p[kind];
  if (!src) return;
  const int gb = granule_bytes(TYPE, c.dim), blocks = c.dim / 32;
  const int key0 = 4 * (g >> 1) + (g & 1);
  for (int w = 0; w < window; ++w) {
    const int i = blockIdx.x * window + w;
    if (i >= b.tokens) return;
    Piece pc;
    if (!piece_at(c, b, i, gb, status, &pc) || !pc.ok) continue;
    uint8_t* dst = c.data + pc.off + (static_cast<int64_t>(kind) * c.kv_heads + head) * c.slab_bytes;
    bool have[2];
    int64_t at[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = key0 + 2 * n;
      have[n] = j >= pc.j0 && j < pc.j0 + pc.cnt;
      at[n] = (pc.token + j - pc.j0) * in.t[kind] + head * in.h[kind] + 8 * t;
    }
    const bool whole = pc.cnt == kGranule;
    for (int blk = 0; blk < blocks; ++blk) {
      float x[2][8];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (have[n])
          load8<AT>(src, at[n] + 32 * blk, x[n]);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e) x[n][e] = 0.0f;
      }
      if constexpr (has_scales(TYPE)) {
        int code[2][8];
        uint16_t d[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) d[n] = quantise8<TYPE>(x[n], t, code[n], status);
        uint8_t* out = dst + blk * block16_bytes(TYPE);
        uint16_t* scales = reinterpret_cast<uint16_t*>(dst + blocks * block16_bytes(TYPE));
        if (t == 0) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (have[n]) scales[16 * blk + (kind == 0 ? 2 * g + n : key0 + 2 * n)] = d[n];
        }
        if constexpr (TYPE == RG_Q8_0) {
          if (kind == 0) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
              if (have[n])
                *reinterpret_cast<uint2*>(out + lane * 16 + 8 * n) =
                    make_uint2(bytes4(code[n][0], code[n][1], code[n][2], code[n][3]),
                               bytes4(code[n][4], code[n][5], code[n][6], code[n][7]));
          } else {
            // dimension 8t + e of token j: [e][j / 4][t][j % 4]
            uint8_t* to = whole ? stage[warp] : out;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int j = key0 + 2 * n;
              if (have[n])
#pragma unroll
                for (int e = 0; e < 8; ++e) to[e * 64 + (j >> 2) * 16 + t * 4 + (j & 3)] = code[n][e];
            }
            if (whole) {
              __syncwarp();
              reinterpret_cast<uint4*>(out)[lane] = reinterpret_cast<uint4*>(stage[warp])[lane];
              __syncwarp();
            }
          }
        } else {
          if (kind == 0) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              uint32_t word = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e) word |= static_cast<uint32_t>(code[n][e]) << (4 * ((e & 1) * 4 + (e >> 1)));
              if (have[n]) *reinterpret_cast<uint32_t*>(out + lane * 8 + 4 * n) = word;
            }
          } else {
            // a byte holds dimensions 8q + e and 8(q + 1) + e, q even: lanes t = q and q + 1.
            // Each pair of lanes exchanges its codes; the even one writes token n = 0, the odd one n = 1.
            uint32_t word[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              word[n] = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e) word[n] |= static_cast<uint32_t>(code[n][e]) << (4 * e);
            }
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, (t & 1) ? word[0] : word[1], 1);
            const uint32_t lo = (t & 1) ? other : word[0], hi = (t & 1) ? word[1] : other;
            const int j = key0 + 2 * (t & 1);
            uint8_t* to = whole ? stage[warp] : out;
            if ((t & 1) ? have[1] : have[0])
#pragma unroll
              for (int e = 0; e < 8; ++e)
                to[e * 32 + (j >> 2) * 8 + (t >> 1) * 4 + (j & 1) * 2 + ((j >> 1) & 1)] =
                    static_cast<uint8_t>(((lo >> (4 * e)) & 15u) | (((hi >> (4 * e)) & 15u) << 4));
            if (whole) {
              __syncwarp();
              reinterpret_cast<uint2*>(out)[lane] = reinterpret_cast<uint2*>(stage[warp])[lane];
              __syncwarp();
            }
          }
        }
      } else {
        constexpr bool BF = TYPE == RG_BF16;
        uint32_t word[2][4];
        bool over = false;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            word[n][e] = pack16<BF>(x[n][2 * e], x[n][2 * e + 1]);
            over |= overflowed16<BF>(x[n][2 * e], word[n][e]) || overflowed16<BF>(x[n][2 * e + 1], word[n][e] >> 16);
          }
        if (over) report_range(status);
        if (kind == 0) {
          uint4* out = reinterpret_cast<uint4*>(dst + blk * 1024);
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (have[n]) out[n * 32 + lane] = make_uint4(word[n][0], word[n][1], word[n][2], word[n][3]);
        } else {
          // dimension 8t + e of token j: [t / 2][e][j / 4][t % 2][j % 4]
          uint16_t* to = reinterpret_cast<uint16_t*>(whole ? stage[warp] : dst + blk * 1024);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int j = key0 + 2 * n;
            if (have[n])
#pragma unroll
              for (int e = 0; e < 8; ++e)
                to[(t >> 1) * 256 + e * 32 + (j >> 2) * 8 + (t & 1) * 4 + (j & 3)] =
                    static_cast<uint16_t>(word[n][e >> 1] >> (16 * (e & 1)));
          }
          if (whole) {
            __syncwarp();
            uint4* out = reinterpret_cast<uint4*>(dst + blk * 1024);
#pragma unroll
            for (int n = 0; n < 2; ++n) out[n * 32 + lane] = reinterpret_cast<uint4*>(stage[warp])[n * 32 + lane];
            __syncwarp();
          }
        }
      }
    }
  }
}

template <int TYPE, int AT>
__global__ void __launch_bounds__(32 * kWarps) kv_read_kernel(Cache c, Batch b, OutRows to, int window, int* status) {
  __shared__ __align__(16) uint8_t stage[kWarps][1024];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.y * kWarps + warp;
  if (unit >= 2 * c.kv_heads) return;
  const int kind = unit / c.kv_heads, head = unit % c.kv_heads;
  void* dst = to.p[kind];
  if (!dst) return;
  const int gb = granule_bytes(TYPE, c.dim), blocks = c.dim / 32;
  const int key0 = 4 * (g >> 1) + (g & 1);
  for (int w = 0; w < window; ++w) {
    const int i = blockIdx.x * window + w;
    if (i >= b.tokens) return;
    Piece pc;
    if (!piece_at(c, b, i, gb, status, &pc)) continue;
    const uint8_t* src = c.data + pc.off + (static_cast<int64_t>(kind) * c.kv_heads + head) * c.slab_bytes;
    bool have[2];
    int64_t at[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = key0 + 2 * n;
      have[n] = j >= pc.j0 && j < pc.j0 + pc.cnt;
      at[n] = (pc.token + j - pc.j0) * to.t[kind] + head * to.h[kind] + 8 * t;
    }
    for (int blk = 0; blk < blocks; ++blk) {
      float x[2][8];
      if (!pc.ok) {  // no place in the cache: zeros
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[n][e] = 0.0f;
      } else if constexpr (has_scales(TYPE)) {
        const uint8_t* in = src + blk * block16_bytes(TYPE);
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(src + blocks * block16_bytes(TYPE)) + 16 * blk;
        float d[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) d[n] = f16_to_f32(scales[kind == 0 ? 2 * g + n : key0 + 2 * n]);
        if constexpr (TYPE == RG_Q8_0) {
          const uint4 v = reinterpret_cast<const uint4*>(in)[lane];
          if (kind == 0) {
            const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[n][e] = d[n] * static_cast<float>(static_cast<int8_t>(word[2 * n + (e >> 2)] >> (8 * (e & 3))));
          } else {
            __syncwarp();
            reinterpret_cast<uint4*>(stage[warp])[lane] = v;
            __syncwarp();
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int j = key0 + 2 * n;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[n][e] = d[n] * static_cast<float>(
                                     static_cast<int8_t>(stage[warp][e * 64 + (j >> 2) * 16 + t * 4 + (j & 3)]));
            }
          }
        } else {
          const uint2 v = reinterpret_cast<const uint2*>(in)[lane];
          if (kind == 0) {
            const uint32_t word[2] = {v.x, v.y};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[n][e] = d[n] * static_cast<float>(
                                     static_cast<int>((word[n] >> (4 * ((e & 1) * 4 + (e >> 1)))) & 15u) - 8);
          } else {
            __syncwarp();
            reinterpret_cast<uint2*>(stage[warp])[lane] = v;
            __syncwarp();
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int j = key0 + 2 * n;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int byte =
                    stage[warp][e * 32 + (j >> 2) * 8 + (t >> 1) * 4 + (j & 1) * 2 + ((j >> 1) & 1)];
                x[n][e] = d[n] * static_cast<float>(((byte >> (4 * (t & 1))) & 15) - 8);
              }
            }
          }
        }
      } else {
        constexpr bool BF = TYPE == RG_BF16;
        const uint4* in = reinterpret_cast<const uint4*>(src + blk * 1024);
        const uint4 v[2] = {in[lane], in[32 + lane]};
        if (kind == 0) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t word[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint16_t h = static_cast<uint16_t>(word[e >> 1] >> (16 * (e & 1)));
              x[n][e] = BF ? bf16_to_f32(h) : f16_to_f32(h);
            }
          }
        } else {
          __syncwarp();
          reinterpret_cast<uint4*>(stage[warp])[lane] = v[0];
          reinterpret_cast<uint4*>(stage[warp])[32 + lane] = v[1];
          __syncwarp();
          const uint16_t* in16 = reinterpret_cast<const uint16_t*>(stage[warp]);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int j = key0 + 2 * n;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint16_t h = in16[(t >> 1) * 256 + e * 32 + (j >> 2) * 8 + (t & 1) * 4 + (j & 3)];
              x[n][e] = BF ? bf16_to_f32(h) : f16_to_f32(h);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (have[n]) store8<AT>(dst, at[n] + 32 * blk, x[n]);
    }
  }
}

// Packed tokens a block looks through for granules that start there: 16 (one
// granule a sequence, mostly) once sequences bring that many tokens, else one,
// so that many sequences' single tokens are handled side by side.
int window_for(const Batch& b) { return b.max_new > kGranule ? kGranule : 1; }

template <template <int, int> class Launch, class R>
cudaError_t dispatch(int type, int atype, const Cache& c, const Batch& b, const R& rows, const DevInfo& dev,
                     cudaStream_t stream) {
  const int window = window_for(b);
  const dim3 grid((b.tokens + window - 1) / window, (2 * c.kv_heads + kWarps - 1) / kWarps);
#define RG_KV_AT(T)                                                                                  \
  switch (atype) {                                                                                   \
    case RG_F32: return Launch<T, RG_F32>::go(grid, c, b, rows, window, dev.status, stream);         \
    case RG_F16: return Launch<T, RG_F16>::go(grid, c, b, rows, window, dev.status, stream);         \
    default: return Launch<T, RG_BF16>::go(grid, c, b, rows, window, dev.status, stream);            \
  }
  switch (type) {
    case RG_F16: RG_KV_AT(RG_F16)
    case RG_BF16: RG_KV_AT(RG_BF16)
    case RG_Q8_0: RG_KV_AT(RG_Q8_0)
    default: RG_KV_AT(RG_Q4_0)
  }
#undef RG_KV_AT
}

template <int T, int A>
struct WriteLaunch {
  static cudaError_t go(dim3 grid, const Cache& c, const Batch& b, const Rows& r, int window, int* status,
                        cudaStream_t s) {
    kv_write_kernel<T, A><<<grid, 32 * kWarps, 0, s>>>(c, b, r, window, status);
    return counted(cudaGetLastError());
  }
};
template <int T, int A>
struct ReadLaunch {
  static cudaError_t go(dim3 grid, const Cache& c, const Batch& b, const OutRows& r, int window, int* status,
                        cudaStream_t s) {
    kv_read_kernel<T, A><<<grid, 32 * kWarps, 0, s>>>(c, b, r, window, status);
    return counted(cudaGetLastError());
  }
};

}  // namespace

cudaError_t launch_write(int type, int atype, const Cache& c, const Batch& b, const void* k, int64_t k_t, int64_t k_h,
                         const void* v, int64_t v_t, int64_t v_h, const DevInfo& dev, cudaStream_t stream) {
  const Rows r{{k, v}, {k_t, v_t}, {k_h, v_h}};
  return dispatch<WriteLaunch>(type, atype, c, b, r, dev, stream);
}
cudaError_t launch_read(int type, int atype, const Cache& c, const Batch& b, void* k, int64_t k_t, int64_t k_h,
                        void* v, int64_t v_t, int64_t v_h, const DevInfo& dev, cudaStream_t stream) {
  const OutRows r{{k, v}, {k_t, v_t}, {k_h, v_h}};
  return dispatch<ReadLaunch>(type, atype, c, b, r, dev, stream);
}

}  // namespace kv
}  // namespace rg
