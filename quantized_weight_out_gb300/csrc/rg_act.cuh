// rg_act.cuh - activations of the indexed calls in registers: eight values of
// a 16-byte aligned row of F32, F16 or BF16 as F32, and back, rounded once.
#pragma once

#include "rg_internal.cuh"

namespace rg {

__host__ __device__ constexpr int act_bytes(int atype) { return atype == RG_F32 ? 4 : 2; }

template <int AT>
__device__ __forceinline__ void load_act8(const void* row, int64_t at, float (&v)[8]) {
  if constexpr (AT == RG_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + at));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (AT == RG_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}

// Four values of a row, 8-byte aligned (16 for F32).
template <int AT>
__device__ __forceinline__ void load_act4(const void* row, int64_t at, float (&v)[4]) {
  if constexpr (AT == RG_F32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + at));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + at));
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (AT == RG_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}

// Two values to the 16 bits of a type, the first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int AT>
__device__ __forceinline__ void store_act8(void* row, int64_t at, const float (&v)[8]) {
  if constexpr (AT == RG_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    constexpr bool B = AT == RG_BF16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + at) =
        make_uint4(pack16<B>(v[0], v[1]), pack16<B>(v[2], v[3]), pack16<B>(v[4], v[5]), pack16<B>(v[6], v[7]));
  }
}

// One value of a row.
__device__ __forceinline__ float load_act(const void* row, int atype, int64_t at) {
  if (atype == RG_F32) return static_cast<const float*>(row)[at];
  const uint16_t h = static_cast<const uint16_t*>(row)[at];
  return atype == RG_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
}
__device__ __forceinline__ void store_act(void* row, int atype, int64_t at, float v) {
  if (atype == RG_F32) static_cast<float*>(row)[at] = v;
  else if (atype == RG_BF16) static_cast<__nv_bfloat16*>(row)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(row)[at] = __float2half_rn(v);
}

// The power of two that brings a row's largest magnitude `top` to 2^14 .. 2^15 (an fp16 copy of it then keeps fp16's 11
// bits down to 2^-28 of that, and none overflows); rows of zeros stay as they are, and one with an infinity is scaled as
// the largest finite magnitudes are, so that no finite value of it becomes infinite, too.
__device__ __forceinline__ int row_shift(float top) {
  const int e = static_cast<int>(__float_as_uint(top) >> 23);  // top in 2^(e - 127) .. 2^(e - 126)
  return top == 0.0f ? 0 : min(141 - min(e, 254), 120);
}

__device__ __forceinline__ void report_index(int* status) { atomicCAS(status, 0, (int)RG_ERR_INDEX); }

}  // namespace rg
