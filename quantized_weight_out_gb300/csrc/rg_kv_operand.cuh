// rg_kv_operand.cuh - device pieces of the attention kernels: operand decode
// from the cache's granules, the warp-level matrix instruction, the exponential.
#pragma once

#include "rg_kv.cuh"

namespace rg {
namespace kv {

template <bool BF>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  if constexpr (BF)
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

// An 8 x 8 matrix of 16-bit values, one row a group of four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 2^x (the hardware's approximation; subnormal results are zero).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// mbar_wait (rg_internal.cuh) as a few instructions: the abort flag and the
// clock are looked at every 4096 tries, in code that stands apart.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const WaitCtl& ctl,
                                         volatile int* abort_flag) {
  uint64_t t0 = 0;
  uint32_t it = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if ((++it & 4095u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort_flag) return false;
      if (now - t0 > ctl.limit_ns) {
        *abort_flag = 1;
        report_timeout(ctl.status);
        return false;
      }
    }
  }
  return true;
}

// Contiguous bytes (a multiple of 16, both addresses 16-byte aligned) from
// global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Codes to fp16 operands.  An integer u < 1024 in the low mantissa bits of the
// half 0x6400 is the value 1024 + u, so a code becomes a half with one byte
// permute (or one mask) and an exact subtraction; the product with the
// block's scale is the only rounding.
__device__ __forceinline__ void q8_pairs(uint32_t w, uint32_t& p01, uint32_t& p23) {
  const uint32_t u = w ^ 0x80808080u;  // q + 128
  const __half2 k = __half2half2(__ushort_as_half(0x6480));  // 1152
  p01 = as_u32(__hsub2(as_h2(__byte_perm(u, 0x64646464u, 0x4140u)), k));
  p23 = as_u32(__hsub2(as_h2(__byte_perm(u, 0x64646464u, 0x4342u)), k));
}
// nibbles (0, 4) and (1, 5) of w, minus 8 each
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t& p04, uint32_t& p15) {
  const __half2 k = __half2half2(__ushort_as_half(0x6408));        // 1032
  const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));  // 1/16
  const __half2 k72 = __half2half2(__ushort_as_half(0xD480));      // -72
  p04 = as_u32(__hsub2(as_h2((w & 0x000F000Fu) | 0x64006400u), k));
  p15 = as_u32(__hfma2(as_h2((w & 0x00F000F0u) | 0x64006400u), sixteenth, k72));
}
__device__ __forceinline__ uint32_t scale2(uint32_t h2, uint32_t s) { return as_u32(__hmul2(as_h2(h2), as_h2(s))); }

// A lane's bytes of one 32-dimension block of a granule, as loaded (q8_0,
// q4_0: codes and scales; else the 16-bit values).
template <int TYPE>
struct KeyWords {
  uint32_t w[TYPE == RG_Q8_0 ? 4 : TYPE == RG_Q4_0 ? 2 : 8];
  uint32_t s;     // scales of the lane's two tokens
};
template <int TYPE>
struct ValueWords {
  uint32_t w[TYPE == RG_Q8_0 ? 4 : TYPE == RG_Q4_0 ? 2 : 8];
  uint32_t s[2];  // scales of the lane's four tokens
};

// `base`: the granule's first byte, in shared (address) or global memory.
template <int TYPE, int D>
__device__ __forceinline__ void load_words(KeyWords<TYPE>& k, uint32_t base, int c, int lane) {
  if constexpr (TYPE == RG_Q4_0) {
    const uint2 v = lds64(base + c * 256 + lane * 8);
    k.w[0] = v.x; k.w[1] = v.y;
  } else {
#pragma unroll
    for (int n = 0; n < (TYPE == RG_Q8_0 ? 1 : 2); ++n) {
      const uint4 v = lds128(base + c * block16_bytes(TYPE) + n * 512 + lane * 16);
      k.w[4 * n] = v.x; k.w[4 * n + 1] = v.y; k.w[4 * n + 2] = v.z; k.w[4 * n + 3] = v.w;
    }
  }
  if constexpr (has_scales(TYPE)) k.s = lds32(base + (D / 32) * block16_bytes(TYPE) + 32 * c + (lane >> 2) * 4);
}
template <int TYPE, int D>
__device__ __forceinline__ void load_words(KeyWords<TYPE>& k, const uint8_t* base, int c, int lane) {
  if constexpr (TYPE == RG_Q4_0) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(base + c * 256) + lane);
    k.w[0] = v.x; k.w[1] = v.y;
  } else {
#pragma unroll
    for (int n = 0; n < (TYPE == RG_Q8_0 ? 1 : 2); ++n) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(base + c * block16_bytes(TYPE) + n * 512) + lane);
      k.w[4 * n] = v.x; k.w[4 * n + 1] = v.y; k.w[4 * n + 2] = v.z; k.w[4 * n + 3] = v.w;
    }
  }
  if constexpr (has_scales(TYPE))
    k.s = __ldg(reinterpret_cast<const uint32_t*>(base + (D / 32) * block16_bytes(TYPE) + 32 * c) + (lane >> 2));
}
template <int TYPE, int D>
__device__ __forceinline__ void load_words(ValueWords<TYPE>& k, uint32_t base, int c, int lane) {
  if constexpr (TYPE == RG_Q4_0) {
    const uint2 v = lds64(base + c * 256 + lane * 8);
    k.w[0] = v.x; k.w[1] = v.y;
  } else {
#pragma unroll
    for (int n = 0; n < (TYPE == RG_Q8_0 ? 1 : 2); ++n) {
      const uint4 v = lds128(base + c * block16_bytes(TYPE) + n * 512 + lane * 16);
      k.w[4 * n] = v.x; k.w[4 * n + 1] = v.y; k.w[4 * n + 2] = v.z; k.w[4 * n + 3] = v.w;
    }
  }
  if constexpr (has_scales(TYPE)) {
    const uint2 v = lds64(base + (D / 32) * block16_bytes(TYPE) + 32 * c + (lane & 3) * 8);
    k.s[0] = v.x; k.s[1] = v.y;
  }
}
template <int TYPE, int D>
__device__ __forceinline__ void load_words(ValueWords<TYPE>& k, const uint8_t* base, int c, int lane) {
  if constexpr (TYPE == RG_Q4_0) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(base + c * 256) + lane);
    k.w[0] = v.x; k.w[1] = v.y;
  } else {
#pragma unroll
    for (int n = 0; n < (TYPE == RG_Q8_0 ? 1 : 2); ++n) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(base + c * block16_bytes(TYPE) + n * 512) + lane);
      k.w[4 * n] = v.x; k.w[4 * n + 1] = v.y; k.w[4 * n + 2] = v.z; k.w[4 * n + 3] = v.w;
    }
  }
  if constexpr (has_scales(TYPE)) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(base + (D / 32) * block16_bytes(TYPE) + 32 * c) + (lane & 3));
    k.s[0] = v.x; k.s[1] = v.y;
  }
}

// Key operands of a block: b[n][i], n8 block n, words of dimensions
// (2i, 2i + 1) of the lane's eight.
template <int TYPE>
__device__ __forceinline__ void key_operand(const KeyWords<TYPE>& k, uint32_t (&b)[2][4]) {
  if constexpr (has_scales(TYPE)) {
    if constexpr (TYPE == RG_Q8_0) {
      q8_pairs(k.w[0], b[0][0], b[0][1]);
      q8_pairs(k.w[1], b[0][2], b[0][3]);
      q8_pairs(k.w[2], b[1][0], b[1][1]);
      q8_pairs(k.w[3], b[1][2], b[1][3]);
    } else {
      q4_pairs(k.w[0], b[0][0], b[0][1]);
      q4_pairs(k.w[0] >> 8, b[0][2], b[0][3]);
      q4_pairs(k.w[1], b[1][0], b[1][1]);
      q4_pairs(k.w[1] >> 8, b[1][2], b[1][3]);
    }
    const uint32_t s0 = __byte_perm(k.s, k.s, 0x1010), s1 = __byte_perm(k.s, k.s, 0x3232);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[0][i] = scale2(b[0][i], s0);
      b[1][i] = scale2(b[1][i], s1);
    }
  } else {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) b[n][i] = k.w[4 * n + i];
  }
}

// Value operands of block c: b[q][i], n8 block q (dimensions 32c + 8q + g),
// tokens 4t + 2i, 4t + 2i + 1.
template <int TYPE>
__device__ __forceinline__ void value_operand(const ValueWords<TYPE>& v, uint32_t (&b)[4][2]) {
  if constexpr (has_scales(TYPE)) {
    if constexpr (TYPE == RG_Q8_0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) q8_pairs(v.w[q], b[q][0], b[q][1]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        q4_pairs(v.w[q / 2], b[q][0], b[q + 1][0]);
        q4_pairs(v.w[q / 2] >> 8, b[q][1], b[q + 1][1]);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      b[q][0] = scale2(b[q][0], v.s[0]);
      b[q][1] = scale2(b[q][1], v.s[1]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i) b[q][i] = v.w[2 * q + i];
  }
}

// Value operands that are not finite (a block's scale may be, or its product pass
// fp16's range) become zero; returns their bits set.
template <int TYPE>
__device__ __forceinline__ uint32_t clean_pair(uint32_t& x) {
  constexpr uint32_t INF = TYPE == RG_BF16 ? 0x7F80u : 0x7C00u;
  const bool lo = (x & INF) == INF, hi = (x & (INF << 16)) == (INF << 16);
  const uint32_t out = (lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
  x &= ~out;
  return out;
}
// (seen[i]: the halves of tokens 4t + 2i, 4t + 2i + 1 that some row may see) True if one
// of those was taken out.
template <int TYPE>
__device__ __forceinline__ bool clean_operand(uint32_t (&b)[4][2], const uint32_t (&seen)[2]) {
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 2; ++i) out[i] |= clean_pair<TYPE>(b[q][i]);
  return ((out[0] & seen[0]) | (out[1] & seen[1])) != 0;
}

__device__ __forceinline__ uint32_t ld32(uint32_t a) { return lds32(a); }
__device__ __forceinline__ uint32_t ld32(const uint8_t* p) { return __ldg(reinterpret_cast<const uint32_t*>(p)); }
__device__ __forceinline__ uint16_t ld16(uint32_t a) { return static_cast<uint16_t>(lds16(a)); }
__device__ __forceinline__ uint16_t ld16(const uint8_t* p) { return __ldg(reinterpret_cast<const uint16_t*>(p)); }

// What clean_operand took out, of token j and dimension d of a granule:
// 0 where the value is finite.
template <int TYPE, int D, class P>
__device__ __forceinline__ float value_not_finite(P base, int j, int d) {
  const int c = d >> 5, q = (d >> 3) & 3, g = d & 7, t = j >> 2, k = j & 3;
  float v;
  if constexpr (has_scales(TYPE)) {
    const float s = f16_to_f32(ld16(base + ((D / 32) * block16_bytes(TYPE) + 32 * c + 2 * j)));
    int code;
    if constexpr (TYPE == RG_Q8_0) {
      const uint32_t w = ld32(base + (c * 512 + (g * 4 + t) * 16 + q * 4));
      code = static_cast<int8_t>(w >> (8 * k));
    } else {
      const uint32_t w = ld32(base + (c * 256 + (g * 4 + t) * 8 + (q >> 1) * 4));
      code = static_cast<int>((w >> (4 * ((k & 1) * 4 + (k >> 1) * 2 + (q & 1)))) & 15u) - 8;
    }
    v = s * static_cast<float>(code);
    if (fabsf(v) >= 65520.0f) v = copysignf(INFINITY, v);  // as the fp16 operand
  } else {
    const uint16_t h = ld16(base + ((2 * c + (q >> 1)) * 512 + (g * 4 + t) * 16 + (q & 1) * 8 + k * 2));
    v = TYPE == RG_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
  }
  return v - v == 0.0f ? 0.0f : v;
}

}  // namespace kv
}  // namespace rg
