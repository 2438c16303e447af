// rg_kv_attend.cuh - what the two attention kernels (few rows: rg_kv_rows.cu;
// tiles of rows: rg_kv_tiles.cu) share: the softmax reference, partial
// results of items that several CTAs work on, queries in and results out.
#pragma once

#include "rg_kv_launch.h"
#include "rg_kv_operand.cuh"

namespace rg {
namespace kv {

constexpr float kNone = -3.40282347e38f;  // the reference before any score above -inf
constexpr float kMinusInf = -3.4e38f;     // ... of a part whose row has seen scores of -inf only
constexpr float kHead = 7.0f;        // probabilities are scaled by 2^7
constexpr float kSlack = 8.0f;       // scores may pass the reference by this

// One partial result: m[BM], l[BM], O[BM][D] (unnormalised, relative to 2^m).
__host__ __device__ constexpr int64_t part_floats(int bm, int dim) { return static_cast<int64_t>(bm) * (dim + 2); }

// The first part of an item that several CTAs share, for the joining kernel.
struct Desc {
  int last;    // last CTA with a part of it; -1: none starts here
  int rows;    // valid rows
  int token;   // row 0's packed token ...
  int lead;    // ... and the row's index in the kv head's group
  int head;    // kv head
};

// What a row's sum of products is multiplied by: 1 / l, 0 where it has seen nothing, NaN
// (the definition's 0 / 0) where all that it has seen scored -inf.
__device__ __forceinline__ float row_factor(float m_ref, float l) {
  return l != 0.0f ? 1.0f / l : m_ref > kNone ? NAN : 0.0f;
}
// Whether the row at `pos` sees one of the positions lo .. hi - 1: asked for rows whose
// reference has not moved, of which there are few.
__device__ __forceinline__ bool sees_any(const Cache& c, const int* table, int window, int pos, int lo, int hi) {
  if (window) lo = max(lo, pos - window + 1);
  hi = min(hi, pos + 1);
  while (lo < hi) {
    const int p = lo / c.page_tokens, page = table[p];
    if (page >= 0 && page < c.pages) return true;
    lo = (p + 1) * c.page_tokens;
  }
  return false;
}

__device__ __forceinline__ void store_out(const Attend& a, int token, int head, int d, const float (&v)[4]) {
  const int64_t at = token * a.o_t + head * a.o_h + d;
  if (a.atype == RG_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  else if (a.atype == RG_F16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// Eight query values from element `at` on as four operand words; finite values beyond fp16 are reported.
template <bool BF>
__device__ __forceinline__ uint4 query8(const Attend& a, int64_t at, int* status) {
  float x[8];
  if (a.atype == RG_F32) {
    load8<RG_F32>(a.q, at, x);
  } else if (BF == (a.atype == RG_BF16)) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at));  // already the operand type
  } else if (a.atype == RG_F16) {
    load8<RG_F16>(a.q, at, x);
  } else {
    load8<RG_BF16>(a.q, at, x);
  }
  uint32_t w[4];
  bool over = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack16<BF>(x[2 * i], x[2 * i + 1]);
    over |= overflowed16<BF>(x[2 * i], w[i]) || overflowed16<BF>(x[2 * i + 1], w[i] >> 16);
  }
  if (over) report_range(status);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace kv
}  // namespace rg
