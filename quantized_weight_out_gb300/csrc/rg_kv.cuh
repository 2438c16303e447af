// rg_kv.cuh - the paged key/value cache: byte layout, the batch description
// as kernels see it, and the loads and stores of activations.
//
// A page holds page_tokens tokens of every kv head, keys then values:
// [kind][kv head][granule].  A granule is 16 tokens of one head and one kind,
// contiguous: the unit one bulk copy fetches.  Inside it the codes are in the
// order in which the lanes of a warp need them as the B operand of
// mma.m16n8k16 (lane = 4 g + t): each lane's bytes of a 32-value block are one
// 8- or 16-byte word and a warp's load is contiguous, so the attention
// kernels read operands without bank conflicts, transposes or shuffles.
//   keys (B[k = dimension][n = token]): token j = 4a + 2n + b belongs to group
//     g = 2a + b of n8 block n; lane t holds dimensions 32c + 8t .. + 7.  The
//     contraction order over dimensions is free as long as the queries use
//     the same one.
//   values (B[k = token][n = dimension]): lane t holds tokens 4t .. 4t + 3 of
//     dimension 32c + 8q + g (n8 block q of block c).  With the keys' token
//     order the probabilities of a score tile are then already the A operand.
// After the codes come the fp16 scales (q8_0, q4_0): keys [c][g][n], values
// [c][token].
#pragma once

#include "rg_internal.cuh"

namespace rg {
namespace kv {

constexpr int kGranule = 16;  // tokens

__host__ __device__ constexpr bool valid_type(int type) {
  return type == RG_F16 || type == RG_BF16 || type == RG_Q8_0 || type == RG_Q4_0;
}
__host__ __device__ constexpr bool has_scales(int type) { return type == RG_Q8_0 || type == RG_Q4_0; }
// bytes of one token's row of one head and kind
__host__ __device__ constexpr int row_bytes(int type, int dim) {
  return type == RG_Q8_0 ? dim / 32 * 34 : type == RG_Q4_0 ? dim / 32 * 18 : 2 * dim;
}
// bytes of the codes of 16 tokens x 32 dimensions, and of a whole granule
__host__ __device__ constexpr int block16_bytes(int type) {
  return type == RG_Q8_0 ? 512 : type == RG_Q4_0 ? 256 : 1024;
}
__host__ __device__ constexpr int granule_bytes(int type, int dim) { return kGranule * row_bytes(type, dim); }

// The cache and the batch, as kernels take them.
struct Cache {
  uint8_t* data;
  int64_t page_bytes;   // a page: both kinds, all heads
  int64_t slab_bytes;   // one kind and head of a page
  int pages, page_tokens, kv_heads, dim;
};
struct Batch {
  const int* new_start;  // [seqs + 1]
  const int* kv_len;     // [seqs]
  const int* table;      // [seqs][max_pages]
  int seqs, max_pages, max_new;
  int tokens;            // rows of the packed arrays
};

// Byte offset of a granule's first byte from the cache's (64 bits: pools pass 4 GB).
__device__ __forceinline__ int64_t granule_offset(const Cache& c, int page, int kind, int head, int pos,
                                                  int gran_bytes) {
  return page * c.page_bytes + (static_cast<int64_t>(kind) * c.kv_heads + head) * c.slab_bytes +
         static_cast<int64_t>(pos % c.page_tokens / kGranule) * gran_bytes;
}

__device__ __forceinline__ void report_index(int* status) { atomicCAS(status, 0, (int)RG_ERR_INDEX); }

// One sequence's place in the batch, checked against it.  A sequence whose
// numbers lie outside the batch counts as empty and is reported.
struct Seq {
  int start, n, len;  // first packed token, new tokens, length with them
};
__device__ __forceinline__ Seq load_seq(const Batch& b, int page_tokens, int s, int* status) {
  Seq q;
  q.start = b.new_start[s];
  q.n = b.new_start[s + 1] - q.start;
  q.len = b.kv_len[s];
  if (q.start < 0 || q.n < 0 || q.start > b.tokens - q.n || q.n > b.max_new || q.len < 0 ||
      q.len > b.max_pages * page_tokens) {
    if (status) report_index(status);
    q.n = 0;
    q.len = 0;
  }
  return q;
}

// Sequence that packed token i belongs to, by the whole warp: the last s with
// new_start[s] <= i (32 probes a step).
__device__ __forceinline__ int find_seq(const Batch& b, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = b.seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int probe = lo + (lane + 1) * step;
    const bool le = probe < hi && b.new_start[probe] <= i;
    const int cnt = __popc(__ballot_sync(0xFFFFFFFFu, le));
    lo = min(lo + cnt * step, hi - 1);
    hi = min(hi, lo + step);
  }
  return lo;
}

// --- activations: 8 consecutive values, 16-byte aligned -------------------
template <int AT>
struct act_bytes { static constexpr int value = AT == RG_F32 ? 4 : 2; };

template <int AT>
__device__ __forceinline__ void load8(const void* base, int64_t elem, float (&x)[8]) {
  if constexpr (AT == RG_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (AT == RG_F16) {
        x[2 * i] = f16_to_f32(static_cast<uint16_t>(w[i] & 0xFFFFu));
        x[2 * i + 1] = f16_to_f32(static_cast<uint16_t>(w[i] >> 16));
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return BF ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}
template <int AT>
__device__ __forceinline__ void store8(void* base, int64_t elem, const float (&x)[8]) {
  if constexpr (AT == RG_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 v;
    v.x = pack16<AT == RG_BF16>(x[0], x[1]);
    v.y = pack16<AT == RG_BF16>(x[2], x[3]);
    v.z = pack16<AT == RG_BF16>(x[4], x[5]);
    v.w = pack16<AT == RG_BF16>(x[6], x[7]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = v;
  }
}

}  // namespace kv
}  // namespace rg
