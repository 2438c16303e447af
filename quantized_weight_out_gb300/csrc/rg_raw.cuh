// rg_raw.cuh - the exact F32 decode of a row's 256-value tile by a warp, eight
// values a lane: the bytes that a lane needs by a few wide loads, then their
// values (the small-T kernels, and the lookup of table rows).
#pragma once

#include "rg_internal.cuh"

namespace rg {
namespace smt {

// Bytes of one row's 256-value tile.
template <int WT>
__host__ __device__ constexpr int tile_bytes() {
  return (256 / block_values(WT)) * block_bytes(WT);
}

// Raw bytes one lane needs from a row for its 8 values (a 256-value tile).
template <int WT>
struct Raw {
  uint32_t v[WT == RG_Q5_K || WT == RG_F32 ? 8
             : WT == RG_Q4_K                  ? 6
             : WT == RG_Q6_K || WT == RG_Q3_K ? 5
             : (WT == RG_Q8_0 || WT == RG_Q4_0 || WT == RG_Q4_1 || WT == RG_MXFP4 ||
                WT == RG_NVFP4)                                                       ? 3
                                                                                    : 4];
};

// The bytes one lane needs for its 8 values, from a row tile staged in
// shared memory, or in place (tile: the row's 256-value tile, aligned as its type's
// rows of whole tiles are).
template <int WT>
__device__ __forceinline__ void load_raw_smem(const uint8_t* tile, int lane, Raw<WT>& r) {
  if constexpr (WT == RG_F32) {
    const uint4 a = reinterpret_cast<const uint4*>(tile)[2 * lane];
    const uint4 b = reinterpret_cast<const uint4*>(tile)[2 * lane + 1];
    r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
    r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
  } else if constexpr (WT == RG_F16 || WT == RG_BF16) {
    const uint4 q = reinterpret_cast<const uint4*>(tile)[lane];
    r.v[0] = q.x; r.v[1] = q.y; r.v[2] = q.z; r.v[3] = q.w;
  } else if constexpr (WT == RG_Q8_0 || WT == RG_Q4_0) {
    constexpr int BB = WT == RG_Q8_0 ? 34 : 18;
    const uint8_t* blk = tile + BB * (lane >> 2);
    const uint8_t* q = blk + 2 + 8 * (WT == RG_Q8_0 ? (lane & 3) : (lane & 1));
    const uint16_t* q16 = reinterpret_cast<const uint16_t*>(q);
    r.v[0] = *reinterpret_cast<const uint16_t*>(blk);
    r.v[1] = static_cast<uint32_t>(q16[0]) | (static_cast<uint32_t>(q16[1]) << 16);
    r.v[2] = static_cast<uint32_t>(q16[2]) | (static_cast<uint32_t>(q16[3]) << 16);
  } else if constexpr (WT == RG_MXFP4) {
    // values 8(lane & 3) .. +7 of block lane >> 2 (17-byte blocks from an
    // 8-byte aligned tile): the scale byte and 8 bytes of nibbles
    const uint8_t* blk = tile + 17 * (lane >> 2);
    const uint8_t* q = blk + 1 + 8 * (lane & 1);
    r.v[0] = blk[0];
    r.v[1] = static_cast<uint32_t>(q[0]) | (static_cast<uint32_t>(q[1]) << 8) |
             (static_cast<uint32_t>(q[2]) << 16) | (static_cast<uint32_t>(q[3]) << 24);
    r.v[2] = static_cast<uint32_t>(q[4]) | (static_cast<uint32_t>(q[5]) << 8) |
             (static_cast<uint32_t>(q[6]) << 16) | (static_cast<uint32_t>(q[7]) << 24);
  } else if constexpr (WT == RG_NVFP4) {
    // values 8 lane .. +7: micro-block s = (lane & 7) >> 1 of block lane >> 3
    // (36-byte blocks from a 16-byte aligned tile): its scale byte and its 8
    // code bytes (low nibbles for even lanes, high for odd)
    const uint8_t* blk = tile + 36 * (lane >> 3);
    const int s = (lane & 7) >> 1;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(blk + 4 + 8 * s);
    r.v[0] = blk[s];
    r.v[1] = q[0];
    r.v[2] = q[1];
  } else if constexpr (WT == RG_Q4_1) {
    const uint8_t* blk = tile + 20 * (lane >> 2);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(blk + 4 + 8 * (lane & 1));
    r.v[0] = *reinterpret_cast<const uint32_t*>(blk);  // d | m << 16
    r.v[1] = q[0];
    r.v[2] = q[1];
  } else if constexpr (WT == RG_Q5_0) {
    const uint8_t* blk = tile + 22 * (lane >> 2);
    const uint16_t* h16 = reinterpret_cast<const uint16_t*>(blk + 2);
    const uint16_t* q16 = reinterpret_cast<const uint16_t*>(blk + 6 + 8 * (lane & 1));
    r.v[0] = *reinterpret_cast<const uint16_t*>(blk);
    r.v[1] = static_cast<uint32_t>(h16[0]) | (static_cast<uint32_t>(h16[1]) << 16);
    r.v[2] = static_cast<uint32_t>(q16[0]) | (static_cast<uint32_t>(q16[1]) << 16);
    r.v[3] = static_cast<uint32_t>(q16[2]) | (static_cast<uint32_t>(q16[3]) << 16);
  } else if constexpr (WT == RG_Q5_1) {
    const uint8_t* blk = tile + 24 * (lane >> 2);
    const uint2 q = *reinterpret_cast<const uint2*>(blk + 8 + 8 * (lane & 1));
    r.v[0] = *reinterpret_cast<const uint32_t*>(blk);      // d | m << 16
    r.v[1] = *reinterpret_cast<const uint32_t*>(blk + 4);  // qh
    r.v[2] = q.x;
    r.v[3] = q.y;
  } else if constexpr (WT == RG_Q6_K) {
    // values 8*lane .. +7 = 128h + 32i + l0 .. +7 (tile: the super-block's
    // first byte, 2-byte aligned): 8 bytes of ql, 8 of qh, one scale, d
    const int h = lane >> 4, i = (lane >> 2) & 3, l0 = 8 * (lane & 3);
    const uint16_t* ql = reinterpret_cast<const uint16_t*>(tile + 64 * h + 32 * (i & 1) + l0);
    const uint16_t* qh = reinterpret_cast<const uint16_t*>(tile + 128 + 32 * h + l0);
    r.v[0] = static_cast<uint32_t>(ql[0]) | (static_cast<uint32_t>(ql[1]) << 16);
    r.v[1] = static_cast<uint32_t>(ql[2]) | (static_cast<uint32_t>(ql[3]) << 16);
    r.v[2] = static_cast<uint32_t>(qh[0]) | (static_cast<uint32_t>(qh[1]) << 16);
    r.v[3] = static_cast<uint32_t>(qh[2]) | (static_cast<uint32_t>(qh[3]) << 16);
    r.v[4] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(tile + 208)) |
             (static_cast<uint32_t>(tile[192 + (lane >> 1)]) << 16);
  } else if constexpr (WT == RG_Q2_K || WT == RG_Q3_K) {
    // values 8*lane .. +7 = 128h + 32j + 16s + l0 .. +7 (tile: the
    // super-block's first byte, 2-byte aligned): 8 bytes of qs (and of
    // hmask), the sub-block's scale byte(s), d (and dmin)
    const int h = lane >> 4, j = (lane >> 2) & 3, sb = (lane >> 1) & 1, l0 = 8 * (lane & 1);
    constexpr int QS = WT == RG_Q2_K ? 16 : 32;
    const uint16_t* q = reinterpret_cast<const uint16_t*>(tile + QS + 32 * h + 16 * sb + l0);
    r.v[0] = static_cast<uint32_t>(q[0]) | (static_cast<uint32_t>(q[1]) << 16);
    r.v[1] = static_cast<uint32_t>(q[2]) | (static_cast<uint32_t>(q[3]) << 16);
    const int si = 8 * h + 2 * j + sb;
    if constexpr (WT == RG_Q2_K) {
      r.v[2] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(tile + 80)) |
               (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(tile + 82)) << 16);
      r.v[3] = tile[si];
    } else {
      const uint16_t* hm = reinterpret_cast<const uint16_t*>(tile + 16 * sb + l0);
      r.v[2] = static_cast<uint32_t>(hm[0]) | (static_cast<uint32_t>(hm[1]) << 16);
      r.v[3] = static_cast<uint32_t>(hm[2]) | (static_cast<uint32_t>(hm[3]) << 16);
      // d, the byte with the scale's low nibble, the byte with its high bits
      r.v[4] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(tile + 108)) |
               (static_cast<uint32_t>(tile[96 + (si & 7)]) << 16) |
               (static_cast<uint32_t>(tile[104 + (si & 3)]) << 24);
    }
  } else {
    // Q4_K, Q5_K: the header, this lane's 8 bytes of nibbles (and of qh)
    constexpr int QS = WT == RG_Q5_K ? 48 : 16;
    const uint4 h = *reinterpret_cast<const uint4*>(tile);
    const int c = lane >> 3, l0 = 8 * (lane & 3);
    const uint2 q = *reinterpret_cast<const uint2*>(tile + QS + 32 * c + l0);
    r.v[0] = h.x; r.v[1] = h.y; r.v[2] = h.z; r.v[3] = h.w; r.v[4] = q.x; r.v[5] = q.y;
    if constexpr (WT == RG_Q5_K) {
      const uint2 qh = *reinterpret_cast<const uint2*>(tile + 16 + l0);
      r.v[6] = qh.x;
      r.v[7] = qh.y;
    }
  }
}

__device__ __forceinline__ int byte_at(const uint32_t* w, int i) {
  return static_cast<int>((w[i >> 2] >> (8 * (i & 3))) & 0xFFu);
}

// Exact F32 decode of the lane's 8 values: the same products and single
// rounding as the format definitions (signed zeros kept).
template <int WT>
__device__ __forceinline__ void decode_raw(const Raw<WT>& r, int lane, float (&w)[8]) {
  if constexpr (WT == RG_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __uint_as_float(r.v[i]);
  } else if constexpr (WT == RG_F16 || WT == RG_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t lo = static_cast<uint16_t>(r.v[i] & 0xFFFFu);
      const uint16_t hi = static_cast<uint16_t>(r.v[i] >> 16);
      w[2 * i] = WT == RG_F16 ? f16_to_f32(lo) : bf16_to_f32(lo);
      w[2 * i + 1] = WT == RG_F16 ? f16_to_f32(hi) : bf16_to_f32(hi);
    }
  } else if constexpr (WT == RG_Q8_0) {
    // int8 q as the byte q + 128, then d * q: an exact product
    const float d = f16_to_f32(static_cast<uint16_t>(r.v[0]));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = r.v[1 + j] ^ 0x80808080u;
      w[4 * j + 0] = d * byte_minus<0>(x, kTwo23 + 128.0f);
      w[4 * j + 1] = d * byte_minus<1>(x, kTwo23 + 128.0f);
      w[4 * j + 2] = d * byte_minus<2>(x, kTwo23 + 128.0f);
      w[4 * j + 3] = d * byte_minus<3>(x, kTwo23 + 128.0f);
    }
  } else if constexpr (WT == RG_Q4_0) {
    const float d = f16_to_f32(static_cast<uint16_t>(r.v[0]));
    const int shift = (lane & 2) ? 4 : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = (r.v[1 + j] >> shift) & 0x0F0F0F0Fu;
      w[4 * j + 0] = d * byte_minus<0>(x, kTwo23 + 8.0f);
      w[4 * j + 1] = d * byte_minus<1>(x, kTwo23 + 8.0f);
      w[4 * j + 2] = d * byte_minus<2>(x, kTwo23 + 8.0f);
      w[4 * j + 3] = d * byte_minus<3>(x, kTwo23 + 8.0f);
    }
  } else if constexpr (WT == RG_MXFP4) {
    // E2M1(code) * 2^(e - 127): exact (low nibbles for the first 16 values
    // of the block, high nibbles for the rest)
    const float sc = e8m0_f32(r.v[0]);
    const int shift = (lane & 2) ? 4 : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = r.v[1 + j] >> shift;
#pragma unroll
      for (int b = 0; b < 4; ++b) w[4 * j + b] = e2m1_f32((x >> (8 * b)) & 15u) * sc;
    }
  } else if constexpr (WT == RG_NVFP4) {
    // E2M1(code) * E4M3(scale): exact
    const float sc = e4m3_f32(r.v[0]);
    const int shift = (lane & 1) ? 4 : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = r.v[1 + j] >> shift;
#pragma unroll
      for (int b = 0; b < 4; ++b) w[4 * j + b] = e2m1_f32((x >> (8 * b)) & 15u) * sc;
    }
  } else if constexpr (WT == RG_Q6_K) {
    // (d * sc) * (q - 32), every step exact
    const int i = (lane >> 2) & 3;
    const float ds = f16_to_f32(static_cast<uint16_t>(r.v[4] & 0xFFFFu)) *
                     static_cast<float>(static_cast<int8_t>((r.v[4] >> 16) & 0xFFu));
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const uint32_t x = ((r.v[jj] >> (i >= 2 ? 4 : 0)) & 0x0F0F0F0Fu) |
                         (((r.v[2 + jj] >> (2 * i)) & 0x03030303u) << 4);
      w[4 * jj + 0] = ds * byte_minus<0>(x, kTwo23 + 32.0f);
      w[4 * jj + 1] = ds * byte_minus<1>(x, kTwo23 + 32.0f);
      w[4 * jj + 2] = ds * byte_minus<2>(x, kTwo23 + 32.0f);
      w[4 * jj + 3] = ds * byte_minus<3>(x, kTwo23 + 32.0f);
    }
  } else if constexpr (WT == RG_Q2_K) {
    // (d * sc) * q exact, minus dmin * m: one rounding, like the definition
    const int j = (lane >> 2) & 3;
    const float ds = f16_to_f32(static_cast<uint16_t>(r.v[2] & 0xFFFFu)) * static_cast<float>(r.v[3] & 15u);
    const float ndm = -(f16_to_f32(static_cast<uint16_t>(r.v[2] >> 16)) * static_cast<float>(r.v[3] >> 4));
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const uint32_t x = (r.v[jj] >> (2 * j)) & 0x03030303u;
      w[4 * jj + 0] = fmaf(ds, byte_minus<0>(x, kTwo23), ndm);
      w[4 * jj + 1] = fmaf(ds, byte_minus<1>(x, kTwo23), ndm);
      w[4 * jj + 2] = fmaf(ds, byte_minus<2>(x, kTwo23), ndm);
      w[4 * jj + 3] = fmaf(ds, byte_minus<3>(x, kTwo23), ndm);
    }
  } else if constexpr (WT == RG_Q3_K) {
    // q + 4 = low bits | third bit << 2; (d * (sc - 32)) * q, all exact
    const int h = lane >> 4, j = (lane >> 2) & 3, sb = (lane >> 1) & 1;
    const int si = 8 * h + 2 * j + sb;
    const uint32_t lob = (r.v[4] >> 16) & 0xFFu, hib = r.v[4] >> 24;
    const int sc = static_cast<int>(((si < 8 ? lob : lob >> 4) & 15u) | (((hib >> (2 * (si >> 2))) & 3u) << 4)) - 32;
    const float ds = f16_to_f32(static_cast<uint16_t>(r.v[4] & 0xFFFFu)) * static_cast<float>(sc);
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const uint32_t x = ((r.v[jj] >> (2 * j)) & 0x03030303u) |
                         (((r.v[2 + jj] >> (4 * h + j)) & 0x01010101u) << 2);
      w[4 * jj + 0] = ds * byte_minus<0>(x, kTwo23 + 4.0f);
      w[4 * jj + 1] = ds * byte_minus<1>(x, kTwo23 + 4.0f);
      w[4 * jj + 2] = ds * byte_minus<2>(x, kTwo23 + 4.0f);
      w[4 * jj + 3] = ds * byte_minus<3>(x, kTwo23 + 4.0f);
    }
  } else if constexpr (WT == RG_Q4_1 || WT == RG_Q5_0 || WT == RG_Q5_1) {
    // values 8(lane & 3) .. +7 of block lane >> 2: nibbles (low for the
    // first 16 values of the block, high for the rest) and the fifth bits
    constexpr int Q0 = WT == RG_Q4_1 ? 1 : 2;
    const float d = f16_to_f32(static_cast<uint16_t>(r.v[0] & 0xFFFFu));
    const float m = WT == RG_Q5_0 ? 0.0f : f16_to_f32(static_cast<uint16_t>(r.v[0] >> 16));
    const int j0 = 8 * (lane & 3);
    const int shift = j0 >= 16 ? 4 : 0;
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      uint32_t x = (r.v[Q0 + jj] >> shift) & 0x0F0F0F0Fu;
      if constexpr (WT != RG_Q4_1) x |= fifth_bits4(r.v[1] >> (j0 + 4 * jj));
      if constexpr (WT == RG_Q5_0) {
        w[4 * jj + 0] = d * byte_minus<0>(x, kTwo23 + 16.0f);
        w[4 * jj + 1] = d * byte_minus<1>(x, kTwo23 + 16.0f);
        w[4 * jj + 2] = d * byte_minus<2>(x, kTwo23 + 16.0f);
        w[4 * jj + 3] = d * byte_minus<3>(x, kTwo23 + 16.0f);
      } else {  // exact product, one rounding of the sum
        w[4 * jj + 0] = fmaf(d, byte_minus<0>(x, kTwo23), m);
        w[4 * jj + 1] = fmaf(d, byte_minus<1>(x, kTwo23), m);
        w[4 * jj + 2] = fmaf(d, byte_minus<2>(x, kTwo23), m);
        w[4 * jj + 3] = fmaf(d, byte_minus<3>(x, kTwo23), m);
      }
    }
  } else {
    const float d = f16_to_f32(static_cast<uint16_t>(r.v[0] & 0xFFFFu));
    const float dmin = f16_to_f32(static_cast<uint16_t>(r.v[0] >> 16));
    const int c = lane >> 3, half = (lane >> 2) & 1;
    const int j = 2 * c + half;  // sub-block
    const uint32_t* S = &r.v[1];
    int sc, m;
    if (j < 4) {
      sc = byte_at(S, j) & 63;
      m = byte_at(S, j + 4) & 63;
    } else {
      sc = (byte_at(S, j + 4) & 15) | ((byte_at(S, j - 4) >> 6) << 4);
      m = (byte_at(S, j + 4) >> 4) | ((byte_at(S, j) >> 6) << 4);
    }
    // (d * sc) * q - dmin * m: the product is exact (at most 21 bits), so the
    // fused form rounds once, like the definition
    const float ds = d * static_cast<float>(sc);
    const float ndm = -(dmin * static_cast<float>(m));
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      uint32_t x = (r.v[4 + jj] >> (4 * half)) & 0x0F0F0F0Fu;
      if constexpr (WT == RG_Q5_K) x |= ((r.v[6 + jj] >> j) & 0x01010101u) << 4;
      w[4 * jj + 0] = fmaf(ds, byte_minus<0>(x, kTwo23), ndm);
      w[4 * jj + 1] = fmaf(ds, byte_minus<1>(x, kTwo23), ndm);
      w[4 * jj + 2] = fmaf(ds, byte_minus<2>(x, kTwo23), ndm);
      w[4 * jj + 3] = fmaf(ds, byte_minus<3>(x, kTwo23), ndm);
    }
  }
}

}  // namespace smt
}  // namespace rg
