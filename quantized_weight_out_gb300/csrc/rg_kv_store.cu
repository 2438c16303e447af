// rg_kv_store.cu - rg_kv_write and rg_kv_read: new tokens' keys and values into
// the paged cache in its storage type, and stored tokens back out.
//
// A warp handles one granule (16 tokens) of one head and kind, as far as the
// new tokens cover it, 32 dimensions at a time: lane (g, t), g = 2a + b, loads 8
// consecutive dimensions of tokens 4a + b and 4a + b + 2, so four lanes hold a
// token's block and two shuffles give its largest magnitude.  Keys leave in that
// arrangement; values are transposed by exchanges between the lanes that share
// the target words (no shared memory), or go out byte by byte when the granule is
// not whole (a byte belongs to one token).  Several blocks' loads are in flight at
// a time.  Bound by memory for prompts, by latency for single tokens.  Measured
// (GB300, a call inside a replayed graph): 121,000 tokens of 8 heads of 128 read back
// from Q8_0 as bf16 in 137 us, 5.5 TB/s of what has to move, four fifths of the copy
// bandwidth; prompts of 15,000 tokens stored in 30 us (instructions issued in 57 % of the
// cycles, a maximum, a product and a rounding per value, and latency for the rest) and read
// back in 21; one token each of 7 sequences stored and read back in 9 us, two launches.
#include "rg_kv.cuh"
#include "rg_kv_launch.h"

namespace rg {
namespace kv {
namespace {

constexpr int kWarps = 8;

// Codes of 8 values of two tokens whose 32-value blocks lie in lanes t = 0..3 of
// the same g: code[n][e], the int8 code's or the unsigned nibble's bits in the low
// byte (the rest is not zero; for blocks with zero[n] set, nothing is).  Returns the
// fp16 scale of token 0 in lane t = 0 and that of token 1 in lane t = 2.
template <int TYPE>
__device__ __forceinline__ uint16_t quantise8(const float (&x)[2][8], int t, uint32_t (&code)[2][8], bool (&zero)[2],
                                              int* status) {
  uint32_t big[2];
  float top[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    // the largest magnitude as an integer: infinities and NaN are larger than every finite value
    uint32_t m = 0;
    int first = 0;  // 2 * its first index + 1 if negative
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(x[n][e]) & 0x7FFFFFFFu;
      if (TYPE == RG_Q4_0 && b > m) first = 2 * (8 * t + e) + (__float_as_uint(x[n][e]) >> 31);
      m = max(m, b);
    }
    uint32_t v = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
    big[n] = v;
    top[n] = __uint_as_float(v);
    if constexpr (TYPE == RG_Q4_0) {
      if (m != v) first = 1 << 16;
      first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 1));
      first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 2));
      if (first & 1) top[n] = -top[n];
    }
  }
  constexpr float kSteps = TYPE == RG_Q8_0 ? 127.0f : -8.0f;
  // four lanes share four divisions: top / steps in t = 0 and 2, steps / top in t = 1 and 3
  const float mine = t & 2 ? top[1] : top[0];
  const float quotient = t & 1 ? kSteps / mine : mine / kSteps;
  uint16_t d = __half_as_ushort(__float2half_rn(quotient));
  const uint32_t mag = t & 2 ? big[1] : big[0];
  if (mag >= 0x7F800000u) d = 0x7E00;  // a value that is not finite: the block reads back as NaN
  // past the fp16 operands of the attention: 65504, and with d rounded up to 516 (from
  // 515.75) 127 d is 65532
  else if (__uint_as_float(mag) > (TYPE == RG_Q8_0 ? 65500.0f : 65504.0f)) report_range(status);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int lane = (threadIdx.x & 28) + 2 * n;
    const float inv = __shfl_sync(0xFFFFFFFFu, quotient, lane + 1);
    const uint16_t dn = static_cast<uint16_t>(__shfl_sync(0xFFFFFFFFu, static_cast<uint32_t>(d), lane));
    // a scale that rounds to zero, and a block that is not finite, have zero codes
    zero[n] = (dn & 0x7FFFu) == 0 || big[n] >= 0x7F800000u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // Adding 1.5 * 2^23 rounds to an integer (nearest even) and leaves it in the low bits.
      const uint32_t r = __float_as_uint(__fadd_rn(__fmul_rn(x[n][e], inv), 12582912.0f));
      // (Q4_0: -8 .. 8, of which 8 has no code and becomes 7; + 8)
      code[n][e] = TYPE == RG_Q8_0 ? r : min(r, 0x4B400007u) + 8u;
    }
  }
  return d;
}

// finite, and more than fp16's largest value
__device__ __forceinline__ bool beyond_f16(float x) { return fabsf(x) > 65504.0f && x - x == 0.0f; }

// the low bytes of four words
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A granule's share of the batch's new tokens.
struct Piece {
  int j0, cnt;   // tokens j0 .. j0 + cnt - 1 of the granule
  int token;     // packed token of j0
  int64_t off;   // byte offset of the granule of (kind 0, head 0)
  bool ok;
};

// The piece that starts at packed token i of sequence s, if one does: i is the
// first new token of its sequence, or the first token of its granule.
__device__ __forceinline__ bool piece_at(const Cache& c, const Batch& b, int i, int s, int gran_bytes, int* status,
                                         Piece* out) {
  const Seq q = load_seq(b, c.page_tokens, s, status);
  if (i < q.start || i >= q.start + q.n) return false;
  const int first = q.len - q.n;              // position of the first new token (negative: before the cache)
  const int pos = first + (i - q.start);
  if (!(pos < 0 || pos % kGranule == 0 || i == q.start)) return false;
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

// The pieces that start among a block's packed tokens, found by the lanes side by
// side (window 16) or by the whole warp (window 1).
struct Pieces {
  Piece mine;
  uint32_t starts;
  __device__ __forceinline__ void find(const Cache& c, const Batch& b, int window, int gran_bytes, int* status) {
    const int lane = threadIdx.x & 31, i = blockIdx.x * window + (window > 1 ? lane : 0);
    bool has = false;
    if (window == 1) {
      has = piece_at(c, b, i, find_seq(b, i), gran_bytes, status, &mine) && lane == 0;
    } else if (lane < window && i < b.tokens) {
      int lo = 0, hi = b.seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (b.new_start[mid] <= i)
          lo = mid;
        else
          hi = mid;
      }
      has = piece_at(c, b, i, lo, gran_bytes, status, &mine);
    }
    starts = __ballot_sync(0xFFFFFFFFu, has);
  }
  __device__ __forceinline__ bool next(Piece* p) {
    if (!starts) return false;
    const int l = __ffs(starts) - 1;
    starts &= starts - 1;
    p->j0 = __shfl_sync(0xFFFFFFFFu, mine.j0, l);
    p->cnt = __shfl_sync(0xFFFFFFFFu, mine.cnt, l);
    p->token = __shfl_sync(0xFFFFFFFFu, mine.token, l);
    p->off = __shfl_sync(0xFFFFFFFFu, mine.off, l);
    p->ok = __shfl_sync(0xFFFFFFFFu, static_cast<int>(mine.ok), l);
    return true;
  }
};

struct Rows {
  const void* p[2];        // keys, values (NULL: left out)
  int64_t t[2], h[2];      // element strides of tokens and heads
};
struct OutRows {
  void* p[2];
  int64_t t[2], h[2];
};

// 8 activations as loaded, and as F32.
template <int AT>
struct Raw {
  uint4 v[AT == RG_F32 ? 2 : 1];
};
template <int AT>
__device__ __forceinline__ Raw<AT> load_raw(const void* base, int64_t elem) {
  Raw<AT> r;
  if constexpr (AT == RG_F32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + elem);
    r.v[0] = __ldg(p);
    r.v[1] = __ldg(p + 1);
  } else {
    r.v[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem));
  }
  return r;
}
template <int AT>
__device__ __forceinline__ void raw_f32(const Raw<AT>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (AT == RG_F32) {
      const uint32_t u[4] = {r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
      x[i] = __uint_as_float(w[i]);
      x[4 + i] = __uint_as_float(u[i]);
    } else if constexpr (AT == RG_F16) {
      x[2 * i] = f16_to_f32(static_cast<uint16_t>(w[i] & 0xFFFFu));
      x[2 * i + 1] = f16_to_f32(static_cast<uint16_t>(w[i] >> 16));
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }
__device__ __forceinline__ uint32_t swap_lane(uint32_t x, int mask) { return __shfl_xor_sync(0xFFFFFFFFu, x, mask); }
// the e-th bytes of four words
__device__ __forceinline__ uint32_t gather_bytes(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t e) {
  const uint32_t s = e | ((4 + e) << 4);
  return prmt(prmt(w0, w1, s), prmt(w2, w3, s), 0x5410);
}

// --- values of a whole granule: lane (a, b, t) has dimensions 8t + e of tokens
// 4a + b (n = 0) and 4a + b + 2 (n = 1); the word of dimension e holds tokens 4a .. 4a + 3

// c[n][h]: codes e = 4h .. 4h + 3 as bytes.  Lane b writes the words of e = 4b .. 4b + 3.
__device__ __forceinline__ void put_values_q8(uint8_t* out, const uint32_t (&c)[2][2], int a, int b, int t) {
  const uint32_t m0 = b ? c[0][1] : c[0][0], m1 = b ? c[1][1] : c[1][0];
  const uint32_t p0 = swap_lane(b ? c[0][0] : c[0][1], 4), p1 = swap_lane(b ? c[1][0] : c[1][1], 4);
  const uint32_t x0 = b ? p0 : m0, y0 = b ? m0 : p0, x1 = b ? p1 : m1, y1 = b ? m1 : p1;
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e) {
    const uint32_t s = e | ((4 + e) << 4);
    *reinterpret_cast<uint32_t*>(out + (4 * b + e) * 64 + a * 16 + t * 4) = prmt(prmt(x0, y0, s), prmt(x1, y1, s), 0x5410);
  }
}
__device__ __forceinline__ void get_values_q8(const uint32_t (&w)[4], uint32_t (&c)[2][2], int b) {
  const uint32_t m0 = gather_bytes(w[0], w[1], w[2], w[3], b), m1 = gather_bytes(w[0], w[1], w[2], w[3], b + 2);
  const uint32_t p0 = swap_lane(gather_bytes(w[0], w[1], w[2], w[3], b ^ 1), 4);
  const uint32_t p1 = swap_lane(gather_bytes(w[0], w[1], w[2], w[3], (b ^ 1) + 2), 4);
  c[0][0] = b ? p0 : m0; c[0][1] = b ? m0 : p0;
  c[1][0] = b ? p1 : m1; c[1][1] = b ? m1 : p1;
}

// c[n]: codes e as nibbles.  A byte joins the nibbles of lanes t and t ^ 1 (dimensions 8t + e,
// 8(t ^ 1) + e), a word the bytes [b][n] of tokens 4a + b + 2n; lane (b, t % 2) writes the words
// of e = 4 (t % 2) + 2b and the next.
__device__ __forceinline__ void put_values_q4(uint8_t* out, const uint32_t (&c)[2], int a, int b, int t) {
  const int n = t & 1;
  const uint32_t other = swap_lane(n ? c[0] : c[1], 1);
  const uint32_t lo = n ? other : c[0], hi = n ? c[1] : other;  // token n: even and odd q
  const uint32_t even = (lo & 0x0F0F0F0Fu) | ((hi & 0x0F0F0F0Fu) << 4), odd = ((lo >> 4) & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u);
  const uint32_t e0 = prmt(even, odd, 0x5140), e1 = prmt(even, odd, 0x7362);  // e = 0 .. 3, 4 .. 7
  const uint32_t got = swap_lane(n ? e0 : e1, 1), own = n ? e1 : e0;
  const uint32_t n0 = n ? got : own, n1 = n ? own : got;                      // e = 4n .. 4n + 3 of both tokens
  const uint32_t first = prmt(n0, n1, 0x5410), second = prmt(n0, n1, 0x7632);
  const uint32_t keep = b ? second : first, r = swap_lane(b ? first : second, 4);
  const uint32_t b0 = b ? r : keep, b1 = b ? keep : r;
  uint8_t* to = out + (4 * n + 2 * b) * 32 + a * 8 + (t >> 1) * 4;
  *reinterpret_cast<uint32_t*>(to) = prmt(b0, b1, 0x6420);
  *reinterpret_cast<uint32_t*>(to + 32) = prmt(b0, b1, 0x7531);
}
// w: the words that put_values_q4 writes; c[n][h]: bytes of e = 4h .. 4h + 3 (both nibbles)
__device__ __forceinline__ void get_values_q4(const uint32_t (&w)[2], uint32_t (&c)[2][2], int b, int t) {
  const int n = t & 1;
  const uint32_t b0 = prmt(w[0], w[1], 0x5140), b1 = prmt(w[0], w[1], 0x7362);
  const uint32_t keep = b ? b1 : b0, r = swap_lane(b ? b0 : b1, 4);
  const uint32_t q0 = b ? r : keep, q1 = b ? keep : r;
  const uint32_t n0 = prmt(q0, q1, 0x5410), n1 = prmt(q0, q1, 0x7632);
  const uint32_t g0 = swap_lane(n0, 1), g1 = swap_lane(n1, 1);
  c[0][0] = n ? g0 : n0; c[0][1] = n ? n0 : g0;
  c[1][0] = n ? g1 : n1; c[1][1] = n ? n1 : g1;
}

// w[n][i]: dimensions 2i, 2i + 1 as halves.  Lane b writes the 8 bytes of e = 4b .. 4b + 3.
__device__ __forceinline__ void put_values_16(uint8_t* out, const uint32_t (&w)[2][4], int a, int b, int t) {
  uint32_t x[2][2], y[2][2];  // tokens of b = 0 and of b = 1
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t own = b ? w[n][2 + i] : w[n][i], got = swap_lane(b ? w[n][i] : w[n][2 + i], 4);
      x[n][i] = b ? got : own;
      y[n][i] = b ? own : got;
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t s = (e & 1) ? 0x7632 : 0x5410;
    *reinterpret_cast<uint2*>(out + (t >> 1) * 512 + (4 * b + e) * 64 + a * 16 + (t & 1) * 8) =
        make_uint2(prmt(x[0][e >> 1], y[0][e >> 1], s), prmt(x[1][e >> 1], y[1][e >> 1], s));
  }
}
__device__ __forceinline__ void get_values_16(const uint2 (&v)[4], uint32_t (&w)[2][4], int b) {
  const uint32_t mine = b ? 0x7632 : 0x5410, theirs = b ? 0x5410 : 0x7632;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t m0 = prmt(v[2 * i].x, v[2 * i + 1].x, mine), m1 = prmt(v[2 * i].y, v[2 * i + 1].y, mine);
    const uint32_t p0 = swap_lane(prmt(v[2 * i].x, v[2 * i + 1].x, theirs), 4);
    const uint32_t p1 = swap_lane(prmt(v[2 * i].y, v[2 * i + 1].y, theirs), 4);
    w[0][i] = b ? p0 : m0; w[0][2 + i] = b ? m0 : p0;
    w[1][i] = b ? p1 : m1; w[1][2 + i] = b ? m1 : p1;
  }
}

// the low nibbles of eight words: word e's at nibble e, or (KEYS) at nibble (e % 2) * 4 + e / 2
template <bool KEYS>
__device__ __forceinline__ uint32_t nibbles8(const uint32_t (&c)[8]) {
  const uint32_t even = bytes4(c[0], c[2], c[4], c[6]) & 0x0F0F0F0Fu, odd = bytes4(c[1], c[3], c[5], c[7]) & 0x0F0F0F0Fu;
  if constexpr (!KEYS) return even | (odd << 4);
  // even values in the low half, odd ones in the high half
  const uint32_t lo = even | (even >> 4), hi = odd | (odd >> 4);  // bytes 0 and 2 hold two nibbles each
  return __byte_perm(lo, hi, 0x6420);
}

// One block (32 dimensions) of up to 16 tokens into the cache.  out: the block's codes,
// scales: the block's scales.
template <int TYPE>
__device__ __forceinline__ void store_block(const float (&x)[2][8], uint8_t* out, uint16_t* scales, int kind, bool whole,
                                            const bool (&have)[2], int* status) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, a = g >> 1, b = g & 1, key0 = 4 * a + b;
  if constexpr (has_scales(TYPE)) {
    uint32_t code[2][8];
    bool zero[2];
    const uint16_t d = quantise8<TYPE>(x, t, code, zero, status);
    if ((t & 1) == 0 && (t ? have[1] : have[0])) scales[kind == 0 ? 2 * g + (t >> 1) : key0 + t] = d;
    if constexpr (TYPE == RG_Q8_0) {
      uint32_t c[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          c[n][i] =
              zero[n] ? 0u : bytes4(code[n][4 * i], code[n][4 * i + 1], code[n][4 * i + 2], code[n][4 * i + 3]);
      if (kind == 0) {
        if (whole) {
          reinterpret_cast<uint4*>(out)[lane] = make_uint4(c[0][0], c[0][1], c[1][0], c[1][1]);
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (have[n]) *reinterpret_cast<uint2*>(out + lane * 16 + 8 * n) = make_uint2(c[n][0], c[n][1]);
        }
      } else if (whole) {
        put_values_q8(out, c, a, b, t);
      } else {
        // dimension 8t + e of token j: [e][j / 4][t][j % 4]
#pragma unroll
        for (int n = 0; n < 2; ++n)
          if (have[n])
#pragma unroll
            for (int e = 0; e < 8; ++e)
              out[e * 64 + a * 16 + t * 4 + b + 2 * n] = static_cast<uint8_t>(c[n][e >> 2] >> (8 * (e & 3)));
      }
    } else if (kind == 0) {
      const uint32_t word[2] = {zero[0] ? 0x88888888u : nibbles8<true>(code[0]),
                                zero[1] ? 0x88888888u : nibbles8<true>(code[1])};
      if (whole) {
        reinterpret_cast<uint2*>(out)[lane] = make_uint2(word[0], word[1]);
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
          if (have[n]) *reinterpret_cast<uint32_t*>(out + lane * 8 + 4 * n) = word[n];
      }
    } else {
      const uint32_t c[2] = {zero[0] ? 0x88888888u : nibbles8<false>(code[0]),
                             zero[1] ? 0x88888888u : nibbles8<false>(code[1])};
      if (whole) {
        put_values_q4(out, c, a, b, t);
      } else {
        // lanes t and t ^ 1 share bytes: the even one writes token n = 0, the odd one n = 1
        const uint32_t other = swap_lane((t & 1) ? c[0] : c[1], 1);
        const uint32_t lo = (t & 1) ? other : c[0], hi = (t & 1) ? c[1] : other;
        if ((t & 1) ? have[1] : have[0])
#pragma unroll
          for (int e = 0; e < 8; ++e)
            out[e * 32 + a * 8 + (t >> 1) * 4 + b * 2 + (t & 1)] =
                static_cast<uint8_t>(((lo >> (4 * e)) & 15u) | (((hi >> (4 * e)) & 15u) << 4));
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
        if constexpr (BF)
          over |= overflowed16<BF>(x[n][2 * e], word[n][e]) || overflowed16<BF>(x[n][2 * e + 1], word[n][e] >> 16);
        else
          over |= beyond_f16(x[n][2 * e]) || beyond_f16(x[n][2 * e + 1]);
      }
    if (over) report_range(status);
    if (kind == 0) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (have[n])
          reinterpret_cast<uint4*>(out)[n * 32 + lane] = make_uint4(word[n][0], word[n][1], word[n][2], word[n][3]);
    } else if (whole) {
      put_values_16(out, word, a, b, t);
    } else {
      // dimension 8t + e of token j: [t / 2][e][j / 4][t % 2][j % 4]
      uint16_t* to = reinterpret_cast<uint16_t*>(out) + (t >> 1) * 256 + a * 8 + (t & 1) * 4 + b;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (have[n])
#pragma unroll
          for (int e = 0; e < 8; ++e) to[e * 32 + 2 * n] = static_cast<uint16_t>(word[n][e >> 1] >> (16 * (e & 1)));
    }
  }
}

// blocks of 32 dimensions whose loads are in flight together
template <int AT>
constexpr int kAhead = AT == RG_F32 ? 2 : 4;

// grid (windows of `window` packed tokens, groups of kWarps (head, kind) pairs)
template <int TYPE, int AT>
__global__ void __launch_bounds__(32 * kWarps, AT == RG_F32 ? 2 : 3) kv_write_kernel(Cache c, Batch b, Rows in, int window, int* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.y * kWarps + warp;
  if (unit >= 2 * c.kv_heads) return;
  const int kind = unit / c.kv_heads, head = unit % c.kv_heads;
  const void* src = in.p[kind];
  if (!src) return;
  const int blocks = c.dim / 32, key0 = 4 * (g >> 1) + (g & 1);
  Pieces pieces;
  pieces.find(c, b, window, granule_bytes(TYPE, c.dim), status);
  Piece pc;
  while (pieces.next(&pc)) {
    if (!pc.ok) continue;
    uint8_t* dst = c.data + pc.off + (static_cast<int64_t>(kind) * c.kv_heads + head) * c.slab_bytes;
    uint16_t* scales = reinterpret_cast<uint16_t*>(dst + blocks * block16_bytes(TYPE));
    bool have[2];
    int64_t at[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = key0 + 2 * n;
      have[n] = j >= pc.j0 && j < pc.j0 + pc.cnt;
      // (a token that is not there loads the piece's first: no branch around the loads)
      at[n] = (pc.token + (have[n] ? j - pc.j0 : 0)) * in.t[kind] + head * in.h[kind] + 8 * t;
    }
    for (int blk = 0; blk < blocks; blk += kAhead<AT>) {
      Raw<AT> raw[kAhead<AT>][2];
#pragma unroll
      for (int u = 0; u < kAhead<AT>; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n) raw[u][n] = load_raw<AT>(src, at[n] + 32 * min(blk + u, blocks - 1));
#pragma unroll
      for (int u = 0; u < kAhead<AT>; ++u) {
        if (blk + u >= blocks) break;
        float x[2][8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          raw_f32<AT>(raw[u][n], x[n]);
          if (pc.cnt < kGranule)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[n][e] = have[n] ? x[n][e] : 0.0f;
        }
        store_block<TYPE>(x, dst + (blk + u) * block16_bytes(TYPE), scales + 16 * (blk + u), kind, pc.cnt == kGranule,
                          have, status);
      }
    }
  }
}

// The stored words of one block, as loaded.
template <int TYPE>
struct Stored {
  uint32_t w[TYPE == RG_Q8_0 ? 4 : TYPE == RG_Q4_0 ? 2 : 8];
  uint32_t d;  // scales of the lane's two tokens
};
template <int TYPE>
__device__ __forceinline__ Stored<TYPE> load_stored(const uint8_t* in, const uint16_t* scales, int kind) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, a = g >> 1, b = g & 1;
  Stored<TYPE> s;
  if constexpr (has_scales(TYPE)) {
    if (kind == 0) {
      s.d = __ldg(reinterpret_cast<const uint32_t*>(scales) + g);
    } else {
      const uint32_t d0 = __ldg(scales + 4 * a + b), d1 = __ldg(scales + 4 * a + b + 2);
      s.d = d0 | (d1 << 16);
    }
  }
  if constexpr (TYPE == RG_Q8_0) {
    if (kind == 0) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(in) + lane);
      s.w[0] = v.x; s.w[1] = v.y; s.w[2] = v.z; s.w[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s.w[e] = __ldg(reinterpret_cast<const uint32_t*>(in + (4 * b + e) * 64 + a * 16 + t * 4));
    }
  } else if constexpr (TYPE == RG_Q4_0) {
    if (kind == 0) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(in) + lane);
      s.w[0] = v.x; s.w[1] = v.y;
    } else {
      const uint8_t* p = in + (4 * (t & 1) + 2 * b) * 32 + a * 8 + (t >> 1) * 4;
      s.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      s.w[1] = __ldg(reinterpret_cast<const uint32_t*>(p + 32));
    }
  } else {
    if (kind == 0) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(in) + n * 32 + lane);
        s.w[4 * n] = v.x; s.w[4 * n + 1] = v.y; s.w[4 * n + 2] = v.z; s.w[4 * n + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint2 v =
            __ldg(reinterpret_cast<const uint2*>(in + (t >> 1) * 512 + (4 * b + e) * 64 + a * 16 + (t & 1) * 8));
        s.w[2 * e] = v.x; s.w[2 * e + 1] = v.y;
      }
    }
  }
  return s;
}
template <int TYPE>
__device__ __forceinline__ void stored_f32(const Stored<TYPE>& s, int kind, float (&x)[2][8]) {
  const int lane = threadIdx.x & 31, t = lane & 3, b = (lane >> 2) & 1;
  if constexpr (has_scales(TYPE)) {
    const float d[2] = {f16_to_f32(static_cast<uint16_t>(s.d & 0xFFFFu)), f16_to_f32(static_cast<uint16_t>(s.d >> 16))};
    if constexpr (TYPE == RG_Q8_0) {
      uint32_t c[2][2] = {{s.w[0], s.w[1]}, {s.w[2], s.w[3]}};
      if (kind != 0) get_values_q8(s.w, c, b);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[n][e] = d[n] * static_cast<float>(static_cast<int8_t>(c[n][e >> 2] >> (8 * (e & 3))));
    } else if (kind == 0) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[n][e] = d[n] * static_cast<float>(static_cast<int>((s.w[n] >> (4 * ((e & 1) * 4 + (e >> 1)))) & 15u) - 8);
    } else {
      uint32_t c[2][2];
      get_values_q4(s.w, c, b, t);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[n][e] = d[n] * static_cast<float>(static_cast<int>((c[n][e >> 2] >> (8 * (e & 3) + 4 * (t & 1))) & 15u) - 8);
    }
  } else {
    constexpr bool BF = TYPE == RG_BF16;
    uint32_t w[2][4];
    if (kind == 0) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[n][i] = s.w[4 * n + i];
    } else {
      const uint2 v[4] = {make_uint2(s.w[0], s.w[1]), make_uint2(s.w[2], s.w[3]), make_uint2(s.w[4], s.w[5]),
                          make_uint2(s.w[6], s.w[7])};
      get_values_16(v, w, b);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t h = static_cast<uint16_t>(w[n][e >> 1] >> (16 * (e & 1)));
        x[n][e] = BF ? bf16_to_f32(h) : f16_to_f32(h);
      }
  }
}

template <int TYPE, int AT>
__global__ void __launch_bounds__(32 * kWarps, 4) kv_read_kernel(Cache c, Batch b, OutRows to, int window, int* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.y * kWarps + warp;
  if (unit >= 2 * c.kv_heads) return;
  const int kind = unit / c.kv_heads, head = unit % c.kv_heads;
  void* dst = to.p[kind];
  if (!dst) return;
  const int blocks = c.dim / 32, key0 = 4 * (g >> 1) + (g & 1);
  constexpr int U = has_scales(TYPE) ? 4 : 2;
  Pieces pieces;
  pieces.find(c, b, window, granule_bytes(TYPE, c.dim), status);
  Piece pc;
  while (pieces.next(&pc)) {
    const uint8_t* src = c.data + pc.off + (static_cast<int64_t>(kind) * c.kv_heads + head) * c.slab_bytes;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(src + blocks * block16_bytes(TYPE));
    bool have[2];
    int64_t at[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = key0 + 2 * n;
      have[n] = j >= pc.j0 && j < pc.j0 + pc.cnt;
      at[n] = (pc.token + j - pc.j0) * to.t[kind] + head * to.h[kind] + 8 * t;
    }
    for (int blk = 0; blk < blocks; blk += U) {
      Stored<TYPE> s[U] = {};
      if (pc.ok) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = min(blk + u, blocks - 1);
          s[u] = load_stored<TYPE>(src + k * block16_bytes(TYPE), scales + 16 * k, kind);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (blk + u >= blocks) break;
        float x[2][8];
        stored_f32<TYPE>(s[u], kind, x);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (!pc.ok) {  // no place in the cache: zeros
#pragma unroll
            for (int e = 0; e < 8; ++e) x[n][e] = 0.0f;
          }
          if (have[n]) store8<AT>(dst, at[n] + 32 * (blk + u), x[n]);
        }
      }
    }
  }
}

// Packed tokens a block looks through for granules that start there: 16 (one
// granule, mostly) once a sequence brings more than that many tokens, else one, so
// that many sequences' single tokens are handled side by side.  Stored and read
// back: prompts of 15,000 tokens 53 us with 16 against 154 with one, one token each of
// 7 / 64 / 256 sequences 9 / 10 / 18 us with one against 38 / 82 / 84 with 16.
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
