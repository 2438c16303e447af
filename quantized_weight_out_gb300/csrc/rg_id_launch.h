// rg_id_launch.h - host-side launchers of the indexed calls: table rows by
// token, the router, and the experts' products by slot (not part of the
// public C ABI).
#pragma once

#include "rg_internal.cuh"
#include "rg_launch.h"

namespace rg {
namespace id {

inline int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

// --- rows of a table (rg_rows.cu) ---
cudaError_t launch_get_rows(int wtype, const void* W, int64_t N, int64_t K, const int32_t* ids, int64_t n,
                            float scale, int atype, void* out, int64_t out_row, const DevInfo& dev,
                            cudaStream_t stream);

// Sorting n ids below `groups` (rg_sort.cu): the bytes of its workspace, and
// order = the positions sorted by (id, position), those of no group (negative,
// or out of range, which is reported) behind the others; sorted (may be NULL):
// the ids in that order, `groups` where there is none; start (may be NULL, only
// for groups <= kMaxExperts): where each group begins, and where the last ends.
// after_prev: the launch may overlap the kernel before it (it waits for its end).
size_t sort_workspace(int64_t n, int64_t groups);
cudaError_t launch_sort(const int32_t* ids, int64_t n, int64_t groups, int32_t* start, int32_t* order,
                        int32_t* sorted, void* ws, const DevInfo& dev, cudaStream_t stream,
                        bool after_prev = true);

// G[r, :] = beta * G[r, :] + scale * sum of dY's rows whose id is r.
size_t rows_back_workspace(int64_t n, int64_t N, int64_t K);
cudaError_t launch_rows_back(int atype, const void* dY, int64_t dy_row, const int32_t* ids, int64_t n, float scale,
                             float* G, int64_t g_row, int64_t N, int64_t K, float beta, void* ws, const DevInfo& dev,
                             cudaStream_t stream);

// --- the router (rg_route.cu) ---
constexpr int kMaxExperts = 1024;
constexpr int kMaxChosen = 32;
// (start and order: both NULL, or what launch_sort gives for ids)
cudaError_t launch_route(const float* logits, int64_t l_row, int64_t T, int experts, int top, int mode, float scale,
                         int32_t* ids, float* weights, int32_t* start, int32_t* order, const DevInfo& dev,
                         cudaStream_t stream);
cudaError_t launch_route_back(const float* logits, int64_t l_row, int64_t T, int experts, int top, int mode,
                              float scale, const int32_t* ids, const float* dweights, float* dlogits, int64_t dl_row,
                              const DevInfo& dev, cudaStream_t stream);

// --- products by slot ---

// A batch of slots, checked; rows of a product are `slots` or slots / per_token.
struct Batch {
  int experts, per_token;
  int slots;
  const int32_t* start;
  const int32_t* order;
};
// One product: fwd Y = X . deq(W_e)^T, else dX = dY . deq(W_e).  `wide` values
// of an input row, `out_w` of an output row.
struct Product {
  bool fwd;
  int wtype;
  const void* W;        // rows padded_row_bytes apart once a launch of the tensor cores has it
  int64_t N, K;
  int atype;
  const void* in;
  int64_t in_row;
  bool in_tokens;       // a row of `in` per token, else per slot
  void* out;
  int64_t out_row;
  bool out_tokens;      // a row of `out` per token: the sum over its slots
  const float* weights; // per slot, may be NULL
  float beta;
  int64_t wide() const { return fwd ? K : N; }
  int64_t out_w() const { return fwd ? N : K; }
};

// Rows of the tile table: one tile is up to `bt` slots of one expert.
struct Tile {
  int expert, first, rows, tile0;  // the expert's first sorted slot, its slots, its first tile's number
};

// Slots of a table's tile, given to the kernels by value.
struct Slots {
  const Tile* tiles;
  const int* n_tiles;
  const int32_t* order;
  int slots, per_token;
  const float* unscale;   // per sorted slot: what undoes the input copy's power of two (NULL: 1)
  const float* weights;   // per slot (NULL: 1)
  void* out;
  int64_t out_row;
  int otype;              // RG_F32, RG_F16 or RG_BF16
  float beta;
  uint8_t* live;          // per slot (NULL: not wanted): set for the slots whose rows are written
};

constexpr int64_t max_tiles(int64_t slots, int64_t experts, int64_t bt) {
  return slots / bt + (experts < slots ? experts : slots);
}

// rg_id.cu: the tile table; the input's 16-bit copy in sorted order (x16 NULL: the table alone), rows ld
// apart, each row scaled by a power of two (fp16 copies) whose inverse goes to `unscale`; `live` [slots]
// (may be NULL) is cleared, for the product's kernel to set.
cudaError_t launch_gather(const Batch& b, int bt, Tile* tiles, int* n_tiles, int cap, const Product& p, bool bf16,
                          uint16_t* x16, int64_t ld, float* unscale, uint8_t* live, const DevInfo& dev,
                          cudaStream_t stream);
// out[t] = beta * out[t] + sum of its live slots' rows (F32, by slot, `width` values), each times its weight.
cudaError_t launch_join(const float* rows, int64_t width, const uint8_t* live, const Batch& b, const Product& p,
                        const DevInfo& dev, cudaStream_t stream);
// Rows of W from one to the next, in bytes: as W lies, and as TMA can address them (multiples of 16).
inline int64_t row_bytes(int wtype, int64_t K) { return K / block_values(wtype) * block_bytes(wtype); }
inline int64_t padded_row_bytes(int wtype, int64_t K) { return (row_bytes(wtype, K) + 15) / 16 * 16; }
// The used experts' rows of W, padded_row_bytes apart.
cudaError_t launch_pad(const Product& p, const Batch& b, void* to, cudaStream_t stream);
// The product with F32 weights, by plain threads.
cudaError_t launch_simt(const Product& p, const Slots& s, int cap, cudaStream_t stream);
constexpr int kSimtTile = 64;

// rg_id_few.cu: the forward for a few slots an expert; whether a batch and product can take it.  Of s, the output, the
// weights and `live` (cleared and set here) are used.
bool few_fits(const Batch& b, const Product& p);
int few_rows(int64_t K);  // slots a chunk of one MMA's columns: up to eight, as their rows of X fit
cudaError_t launch_few(const Product& p, const Batch& b, const Slots& s, const DevInfo& dev, cudaStream_t stream);

// rg_mm_id.cu, rg_tc_id.cu: the tensor-core kernel over the tile table.
cudaError_t launch_mm_id(int wtype, const void* W, int64_t experts, int64_t N, int64_t K, const uint16_t* x16,
                         int64_t ld, const Slots& s, int cg, const DevInfo& dev, cudaStream_t stream);
cudaError_t launch_tc_id(int wtype, const void* W, int64_t experts, int64_t N, int64_t K, const uint16_t* x16,
                         int64_t ld, const Slots& s, int cg, const DevInfo& dev, cudaStream_t stream);

}  // namespace id
}  // namespace rg
