// rg_id_api.cu - the C ABI of the indexed calls: argument checks and
// workspaces.
#include <algorithm>

#include "rg_id_launch.h"
#include "rg_internal.cuh"

using namespace rg;

namespace {

constexpr int64_t kMaxDim = 2147483647;
// Places inside a row are 32-bit in the kernels, with room for a tile past the end.
constexpr int64_t kMaxWidth = int64_t{1} << 30;
// Columns of the widest launches (65535 blocks along a row).
constexpr int64_t kMaxBackWidth = int64_t{65535} * 1024, kMaxSimtWidth = int64_t{65535} * id::kSimtTile;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_act(int t) { return t == RG_F32 || t == RG_F16 || t == RG_BF16; }
bool finite(float x) { return x - x == 0.0f; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? RG_OK : RG_ERR_CUDA; }

// Rows of `width` values of an activation type, `row` apart: 16-byte aligned.
int check_rows(const void* p, int64_t row, int64_t width, int atype) {
  if (!p || row < width) return RG_ERR_ARG;
  if (!aligned(p, 16) || row % (atype == RG_F32 ? 4 : 8)) return RG_ERR_ALIGN;
  return RG_OK;
}

// A weight of rows of K values (and how many rows): types, sizes and shapes.
int check_weight(int wtype, int64_t N, int64_t K) {
  if (!valid_wtype(wtype)) return RG_ERR_TYPE;
  if (N < 0 || K < 0 || N > kMaxDim || K > kMaxWidth) return RG_ERR_ARG;
  return K % (is_quant(wtype) ? 256 : 8) ? RG_ERR_SHAPE : RG_OK;
}

// Memory from the library's pool for one call, or the caller's.
struct Work {
  void* p = nullptr;
  bool own = false;
  cudaStream_t stream = nullptr;
  int take(size_t need, void* ws, size_t ws_bytes, bool own_ws, const DevInfo& dev, cudaStream_t s) {
    stream = s;
    if (!own_ws) {
      if (need && (!ws || ws_bytes < need)) return RG_ERR_ARG;
      if (!aligned(ws, 256)) return RG_ERR_ALIGN;
      p = ws;
      return RG_OK;
    }
    if (!need) return RG_OK;
    cudaMemPool_t pool{};
    const int st = pool_for(dev.device, &pool);
    if (st != RG_OK) return st;
    if (cudaMallocFromPoolAsync(&p, need, pool, s) != cudaSuccess) return RG_ERR_CUDA;
    own = true;
    return RG_OK;
  }
  int done(cudaError_t e) {
    if (own) {
      const cudaError_t f = cudaFreeAsync(p, stream);
      if (e == cudaSuccess) e = f;
    }
    return from_cuda(e);
  }
};

// --- products by slot ---

int check_batch(const rg_id_batch* x, id::Batch* b) {
  if (!x) return RG_ERR_ARG;
  if (x->experts < 0 || x->per_token < 1 || x->slots < 0 || x->slots > kMaxDim) return RG_ERR_ARG;
  if (x->experts > id::kMaxExperts || x->slots % x->per_token) return RG_ERR_SHAPE;
  b->experts = x->experts;
  b->per_token = x->per_token;
  b->slots = static_cast<int>(x->slots);
  b->start = x->start;
  b->order = x->order;
  return RG_OK;
}

struct Plan {
  bool simt, few;
  bool padded;    // W's rows are copied first, to multiples of 16 bytes
  int cg, bt, cap;
  bool joined;    // rows of `out` are the tokens'
  bool bf16;
  size_t tiles, count, x16, unscale, live, rows, w, total;  // offsets, and the bytes of all
};

// The most slots with which the streaming kernel runs. It decodes W anew for each
// chunk of an expert's slots (`rows`, at most 8, fewer where rows of X are long),
// a tile of 128 slots decodes once: so the limit, in eighths of a slot an expert
// on average, falls where the decoding costs it most, and with the chunks that an
// expert's slots make. us of tiles / streaming, a batch of random routes to 2 and
// 4 experts a token; [8a] 8 experts of 14336 x 4096 (rows 8), [8b] 4096 x 14336
// (rows 3), [8c] 4096 x 8192 (rows 5), [32] 4096 x 4096, [64] 2048 x 2048, [128] 1536
// x 2048; at the limit, then above it:
//   Q4_K 5 slots an expert: [8a] 150 / 101, 150 / 99 [64] 94 / 66, 95 / 64; [8b] 3: 168 / 148, 168 / 143,
//     4: 168 / 176, 168 / 173; 6: [64] 94 / 98, 96 / 96, [32] 174 / 170, 8: 174 / 195 (but [8a] 8: 152 / 140)
//   Q8_0 [8b] 3: 172 / 157, 4: 172 / 194; 6: [64] 97 / 97, 8: 96 / 105; Q4_0 as Q4_K
//   MXFP4 5: [8a] 174 / 166, [64] 110 / 93, [32] 202 / 216, 202 / 209; [8b] 2: 195 / 194, 196 / 166, 3: 196 / 236;
//     [8c] 3: 117 / 127, 118 / 112, 4: 117 / 134; 6: [8a] 174 / 188, [64] 110 / 125; Q4_1, Q2_K alike
//   Q6_K 8: [8a] 236 / 160, [64] 144 / 117, [32] 275 / 213; [8b] 3: 265 / 225, 5: 265 / 269; [8c] 5: 156 / 147,
//     6: 156 / 162; Q3_K 8: [8a] 262 / 204, [32] 305 / 279; [8b] 3: 297 / 259, 4: 297 / 303
//     (their tiles take two scales for 32 values)
//   Q5_0 2: [8a] 141 / 131, [64] 92 / 96, [32] 191 / 181; [8b] 1: 182 / 141, 2: 183 / 206; 3: [8a] 167 / 170
//   Q5_1 1: [8a] 179 / 125, [64] 78 / 64, [32] 140 / 140; 2: [8a] 140 / 158, [32] 189 / 217, [128] 133 / 117
//   Q5_K 1: [8a] 266 / 125, [64] 80 / 74, [32] 144 / 149, [128] 108 / 108; 2: [8a] 144 / 152, [64] 94 / 107
//   BF16 (F16 alike), experts of 64 MB and more: 1: [8a] 174 / 101, [8c] 95 / 91, but [8b] 158 / 255 (1/2: 122 /
//     122); 2: [8a] 129 / 155.  Of 32 MB: 1/2: [32] 87 / 77, 1: 131 / 176.  Smaller: 1/16: [128] 23 / 20,
//     1/8: 35 / 30, [64] 24 / 25; 1/2: [64] 47 / 57, 1: 69 / 85 (but [128] 93 / 85)
//   NVFP4, slots in all: 2: [8a] 96 / 80, [8b] 99 / 98, [64] 22 / 12; 4: [8a] 147 / 152, [64] 23 / 19; 8: [64] 31 /
//     32, [32] 93 / 105; 5 an expert: [8a] 170 / 316 (a nibble's E2M1 value and its scale through F32 and back)
// Up to four slots in all the launch counts, whatever the rest: [64] BF16 20 / 15, Q5_K 22 / 15.
int64_t few_slots_limit(int wtype, int64_t experts, int64_t expert_bytes, int rows) {
  int64_t eighths;
  switch (wtype) {
    case RG_NVFP4: return 2;
    case RG_F16:
    case RG_BF16: eighths = expert_bytes < (16 << 20) ? 1 : expert_bytes < (64 << 20) || rows < 5 ? 4 : 8; break;
    case RG_Q5_K: eighths = 8; break;
    case RG_Q5_1: eighths = std::min(8, 4 * rows); break;
    case RG_Q5_0: eighths = std::min(16, 4 * rows); break;
    case RG_Q6_K:
    case RG_Q3_K: eighths = 8 * rows; break;
    case RG_MXFP4:
    case RG_Q4_1:
    case RG_Q2_K: eighths = std::min(40, 16 * rows / 3); break;
    default: eighths = std::min(40, 8 * rows); break;
  }
  return std::max<int64_t>(4, experts * eighths / 8);
}

// Slots an expert on average from which a tile is a pair of blocks' (256 slots,
// each decoding half of W's rows). A half-empty pair costs more than a single
// block; a group in two single tiles decodes W twice. Single / pair, us, 32
// experts of 2048 x 2048: 96 slots Q4_K 71 / 75, BF16 79 / 80, MXFP4 84 / 85; 128
// slots 86 / 78, 88 / 81, 100 / 90; 256 slots 140 / 98, 115 / 100, 161 / 118.
constexpr int64_t kPairSlots = 128;

Plan plan(const id::Product& p, const id::Batch& b) {
  Plan r{};
  r.simt = p.wtype == RG_F32;
  r.padded = !r.simt && id::padded_row_bytes(p.wtype, p.K) != id::row_bytes(p.wtype, p.K);
  // a few slots an expert: W's rows streamed once; else tiles of 128 or 256 slots
  r.few = !r.simt && id::few_fits(b, p) &&
          b.slots <= few_slots_limit(p.wtype, b.experts, p.N * id::row_bytes(p.wtype, p.K), id::few_rows(p.K));
  r.cg = b.slots >= kPairSlots * b.experts ? 2 : 1;
  r.bt = r.simt ? id::kSimtTile : 128 * r.cg;
  r.cap = static_cast<int>(id::max_tiles(b.slots, b.experts, r.bt));
  r.joined = p.out_tokens;
  r.bf16 = p.wtype == RG_BF16;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = at;
    at += static_cast<size_t>(id::up256(bytes));
    return o;
  };
  const int64_t slots = b.slots;
  r.tiles = take(r.few ? 0 : static_cast<int64_t>(sizeof(id::Tile)) * r.cap);
  r.count = take(r.few ? 0 : 4);
  r.x16 = take(r.simt || r.few ? 0 : slots * p.wide() * 2);
  r.unscale = take(r.simt || r.few || r.bf16 ? 0 : slots * 4);
  r.live = take(r.joined ? slots : 0);
  r.rows = take(r.joined ? slots * p.out_w() * 4 : 0);
  r.w = take(r.padded ? b.experts * p.N * id::padded_row_bytes(p.wtype, p.K) : 0);
  r.total = at;
  return r;
}

cudaError_t launch(id::Product p, const id::Batch& b, const Plan& r, void* ws, const DevInfo& dev,
                   cudaStream_t stream) {
  char* base = static_cast<char*>(ws);
  id::Tile* tiles = reinterpret_cast<id::Tile*>(base + r.tiles);
  int* count = reinterpret_cast<int*>(base + r.count);
  uint16_t* x16 = r.simt ? nullptr : reinterpret_cast<uint16_t*>(base + r.x16);
  float* unscale = r.simt || r.bf16 ? nullptr : reinterpret_cast<float*>(base + r.unscale);
  uint8_t* live = r.joined ? reinterpret_cast<uint8_t*>(base + r.live) : nullptr;
  float* rows = reinterpret_cast<float*>(base + r.rows);
  id::Slots s{};
  s.tiles = tiles;
  s.n_tiles = count;
  s.order = b.order;
  s.slots = b.slots;
  s.per_token = b.per_token;
  s.unscale = unscale;
  s.weights = r.joined ? nullptr : p.weights;
  s.out = r.joined ? rows : p.out;
  s.out_row = r.joined ? p.out_w() : p.out_row;
  s.otype = r.joined ? RG_F32 : p.atype;
  s.beta = r.joined ? 0.0f : p.beta;
  s.live = live;
  cudaError_t e = cudaSuccess;
  if (r.padded) {
    e = id::launch_pad(p, b, base + r.w, stream);
    if (e != cudaSuccess) return e;
    p.W = base + r.w;
  }
  if (r.few) {
    e = id::launch_few(p, b, s, dev, stream);
    if (e == cudaSuccess && r.joined) e = id::launch_join(rows, p.out_w(), live, b, p, dev, stream);
    return e;
  }
  e = id::launch_gather(b, r.bt, tiles, count, r.cap, p, r.bf16, x16, p.wide(), unscale, live, dev, stream);
  if (e != cudaSuccess) return e;
  if (r.simt)
    e = id::launch_simt(p, s, r.cap, stream);
  else
    e = (p.fwd ? id::launch_mm_id : id::launch_tc_id)(p.wtype, p.W, b.experts, p.N, p.K, x16, p.wide(), s, r.cg, dev,
                                                      stream);
  if (e == cudaSuccess && r.joined) e = id::launch_join(rows, p.out_w(), live, b, p, dev, stream);
  return e;
}

// Everything but the pointers, as the workspace query has it too.
int check_shape(bool fwd, int wtype, int64_t N, int64_t K, const rg_id_batch* batch, int out_of, id::Batch* b,
                id::Product* p) {
  int st = check_batch(batch, b);
  if (st != RG_OK || (st = check_weight(wtype, N, K)) != RG_OK) return st;
  if (N % 8) return RG_ERR_SHAPE;
  if (N > kMaxWidth) return RG_ERR_ARG;
  if (out_of != RG_ROWS_SLOT && out_of != RG_ROWS_TOKEN) return RG_ERR_ARG;
  p->fwd = fwd;
  p->wtype = wtype;
  p->N = N;
  p->K = K;
  p->out_tokens = out_of == RG_ROWS_TOKEN;
  // (a stack of 2^46 bytes lies in no device's memory; its copy's size stays within 64 bits)
  if (K > 0 && b->experts * N > (int64_t{1} << 46) / id::padded_row_bytes(wtype, K)) return RG_ERR_ARG;
  return wtype == RG_F32 && p->out_w() > kMaxSimtWidth ? RG_ERR_ARG : RG_OK;
}

int product(bool fwd, int wtype, const void* W, int64_t N, int64_t K, const rg_id_batch* batch, int atype,
            const void* in, int64_t in_row, int in_of, void* out, int64_t out_row, int out_of, const float* weights,
            float beta, void* ws, size_t ws_bytes, bool own_ws, cudaStream_t stream) {
  id::Batch b;
  id::Product p{};
  int st = check_shape(fwd, wtype, N, K, batch, out_of, &b, &p);
  if (st != RG_OK) return st;
  if (!valid_act(atype)) return RG_ERR_TYPE;
  if (in_of != RG_ROWS_SLOT && in_of != RG_ROWS_TOKEN) return RG_ERR_ARG;
  if (b.slots == 0 || p.out_w() == 0) return RG_OK;
  // (no contraction, or no experts: nothing to multiply with; the rows would be beta times themselves)
  if (p.wide() == 0 || b.experts == 0) return RG_ERR_SHAPE;
  if (!W || !b.start || !b.order) return RG_ERR_ARG;
  if (!aligned(W, 16) || !aligned(b.start, 4) || !aligned(b.order, 4) || !aligned(weights, 4)) return RG_ERR_ALIGN;
  if ((st = check_rows(in, in_row, p.wide(), atype)) != RG_OK) return st;
  if ((st = check_rows(out, out_row, p.out_w(), atype)) != RG_OK) return st;
  DevInfo* dev = nullptr;
  if ((st = current_dev(&dev)) != RG_OK) return st;
  p.W = W;
  p.atype = atype;
  p.in = in;
  p.in_row = in_row;
  p.in_tokens = in_of == RG_ROWS_TOKEN;
  p.out = out;
  p.out_row = out_row;
  p.weights = weights;
  p.beta = beta;
  const Plan r = plan(p, b);
  Work w;
  if ((st = w.take(r.total, ws, ws_bytes, own_ws, *dev, stream)) != RG_OK) return st;
  return w.done(launch(p, b, r, w.p, *dev, stream));
}

size_t product_bytes(bool fwd, int wtype, int64_t N, int64_t K, const rg_id_batch* batch, int out_of) {
  id::Batch b;
  id::Product p{};
  if (check_shape(fwd, wtype, N, K, batch, out_of, &b, &p) != RG_OK || b.slots == 0 || N == 0 || K == 0 ||
      b.experts == 0)
    return 0;
  return plan(p, b).total;
}

int check_route(const float* logits, int64_t l_row, int64_t T, int experts, int top, int mode, float scale) {
  if (mode != RG_ROUTE_TOP && mode != RG_ROUTE_ALL) return RG_ERR_TYPE;
  if (T < 0 || T > kMaxDim || experts < 1 || top < 1 || T * top > kMaxDim || !finite(scale)) return RG_ERR_ARG;
  if (experts > id::kMaxExperts || top > id::kMaxChosen || top > experts) return RG_ERR_SHAPE;
  if (T == 0) return RG_OK;
  if (!logits || l_row < experts) return RG_ERR_ARG;
  return aligned(logits, 4) ? RG_OK : RG_ERR_ALIGN;
}

}  // namespace

extern "C" {

int rg_get_rows(int wtype, const void* W, int64_t N, int64_t K, const int32_t* ids, int64_t n, float scale, int atype,
                void* out, int64_t out_row, void* stream) {
  int st = check_weight(wtype, N, K);
  if (st != RG_OK) return st;
  if (!valid_act(atype)) return RG_ERR_TYPE;
  if (n < 0 || n > kMaxDim) return RG_ERR_ARG;
  if (n == 0 || K == 0) return RG_OK;
  if ((N > 0 && !W) || !ids) return RG_ERR_ARG;
  if (!aligned(W, 16) || !aligned(ids, 4)) return RG_ERR_ALIGN;
  if ((st = check_rows(out, out_row, K, atype)) != RG_OK) return st;
  DevInfo* dev = nullptr;
  if ((st = current_dev(&dev)) != RG_OK) return st;
  return from_cuda(id::launch_get_rows(wtype, W, N, K, ids, n, scale, atype, out, out_row, *dev,
                                       static_cast<cudaStream_t>(stream)));
}

size_t rg_get_rows_back_workspace_bytes(int64_t n, int64_t N, int64_t K) {
  if (n < 1 || N < 1 || K < 1 || n > kMaxDim || N > kMaxDim || K > kMaxBackWidth || K % 8) return 0;
  return id::rows_back_workspace(n, N, K);
}

}  // extern "C"

namespace {

int rows_back(int atype, const void* dY, int64_t dy_row, const int32_t* ids, int64_t n, float scale, float* G,
              int64_t g_row, int64_t N, int64_t K, float beta, void* ws, size_t ws_bytes, bool own_ws,
              cudaStream_t stream) {
  if (!valid_act(atype)) return RG_ERR_TYPE;
  if (n < 0 || N < 0 || K < 0 || n > kMaxDim || N > kMaxDim || K > kMaxBackWidth) return RG_ERR_ARG;
  if (K % 8) return RG_ERR_SHAPE;
  if (N == 0 || K == 0) return RG_OK;
  int st = check_rows(G, g_row, K, RG_F32);
  if (st != RG_OK) return st;
  if (n > 0) {
    if (!ids) return RG_ERR_ARG;
    if (!aligned(ids, 4)) return RG_ERR_ALIGN;
    if ((st = check_rows(dY, dy_row, K, atype)) != RG_OK) return st;
  }
  DevInfo* dev = nullptr;
  if ((st = current_dev(&dev)) != RG_OK) return st;
  if (n == 0) return beta == 1.0f ? RG_OK : from_cuda(launch_scale(G, N, K, g_row, beta, *dev, stream));
  Work w;
  if ((st = w.take(id::rows_back_workspace(n, N, K), ws, ws_bytes, own_ws, *dev, stream)) != RG_OK) return st;
  return w.done(id::launch_rows_back(atype, dY, dy_row, ids, n, scale, G, g_row, N, K, beta, w.p, *dev, stream));
}

}  // namespace

extern "C" {

int rg_get_rows_back(int atype, const void* dY, int64_t dy_row, const int32_t* ids, int64_t n, float scale, float* G,
                     int64_t g_row, int64_t N, int64_t K, float beta, void* stream) {
  return rows_back(atype, dY, dy_row, ids, n, scale, G, g_row, N, K, beta, nullptr, 0, true,
                   static_cast<cudaStream_t>(stream));
}

int rg_get_rows_back_ws(int atype, const void* dY, int64_t dy_row, const int32_t* ids, int64_t n, float scale, float* G,
                        int64_t g_row, int64_t N, int64_t K, float beta, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return rows_back(atype, dY, dy_row, ids, n, scale, G, g_row, N, K, beta, workspace, workspace_bytes, false,
                   static_cast<cudaStream_t>(stream));
}

int rg_group(const int32_t* ids, int64_t n, int groups, int32_t* start, int32_t* order, void* stream) {
  if (n < 0 || n > kMaxDim || groups < 1) return RG_ERR_ARG;
  if (groups > id::kMaxExperts) return RG_ERR_SHAPE;
  if (!start || (n > 0 && (!ids || !order))) return RG_ERR_ARG;
  if (!aligned(ids, 4) || !aligned(start, 4) || !aligned(order, 4)) return RG_ERR_ALIGN;
  DevInfo* dev = nullptr;
  const int st = current_dev(&dev);
  if (st != RG_OK) return st;
  return from_cuda(
      id::launch_sort(ids, n, groups, start, order, nullptr, nullptr, *dev, static_cast<cudaStream_t>(stream)));
}

int rg_route(const float* logits, int64_t l_row, int64_t T, int experts, int top, int mode, float scale, int32_t* ids,
             float* weights, int32_t* start, int32_t* order, void* stream) {
  int st = check_route(logits, l_row, T, experts, top, mode, scale);
  if (st != RG_OK) return st;
  if (T > 0 && (!ids || !weights || !start != !order)) return RG_ERR_ARG;
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(start, 4) || !aligned(order, 4)) return RG_ERR_ALIGN;
  if (T == 0 && !start) return RG_OK;
  DevInfo* dev = nullptr;
  if ((st = current_dev(&dev)) != RG_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) return from_cuda(id::launch_sort(nullptr, 0, experts, start, order, nullptr, nullptr, *dev, s));
  return from_cuda(id::launch_route(logits, l_row, T, experts, top, mode, scale, ids, weights, start, order, *dev, s));
}

int rg_route_back(const float* logits, int64_t l_row, int64_t T, int experts, int top, int mode, float scale,
                  const int32_t* ids, const float* dweights, float* dlogits, int64_t dl_row, void* stream) {
  int st = check_route(logits, l_row, T, experts, top, mode, scale);
  if (st != RG_OK || T == 0) return st;
  if (!ids || !dweights || !dlogits || dl_row < experts) return RG_ERR_ARG;
  if (!aligned(ids, 4) || !aligned(dweights, 4) || !aligned(dlogits, 4)) return RG_ERR_ALIGN;
  DevInfo* dev = nullptr;
  if ((st = current_dev(&dev)) != RG_OK) return st;
  return from_cuda(id::launch_route_back(logits, l_row, T, experts, top, mode, scale, ids, dweights, dlogits, dl_row,
                                         *dev, static_cast<cudaStream_t>(stream)));
}

int rg_mul_mat_id(int wtype, const void* W, int64_t N, int64_t K, const rg_id_batch* batch, int atype, const void* X,
                  int64_t x_row, int x_of, void* Y, int64_t y_row, int y_of, const float* weights, float beta,
                  void* stream) {
  return product(true, wtype, W, N, K, batch, atype, X, x_row, x_of, Y, y_row, y_of, weights, beta, nullptr, 0, true,
                 static_cast<cudaStream_t>(stream));
}

int rg_mul_mat_id_ws(int wtype, const void* W, int64_t N, int64_t K, const rg_id_batch* batch, int atype, const void* X,
                     int64_t x_row, int x_of, void* Y, int64_t y_row, int y_of, const float* weights, float beta,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return product(true, wtype, W, N, K, batch, atype, X, x_row, x_of, Y, y_row, y_of, weights, beta, workspace,
                 workspace_bytes, false, static_cast<cudaStream_t>(stream));
}

size_t rg_mul_mat_id_workspace_bytes(int wtype, int64_t N, int64_t K, const rg_id_batch* batch, int y_of) {
  return product_bytes(true, wtype, N, K, batch, y_of);
}

int rg_out_prod_id(int wtype, const void* W, int64_t N, int64_t K, const rg_id_batch* batch, int atype, const void* dY,
                   int64_t dy_row, int dy_of, void* dX, int64_t dx_row, int dx_of, const float* weights, float beta,
                   void* stream) {
  return product(false, wtype, W, N, K, batch, atype, dY, dy_row, dy_of, dX, dx_row, dx_of, weights, beta, nullptr, 0,
                 true, static_cast<cudaStream_t>(stream));
}

int rg_out_prod_id_ws(int wtype, const void* W, int64_t N, int64_t K, const rg_id_batch* batch, int atype,
                      const void* dY, int64_t dy_row, int dy_of, void* dX, int64_t dx_row, int dx_of,
                      const float* weights, float beta, void* workspace, size_t workspace_bytes, void* stream) {
  return product(false, wtype, W, N, K, batch, atype, dY, dy_row, dy_of, dX, dx_row, dx_of, weights, beta, workspace,
                 workspace_bytes, false, static_cast<cudaStream_t>(stream));
}

size_t rg_out_prod_id_workspace_bytes(int wtype, int64_t N, int64_t K, const rg_id_batch* batch, int dx_of) {
  return product_bytes(false, wtype, N, K, batch, dx_of);
}

}  // extern "C"
