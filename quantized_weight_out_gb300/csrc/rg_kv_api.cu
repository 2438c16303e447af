// rg_kv_api.cu - the C ABI of the paged key/value cache: argument checks and
// workspaces.
#include "rg_kv_launch.h"

using namespace rg;

namespace {

constexpr int64_t kMaxDim = 2147483647;
// Positions, and rows of a sequence, are 32-bit in the kernels, with room for a tile past the end.
constexpr int64_t kMaxLen = int64_t{1} << 30;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The cache and batch descriptions, checked and turned into what kernels take.
int check(const rg_kv_cache* cache, const rg_kv_batch* batch, int atype, kv::Cache* c, kv::Batch* b, bool* empty) {
  *empty = false;
  if (!cache || !batch) return RG_ERR_ARG;
  if (!kv::valid_type(cache->type)) return RG_ERR_TYPE;
  if (atype != RG_F32 && atype != RG_F16 && atype != RG_BF16) return RG_ERR_TYPE;
  if (cache->kv_heads < 1 || cache->kv_heads > 4096 || cache->page_tokens < 1 || cache->pages < 0 ||
      cache->pages > kMaxDim)
    return RG_ERR_ARG;
  if ((cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 256) || cache->page_tokens % 16 ||
      cache->page_tokens > 4096)
    return RG_ERR_SHAPE;
  if (batch->seqs < 0 || batch->max_pages < 0 || batch->max_new < 0 || batch->reserved != 0 || batch->tokens < 0 ||
      batch->tokens > kMaxDim || static_cast<int64_t>(batch->max_pages) * cache->page_tokens > kMaxLen)
    return RG_ERR_ARG;
  if (batch->seqs == 0 || batch->tokens == 0 || batch->max_new == 0) {
    *empty = true;
    return RG_OK;
  }
  if (!batch->new_start || !batch->kv_len || (batch->max_pages > 0 && !batch->page_table) ||
      (cache->pages > 0 && !cache->data))
    return RG_ERR_ARG;
  if (!aligned(cache->data, 16) || !aligned(batch->new_start, 4) || !aligned(batch->kv_len, 4) ||
      !aligned(batch->page_table, 4))
    return RG_ERR_ALIGN;
  c->data = static_cast<uint8_t*>(cache->data);
  c->pages = static_cast<int>(cache->pages);
  c->page_tokens = cache->page_tokens;
  c->kv_heads = cache->kv_heads;
  c->dim = cache->head_dim;
  c->slab_bytes = static_cast<int64_t>(cache->page_tokens) * kv::row_bytes(cache->type, cache->head_dim);
  c->page_bytes = 2 * c->slab_bytes * cache->kv_heads;
  b->new_start = batch->new_start;
  b->kv_len = batch->kv_len;
  b->table = batch->page_table;
  b->seqs = batch->seqs;
  b->max_pages = batch->max_pages;
  b->max_new = static_cast<int>(std::min<int64_t>(batch->max_new, batch->tokens));
  b->tokens = static_cast<int>(batch->tokens);
  return RG_OK;
}

// A packed array of `heads` rows of head_dim values a token: 16-byte aligned
// rows; strides at least a row long.
int check_rows(const void* p, int64_t st, int64_t sh, int heads, int dim, int atype) {
  if (st < 0 || sh < 0) return RG_ERR_ARG;
  const int64_t unit = atype == RG_F32 ? 4 : 8;
  if (!aligned(p, 16) || st % unit || sh % unit) return RG_ERR_ALIGN;
  if (st < dim || (heads > 1 && sh < dim)) return RG_ERR_ARG;
  return RG_OK;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? RG_OK : RG_ERR_CUDA; }

// Sequences of more rows (new tokens x query heads of a kv head) than this run in
// the tile kernel; the others, which would leave most of a tile empty, in the few-row
// kernel.  One sequence over 15,000 tokens, 4 kv heads, us few-row / tile: 32 rows of 128
// dimensions 39 / 44, 64 rows 39 / 45, 64 rows of 256 dimensions 45 / 62; 16 sequences of 8 to
// 36 rows 81 / 195.  Beyond 64 rows the few-row kernel reads the cache a third time.
constexpr int kRowsLimit = 64;

// How a batch is run: the few-row kernel for its short sequences, the tile
// kernel as well when there may be longer ones.
struct Route {
  bool tiles;
  int rows_limit;
  size_t rows_bytes, tiles_bytes;
};
Route route_of(const kv::Cache& c, const kv::Batch& b, int group, const DevInfo& dev) {
  Route r;
  r.tiles = static_cast<int64_t>(b.max_new) * group > kRowsLimit;
  // (one sequence alone: whatever its length turns out to be, one kernel has it; and where
  // one token is more rows than that, none is left for the few-row kernel)
  r.rows_limit = !r.tiles ? 2147483647 : b.seqs == 1 || group > kRowsLimit ? 0 : kRowsLimit;
  kv::Batch few = b;
  if (r.tiles) few.max_new = std::max(1, kRowsLimit / group);
  r.rows_bytes = r.rows_limit ? (kv::rows_workspace(c, few, group, dev) + 255) / 256 * 256 : 0;
  r.tiles_bytes = r.tiles ? kv::tiles_workspace(c, dev) : 0;
  return r;
}

int attend(const rg_kv_cache* cache, const rg_kv_batch* batch, int atype, const void* q, int64_t q_t, int64_t q_h,
           int heads, void* out, int64_t o_t, int64_t o_h, float scale, int window, void* ws, size_t ws_bytes,
           bool own_ws, cudaStream_t stream) {
  kv::Cache c;
  kv::Batch b;
  bool empty;
  int st = check(cache, batch, atype, &c, &b, &empty);
  if (st != RG_OK) return st;
  if (heads < 1 || window < 0) return RG_ERR_ARG;
  if (heads % cache->kv_heads || heads / cache->kv_heads > 1024) return RG_ERR_SHAPE;
  if (!(scale - scale == 0.0f)) return RG_ERR_ARG;  // not finite
  if (empty) return RG_OK;
  if (!q || !out) return RG_ERR_ARG;
  if ((st = check_rows(q, q_t, q_h, heads, c.dim, atype)) != RG_OK) return st;
  if ((st = check_rows(out, o_t, o_h, heads, c.dim, atype)) != RG_OK) return st;
  if (static_cast<int64_t>(b.max_new) * (heads / c.kv_heads) > kMaxLen) return RG_ERR_ARG;
  DevInfo* dev = nullptr;
  if (own_ws || ws) {
    if ((st = current_dev(&dev)) != RG_OK) return st;
  } else {
    return RG_ERR_ARG;
  }
  kv::Attend a;
  a.q = q;
  a.out = out;
  a.q_t = q_t;
  a.q_h = q_h;
  a.o_t = o_t;
  a.o_h = o_h;
  a.heads = heads;
  a.group = heads / c.kv_heads;
  a.atype = atype;
  // a window as long as a sequence can be hides nothing
  a.window = window >= static_cast<int64_t>(b.max_pages) * c.page_tokens ? 0 : window;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const Route r = route_of(c, b, a.group, *dev);
  const size_t need = r.rows_bytes + r.tiles_bytes;
  a.rows_limit = r.rows_limit;
  void* buf = ws;
  if (own_ws) {
    cudaMemPool_t pool{};
    if ((st = pool_for(dev->device, &pool)) != RG_OK) return st;
    if (cudaMallocFromPoolAsync(&buf, need, pool, stream) != cudaSuccess) return RG_ERR_CUDA;
  } else {
    if (ws_bytes < need) return RG_ERR_ARG;
    if (!aligned(ws, 256)) return RG_ERR_ALIGN;
  }
  cudaError_t e = cudaSuccess;
  if (r.tiles)
    e = kv::launch_tiles(cache->type, c, b, a, static_cast<char*>(buf) + r.rows_bytes, *dev, stream);
  if (e == cudaSuccess && a.rows_limit > 0)
    e = kv::launch_rows(cache->type, c, b, a, buf, *dev, stream);
  if (own_ws) {
    const cudaError_t f = cudaFreeAsync(buf, stream);
    if (e == cudaSuccess) e = f;
  }
  return from_cuda(e);
}

}  // namespace

extern "C" {

size_t rg_kv_page_bytes(int type, int head_dim, int kv_heads, int page_tokens) {
  if (!kv::valid_type(type) || (head_dim != 64 && head_dim != 128 && head_dim != 256) || kv_heads < 1 ||
      kv_heads > 4096 || page_tokens < 16 || page_tokens > 4096 || page_tokens % 16)
    return 0;
  return 2 * static_cast<size_t>(kv_heads) * static_cast<size_t>(page_tokens) *
         static_cast<size_t>(kv::row_bytes(type, head_dim));
}

int rg_kv_write(const rg_kv_cache* cache, const rg_kv_batch* batch, int atype, const void* k, int64_t k_t,
                int64_t k_h, const void* v, int64_t v_t, int64_t v_h, void* stream) {
  kv::Cache c;
  kv::Batch b;
  bool empty;
  int st = check(cache, batch, atype, &c, &b, &empty);
  if (st != RG_OK || empty) return st;
  if (!k && !v) return RG_ERR_ARG;
  if (k && (st = check_rows(k, k_t, k_h, c.kv_heads, c.dim, atype)) != RG_OK) return st;
  if (v && (st = check_rows(v, v_t, v_h, c.kv_heads, c.dim, atype)) != RG_OK) return st;
  DevInfo* dev = nullptr;
  if ((st = current_dev(&dev)) != RG_OK) return st;
  return from_cuda(kv::launch_write(cache->type, atype, c, b, k, k_t, k_h, v, v_t, v_h, *dev,
                                    static_cast<cudaStream_t>(stream)));
}

int rg_kv_read(const rg_kv_cache* cache, const rg_kv_batch* batch, int atype, void* k, int64_t k_t, int64_t k_h,
               void* v, int64_t v_t, int64_t v_h, void* stream) {
  kv::Cache c;
  kv::Batch b;
  bool empty;
  int st = check(cache, batch, atype, &c, &b, &empty);
  if (st != RG_OK || empty) return st;
  if (!k && !v) return RG_ERR_ARG;
  if (k && (st = check_rows(k, k_t, k_h, c.kv_heads, c.dim, atype)) != RG_OK) return st;
  if (v && (st = check_rows(v, v_t, v_h, c.kv_heads, c.dim, atype)) != RG_OK) return st;
  DevInfo* dev = nullptr;
  if ((st = current_dev(&dev)) != RG_OK) return st;
  return from_cuda(kv::launch_read(cache->type, atype, c, b, k, k_t, k_h, v, v_t, v_h, *dev,
                                   static_cast<cudaStream_t>(stream)));
}

size_t rg_kv_attend_workspace_bytes(const rg_kv_cache* cache, const rg_kv_batch* batch, int heads) {
  kv::Cache c;
  kv::Batch b;
  bool empty;
  if (check(cache, batch, RG_F32, &c, &b, &empty) != RG_OK || empty || heads < 1 || heads % c.kv_heads ||
      heads / c.kv_heads > 1024 || static_cast<int64_t>(b.max_new) * (heads / c.kv_heads) > kMaxLen)
    return 0;
  DevInfo* dev = nullptr;
  if (current_dev(&dev) != RG_OK) return 0;
  const Route r = route_of(c, b, heads / c.kv_heads, *dev);
  return r.rows_bytes + r.tiles_bytes;
}

int rg_kv_attend(const rg_kv_cache* cache, const rg_kv_batch* batch, int atype, const void* q, int64_t q_t,
                 int64_t q_h, int heads, void* out, int64_t o_t, int64_t o_h, float scale, int window, void* stream) {
  return attend(cache, batch, atype, q, q_t, q_h, heads, out, o_t, o_h, scale, window, nullptr, 0, true,
                static_cast<cudaStream_t>(stream));
}

int rg_kv_attend_ws(const rg_kv_cache* cache, const rg_kv_batch* batch, int atype, const void* q, int64_t q_t,
                    int64_t q_h, int heads, void* out, int64_t o_t, int64_t o_h, float scale, int window,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return attend(cache, batch, atype, q, q_t, q_h, heads, out, o_t, o_h, scale, window, workspace, workspace_bytes,
                false, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
