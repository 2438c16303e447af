// rg_kv_launch.h - host-side launchers of the paged cache's kernels.  All
// enqueue on `stream` and return the launch status; arguments are validated
// by the entry points.
#pragma once

#include "rg_kv.cuh"
#include "rg_launch.h"

namespace rg {
namespace kv {

cudaError_t launch_write(int type, int atype, const Cache& c, const Batch& b, const void* k, int64_t k_t, int64_t k_h,
                         const void* v, int64_t v_t, int64_t v_h, const DevInfo& dev, cudaStream_t stream);
cudaError_t launch_read(int type, int atype, const Cache& c, const Batch& b, void* k, int64_t k_t, int64_t k_h,
                        void* v, int64_t v_t, int64_t v_h, const DevInfo& dev, cudaStream_t stream);

// Attention arguments.
struct Attend {
  const void* q;
  void* out;
  int64_t q_t, q_h, o_t, o_h;  // element strides of tokens and heads
  int heads, group;            // query heads, query heads per kv head
  int atype;
  int window;                  // 0: none
  float scale_log2;            // scale * log2(e)
  int rows_limit;              // sequences of more rows (new tokens x group) are the tile kernel's
};
// Few rows a sequence (rg_kv_rows.cu): those of at most a.rows_limit rows.
size_t rows_workspace(const Cache& c, const Batch& b, int group, const DevInfo& dev);
cudaError_t launch_rows(int type, const Cache& c, const Batch& b, const Attend& a, void* workspace,
                        const DevInfo& dev, cudaStream_t stream);
// Tiles of rows on the 5th-generation tensor cores (rg_kv_tiles.cu): the others.
size_t tiles_workspace(const Cache& c, const DevInfo& dev);
cudaError_t launch_tiles(int type, const Cache& c, const Batch& b, const Attend& a, void* workspace,
                         const DevInfo& dev, cudaStream_t stream);

// Joins the parts of items that several CTAs share (rg_kv_rows.cu).
struct Desc;
cudaError_t launch_join(const Attend& a, const Desc* desc, const float* parts, int bm, int dim, int ctas,
                        cudaStream_t stream);

}  // namespace kv
}  // namespace rg
