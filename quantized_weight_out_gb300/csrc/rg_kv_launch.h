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
};
size_t attend_workspace(int type, const Cache& c, const Batch& b, int heads, const DevInfo& dev);
cudaError_t launch_attend(int type, const Cache& c, const Batch& b, const Attend& a, void* workspace,
                          const DevInfo& dev, cudaStream_t stream);

}  // namespace kv
}  // namespace rg
