// rg_mm_id.cu - the forward by slot on the tensor cores (a translation unit of
// its own, as rg_mm.cu).
#include "rg_tc_id.cuh"

namespace rg {
namespace id {

cudaError_t launch_mm_id(int wtype, const void* W, int64_t experts, int64_t N, int64_t K, const uint16_t* x16,
                         int64_t ld, const Slots& s, int cg, const DevInfo& dev, cudaStream_t stream) {
  return launch_grp<true>(wtype, W, experts, N, K, x16, ld, s, cg, dev, stream);
}

}  // namespace id
}  // namespace rg
