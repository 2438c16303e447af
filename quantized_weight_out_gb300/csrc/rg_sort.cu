// rg_sort.cu - the sort of indices by one block or a cluster (rg_sort.cuh) as
// a launch of its own.
#include "rg_sort.cuh"

namespace rg {
namespace id {

namespace {

__global__ void __launch_bounds__(SORT_THREADS, 1) sort_kernel(Sort p, int* status) {
  extern __shared__ int hist[];
  pdl_wait();
  pdl_launch_dependents();
  if (sort_block<false>(p, hist)) report_index(status);
}

}  // namespace

size_t sort_workspace(int64_t n, int64_t groups) {
  Sort p{};
  sort_plan(groups, false, &p);
  return static_cast<size_t>(p.passes > 2 ? 2 : p.passes - 1) * static_cast<size_t>(up256(n * 8));
}

cudaError_t launch_sort(const int32_t* ids, int64_t n, int64_t groups, int32_t* start, int32_t* order,
                        int32_t* sorted, void* ws, const DevInfo& dev, cudaStream_t stream, bool after_prev) {
  Sort p{};
  sort_plan(groups, start != nullptr, &p);
  p.ids = ids;
  p.buf[0] = static_cast<uint2*>(ws);
  p.buf[1] = reinterpret_cast<uint2*>(static_cast<char*>(ws) + up256(n * 8));
  p.order = order;
  p.sorted = sorted;
  p.start = start;
  p.n = n;
  p.groups = static_cast<int>(groups);
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(sort_kernel), kSortMostSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // more than two steps a warp: eight blocks, more than two with these: sixteen where the GPU
  // holds such a cluster (65536 slots: the walk and the scattered stores 16 us with eight); few
  // ids: fewer warps
  int blocks = n > 64 * SORT_MAX_WARPS ? 8 : 1;
  const int threads = n <= 512 ? 256 : SORT_THREADS;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(sort_smem(p.bins, threads / 32));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = after_prev ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (n > 8 * 64 * SORT_MAX_WARPS) {
    static std::atomic<int> sixteen[64];  // per device: 1 + whether a cluster of sixteen may be resident
    const int yes = resident(sixteen[dev.device & 63], 1, [&](int* ok) {
      cfg.gridDim = dim3(SORT_MAX_BLOCKS);
      cfg.dynamicSmemBytes = kSortMostSmem;
      attr[0].val.clusterDim.x = SORT_MAX_BLOCKS;
      cudaError_t r = cudaFuncSetAttribute(reinterpret_cast<const void*>(sort_kernel),
                                           cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      int clusters = 0;
      if (r == cudaSuccess) r = cudaOccupancyMaxActiveClusters(&clusters, sort_kernel, &cfg);
      *ok = clusters > 0 ? 2 : 1;
      return r;
    });
    if (yes == 2) blocks = SORT_MAX_BLOCKS;
    cfg.dynamicSmemBytes = static_cast<size_t>(sort_smem(p.bins, threads / 32));
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
  }
  return counted(cudaLaunchKernelEx(&cfg, sort_kernel, p, dev.status));
}

}  // namespace id
}  // namespace rg
