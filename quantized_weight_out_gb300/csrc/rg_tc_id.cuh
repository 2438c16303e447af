// rg_tc_id.cuh - launch of the tensor-core kernel over a table of tiles of
// slots (its GRP instances), shared by rg_mm_id.cu and rg_tc_id.cu.
#pragma once

#include "rg_tc_kernel.cuh"

namespace rg {
namespace id {

template <int WT, int CG, int BT, bool FWD>
static cudaError_t launch_grp_t(const CUtensorMap& mw, const CUtensorMap& mx, const CUtensorMap& ml,
                                const CUtensorMap& mq, int K, int n_kunits, int band, int n_chunks, const Slots& s,
                                const DevInfo& dev, cudaStream_t stream) {
  using C = tc::Cfg<WT, CG, BT, FWD, true>;
  auto kern = tc::out_prod_tc_kernel<WT, CG, BT, false, false, FWD, true>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  WaitCtl ctl{dev.status, dev.wait_limit_ns};
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(tc::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(static_cast<unsigned>(CG * (dev.num_sms / CG)), 1, 1);
  static std::atomic<int> max_clusters[64];
  const int units = resident(max_clusters[dev.device & 63], dev.num_sms / CG, [&](int* n) {
    return cudaOccupancyMaxActiveClusters(n, kern, &cfg);
  });
  cfg.gridDim = dim3(static_cast<unsigned>(CG * std::min(units, dev.num_sms / CG)), 1, 1);
  return counted(cudaLaunchKernelEx(&cfg, kern, mw, mx, ml, mw, mw, mq, 1 << 30, static_cast<float*>(nullptr),
                                    int64_t{0}, 0.0f, 0, K, n_kunits, 1, band, n_chunks, 1,
                                    static_cast<float*>(nullptr), ctl, tc::GrpArg<true>{s}));
}

// W: `experts` matrices of N rows of K values, padded_row_bytes apart; x16: the
// slots' 16-bit copy in sorted order.
template <bool FWD>
static cudaError_t launch_grp(int wtype, const void* W, int64_t experts, int64_t N, int64_t K, const uint16_t* x16,
                              int64_t ld, const Slots& s, int cg, const DevInfo& dev, cudaStream_t stream) {
  const int64_t n_contr = FWD ? K : N, k_out = FWD ? N : K;
  TcPlan p{};
  p.cg = cg;
  p.bt = 128 * cg;
  p.n_kunits = static_cast<int>((k_out + 128 * cg - 1) / (128 * cg));
  p.n_chunks = static_cast<int>((n_contr + tc::BC - 1) / tc::BC);
  p.band = tc_band(wtype, n_contr, p);
  CUtensorMap mw, ml, mq, mx;
  const uint32_t rows = FWD ? 2 * tc::BC : tc::BC;
  const uint64_t n = static_cast<uint64_t>(N), e = static_cast<uint64_t>(experts);
  CUresult r;
  if (is_quant(wtype)) {
    const uint64_t rb = static_cast<uint64_t>(padded_row_bytes(wtype, K));
    auto words = [&](CUtensorMap* m, uint32_t w) {
      return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, W, rb / 4, n, rb, w, rows, CU_TENSOR_MAP_SWIZZLE_NONE, e,
                          n * rb);
    };
    const uint32_t box = static_cast<uint32_t>(with_wtype(wtype, 0, [](auto wt) {
                           return FWD ? tc::p_fwd_bytes<decltype(wt)::value, true>()
                                      : tc::p_row_bytes<decltype(wt)::value>();
                         })) / 4;
    // (the forward's Q4_K and Q6_K windows are split, as in launch_tc_impl)
    const bool q4k = FWD && wtype == RG_Q4_K, q6k = FWD && wtype == RG_Q6_K;
    r = words(&mw, q4k ? 4 : q6k ? tc::Q6F_A / 4 : box);
    ml = mq = mw;
    if (r == CUDA_SUCCESS && (q4k || q6k)) r = words(&ml, q4k ? 8 : tc::Q6F_H / 4);
    if (r == CUDA_SUCCESS && q6k) r = words(&mq, tc::Q6F_S / 4);
  } else {
    r = encode_tiled(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT16, W, static_cast<uint64_t>(K), n,
                     static_cast<uint64_t>(K) * 2, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B, e,
                     n * static_cast<uint64_t>(K) * 2);
    ml = mq = mw;
  }
  if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  r = encode_tiled(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT16, x16, static_cast<uint64_t>(n_contr),
                   static_cast<uint64_t>(s.slots), static_cast<uint64_t>(ld) * 2, tc::BC, tc::B_ROWS,
                   CU_TENSOR_MAP_SWIZZLE_128B);
  if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  const int k = static_cast<int>(k_out);
  return with_wtype(wtype, cudaErrorInvalidValue, [&](auto wt) {
    constexpr int WT = decltype(wt)::value;
    if constexpr (WT == RG_F32) {
      return cudaErrorInvalidValue;  // (F32 weights take the plain threads' route)
    } else if (cg == 2) {
      return launch_grp_t<WT, 2, 256, FWD>(mw, mx, ml, mq, k, p.n_kunits, p.band, p.n_chunks, s, dev, stream);
    } else {
      return launch_grp_t<WT, 1, 128, FWD>(mw, mx, ml, mq, k, p.n_kunits, p.band, p.n_chunks, s, dev, stream);
    }
  });
}

}  // namespace id
}  // namespace rg
