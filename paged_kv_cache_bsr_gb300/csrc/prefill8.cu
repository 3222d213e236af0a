// prefill8.cu -- the prefill kernel (prefill_kernel.cuh) over the expanded copy of the
// 8-bit cache's pages, for plans with split tiles.
//
// The same CTA as the plain instances, with two differences that pay where tiles are
// split over their keys (few query rows before many keys): the fp32 partial states go
// out through shared memory, whole 128-byte segments a store, and the kernel is a
// programmatic dependent of the expansion, which hides the gap between the two.  Measured
// against the plain instances: 64 rows over 8192 keys 39.2 -> 36.4 us, two short prompts
// 16.1 -> 13.2 us, a 512-row chunk behind 8192 keys 113.7 -> 108.5 us.  Batches without
// splits keep the plain instances (staging costs a ragged causal batch 1.6 %).
#include "prefill_kernel.cuh"

namespace pkv {
namespace {

using namespace prefill_impl;

template <int G, typename T, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    prefill8_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap tq,
                    const __grid_constant__ CUtensorMap tkv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // Launched as a programmatic dependent of the expansion: nothing global is touched
  // before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  prefill_cta<G, T, CAP, false, false, true>(a, tq, tkv, blockIdx.x, smem_raw);
}

template <typename T>
cudaError_t launch_t(const PrefillArgs& a, int G, bool cap, int grid, const CUtensorMap& tq, const CUtensorMap& tkv,
                     cudaStream_t s) {
  void (*kern)(PrefillArgs, CUtensorMap, CUtensorMap) = nullptr;
#define PKV_PF8_CASE(GG)                                                       \
  case GG:                                                                     \
    kern = cap ? prefill8_kernel<GG, T, true> : prefill8_kernel<GG, T, false>; \
    break;
  switch (G) {
    PKV_PF8_CASE(1) PKV_PF8_CASE(2) PKV_PF8_CASE(4) PKV_PF8_CASE(8)
    default: return cudaErrorInvalidValue;
  }
#undef PKV_PF8_CASE
  cudaError_t e = ensure_smem_limit(kern, kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, grid, kThreads, kSmemBytes, s, a, tq, tkv);
}

}  // namespace

cudaError_t launch_prefill8(const PrefillArgs& a, int head_dim, int group, int dtype, bool cap, int grid,
                            int64_t total_q, int64_t num_pages, cudaStream_t stream) {
  if (!prefill_supported(head_dim, group, dtype, a.page_size) || a.page_size < 8 || a.mask) return cudaErrorInvalidValue;
  CUtensorMap tq, tkv;
  cudaError_t e = make_tensor_maps(a, group, dtype, total_q, num_pages, tq, tkv);
  if (e != cudaSuccess) return e;
  return dtype == PKV_BF16 ? launch_t<__nv_bfloat16>(a, group, cap, grid, tq, tkv, stream)
                           : launch_t<__half>(a, group, cap, grid, tq, tkv, stream);
}

}  // namespace pkv
