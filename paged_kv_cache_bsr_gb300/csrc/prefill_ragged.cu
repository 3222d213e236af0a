// prefill_ragged.cu -- the prefill kernel (prefill_kernel.cuh) over keys and values that
// are not in pages: rows packed request behind request, as a projection leaves them.
//
// The attention is the paged kernel's, with keys taken 64 at a time (see there); what
// differs else is where a 128-key block comes from: one TMA box per 64 columns of a tensor map over the packed rows,
// whose row stride may be any multiple of 16 bytes, so queries, keys and values may be
// views of one projection's output and are read in place.  A box is one copy whatever
// the request's length: 128 rows from its first key on.  Rows past the request's last
// key are the next request's; they are masked in S and zeroed in V before the product,
// so that nothing of one request (a NaN) reaches another.
// With split tiles the instance whose fp32 partial states go out through shared memory
// is launched, without them the plain one, as over the 8-bit cache (prefill8.cu).
#include "prefill_kernel.cuh"

namespace pkv {
namespace {

using namespace prefill_impl;

template <int G, typename T, bool CAP, bool STAGED>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_ragged_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap tq,
                          const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  prefill_cta<G, T, CAP, false, false, STAGED, true>(a, tq, tk, tv, blockIdx.x, smem_raw);
}

template <typename T, bool STAGED>
cudaError_t launch_t(const PrefillArgs& a, int G, bool cap, int grid, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, cudaStream_t s) {
  void (*kern)(PrefillArgs, CUtensorMap, CUtensorMap, CUtensorMap) = nullptr;
#define PKV_RG_CASE(GG)                                                                                    \
  case GG:                                                                                                 \
    kern = cap ? prefill_ragged_kernel<GG, T, true, STAGED> : prefill_ragged_kernel<GG, T, false, STAGED>; \
    break;
  switch (G) {
    PKV_RG_CASE(1) PKV_RG_CASE(2) PKV_RG_CASE(4) PKV_RG_CASE(8)
    default: return cudaErrorInvalidValue;
  }
#undef PKV_RG_CASE
  cudaError_t e = ensure_smem_limit(kern, kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, grid, kThreads, kSmemBytes, s, a, tq, tk, tv);
}

}  // namespace

cudaError_t launch_prefill_ragged(const PrefillArgs& a, const RaggedRows& r, int group, int dtype, bool cap, bool split,
                                  int grid, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const void* none = a.q;  // a batch without keys: the maps are not read
  cudaError_t e = make_rows_map(a.q, dtype, a.num_qo_heads, r.total_q, r.q_stride, group, kTM / group, tq);
  if (e == cudaSuccess) e = make_rows_map(r.k ? r.k : none, dtype, a.num_kv_heads, r.total_kv, r.k_stride, 1, kBN, tk);
  if (e == cudaSuccess) e = make_rows_map(r.v ? r.v : none, dtype, a.num_kv_heads, r.total_kv, r.v_stride, 1, kBN, tv);
  if (e != cudaSuccess) return e;
  if (dtype == PKV_BF16)
    return split ? launch_t<__nv_bfloat16, true>(a, group, cap, grid, tq, tk, tv, stream)
                 : launch_t<__nv_bfloat16, false>(a, group, cap, grid, tq, tk, tv, stream);
  return split ? launch_t<__half, true>(a, group, cap, grid, tq, tk, tv, stream)
               : launch_t<__half, false>(a, group, cap, grid, tq, tk, tv, stream);
}

}  // namespace pkv
