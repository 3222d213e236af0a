// expand.cu -- the keys and values of an 8-bit cache's pages as 16-bit values, packed
// into 16-row pages of a plan's workspace for the tensor-core prefill kernel.
//
// value = e4m3(code) * 2^(s - 127): 4 significant bits and a power of two, so the
// bf16 (or, within its range, fp16) value is exact and the prefill over the copy
// computes with the cache's own values.  One pass over the batch's keys, whatever the
// number of query rows: 1 byte read and 2 written per element, HBM-bound.
#include <cuda_runtime.h>

#include "pkv_bsr.h"
#include "pkv_device.cuh"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr int kExpandThreads = 256;

// Four codes times 2^(s - 127) to two pairs of T.
template <typename T>
__device__ __forceinline__ uint2 expand4(uint32_t w, float scale) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_uint2(pack2<T>(a.x * scale, a.y * scale), pack2<T>(b.x * scale, b.y * scale));
}

// One CTA per packed page at a time.  Thread t owns row (t / 8) % 16 and its 16-byte
// piece t % 8 (16 codes) in every second (K|V, head) block, so it looks its source row
// up once and then moves its pieces back to back.
template <typename T>
__global__ void __launch_bounds__(kExpandThreads) expand_pages_kernel(const __grid_constant__ PackArgs a,
                                                                      const uint8_t* __restrict__ scales) {
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nblk = 2 * a.num_kv_heads;  // (K|V, head) blocks of a page
  const int n_packed = a.hdr->num_packed;
  const int t = threadIdx.x, piece = t % 8, r = (t / 8) % 16, half = t / 128;
  const uint8_t* kv = static_cast<const uint8_t*>(a.kv);
  uint4* out = static_cast<uint4*>(a.packed);
  for (int p = blockIdx.x; p < n_packed; p += gridDim.x) {
    const PackedSrc sp = a.src[p];
    int64_t row0 = -1;  // this thread's row in block 0 of its source page
    if (r < sp.ntok) {
      const int u = sp.tok0 + r;
      const int page = __ldg(a.kv_indices + u / a.page_size);
      if (page >= 0 && page < a.num_pages)
        row0 = static_cast<int64_t>(page) * nblk * a.page_size + u % a.page_size;
      else
        atomicOr(a.err, kErrPageIndex);
    }
    uint4* dst = out + (static_cast<int64_t>(p) * nblk * 16 + r) * (kD * 2 / 16) + piece * 2;
#pragma unroll 4
    for (int hs = half; hs < nblk; hs += 2) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      float scale = 0.f;
      if (row0 >= 0) {
        const int64_t row = row0 + static_cast<int64_t>(hs) * a.page_size;
        x = ld_nc_v4(kv + row * kD + piece * 16);
        scale = __uint_as_float(static_cast<uint32_t>(__ldg(scales + row)) << 23);
      }
      const uint2 v0 = expand4<T>(x.x, scale), v1 = expand4<T>(x.y, scale), v2 = expand4<T>(x.z, scale),
                  v3 = expand4<T>(x.w, scale);
      uint4* d = dst + static_cast<int64_t>(hs) * 16 * (kD * 2 / 16);
      d[0] = make_uint4(v0.x, v0.y, v1.x, v1.y);
      d[1] = make_uint4(v2.x, v2.y, v3.x, v3.y);
    }
  }
}

}  // namespace

cudaError_t launch_expand_pages(const PackArgs& a, const uint8_t* scales, int head_dim, int dtype, int grid,
                                cudaStream_t stream) {
  if (head_dim != kD || a.page_size <= 0) return cudaErrorInvalidValue;
  if (dtype == PKV_BF16)
    return launch_dependent(expand_pages_kernel<__nv_bfloat16>, grid, kExpandThreads, 0, stream, a, scales);
  if (dtype == PKV_F16) return launch_dependent(expand_pages_kernel<__half>, grid, kExpandThreads, 0, stream, a, scales);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
