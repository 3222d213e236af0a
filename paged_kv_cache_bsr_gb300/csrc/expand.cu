// expand.cu -- the keys and values of an 8-bit cache's pages as 16-bit values, packed
// into 16-row pages of a plan's workspace for the tensor-core prefill kernel.
//
// value = e4m3(code) * 2^(s - 127): 4 significant bits and a power of two, so the
// 16-bit value is exact within the type's range (past it infinite, below its subnormals'
// step rounded) and the prefill over the copy computes with the cache's own values.  One pass over the batch's keys, whatever the
// number of query rows: 1 byte read and 2 written per element.  32-byte stores matter
// most: with two 16-byte stores per lane, each of which fills half of every sector, a
// batch of 15 000 tokens x 8 kv heads took 25 us, with whole sectors 16 us.
#include <cuda_runtime.h>

#include "pkv_bsr.h"
#include "pkv_device.cuh"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr int kExpandThreads = 256;

// 16 bytes or one, or zeros (`other`) where `use` is 0.
__device__ __forceinline__ uint4 ld_nc_v4_if(const void* p, int use) {
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"(use));
  return r;
}
__device__ __forceinline__ uint32_t ld_nc_u8_if(const void* p, int use, uint32_t other) {
  uint32_t r = other;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\t@p ld.global.nc.u8 %0, [%1];\n\t}"
      : "+r"(r)
      : "l"(p), "r"(use));
  return r;
}

// 32 bytes as one store (a whole sector; two 16-byte stores write each sector twice).
__device__ __forceinline__ void st_v8(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

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

// One CTA takes kBlocks (K|V, head) blocks of a packed page at a time, so that a short
// batch still reaches every SM.  Thread t owns row (t / 8) % 16 and its 16-byte piece
// t % 8 (16 codes) in every second block; all its pieces and their exponent bytes load
// together (predicated, so that nothing waits between them).
constexpr int kBlocks = 8;
template <typename T>
__global__ void __launch_bounds__(kExpandThreads, 4) expand_pages_kernel(const __grid_constant__ PackArgs a,
                                                                      const uint8_t* __restrict__ scales) {
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nblk = 2 * a.num_kv_heads;  // (K|V, head) blocks of a page
  const int parts = (nblk + kBlocks - 1) / kBlocks;
  const int64_t items = static_cast<int64_t>(a.hdr->num_packed) * parts;
  const int t = threadIdx.x, piece = t % 8, r = (t / 8) % 16, half = t / 128;
  const uint8_t* kv = static_cast<const uint8_t*>(a.kv);
  uint4* out = static_cast<uint4*>(a.packed);
  for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
    const int p = static_cast<int>(w / parts), h0 = static_cast<int>(w % parts) * kBlocks + half;
    const PackedSrc sp = a.src[p];
    int64_t row0 = 0;  // this thread's row in block 0 of its source page
    int have = 0;
    if (r < sp.ntok) {
      const int u = sp.tok0 + r;
      const int page = __ldg(a.kv_indices + u / a.page_size);
      if (page >= 0 && page < a.num_pages) {
        row0 = static_cast<int64_t>(page) * nblk * a.page_size + u % a.page_size;
        have = 1;
      } else {
        atomicOr(a.err, kErrPageIndex);
      }
    }
    uint4 x[kBlocks / 2];
    uint32_t s[kBlocks / 2];
#pragma unroll
    for (int i = 0; i < kBlocks / 2; ++i) {
      const int64_t row = row0 + static_cast<int64_t>(h0 + 2 * i) * a.page_size;
      const int use = have & (h0 + 2 * i < nblk ? 1 : 0);
      x[i] = ld_nc_v4_if(kv + row * kD + piece * 16, use);
      s[i] = ld_nc_u8_if(scales + row, use, 127u);
    }
    uint4* dst = out + (static_cast<int64_t>(p) * nblk * 16 + r) * (kD * 2 / 16) + piece * 2;
#pragma unroll
    for (int i = 0; i < kBlocks / 2; ++i) {
      const float scale = __uint_as_float(s[i] << 23);
      const uint2 v0 = expand4<T>(x[i].x, scale), v1 = expand4<T>(x[i].y, scale), v2 = expand4<T>(x[i].z, scale),
                  v3 = expand4<T>(x[i].w, scale);
      uint4* d = dst + static_cast<int64_t>(h0 + 2 * i) * 16 * (kD * 2 / 16);
      if (h0 + 2 * i < nblk) {
        st_v8(d, make_uint4(v0.x, v0.y, v1.x, v1.y), make_uint4(v2.x, v2.y, v3.x, v3.y));
      }
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
