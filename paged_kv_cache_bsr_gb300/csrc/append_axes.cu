// append_axes.cu -- append new tokens' K/V into their pages with rotary positions
// on several axes, into the 16-bit cache or into the 8-bit one.
//
// A token of a picture or a video has a position on each axis (time, height,
// width); a text token has the same position on all of them.  The head row's
// rotated part of R elements holds R/2 pairs (i, i + R/2), pair i turns by
//     angle = pos[axis(i)] * theta^(-2i/R)
//     x'_i       = x_i cos - x_{i+R/2} sin
//     x'_{i+R/2} = x_{i+R/2} cos + x_i sin,
// and elements from R on are copied.  The caller's sections say how many pairs
// each axis has; pkv_append_paged_kv (append.cu) is the one-axis case whose
// positions come from the page table.
//
// Angles.  theta^(-2i/R) / (2 pi) is held as a 64-bit binary fraction F of a turn,
// so pos * F modulo 2^64 is the angle modulo a turn, with no rounding for any int32
// position: two integer multiplications, no argument reduction in floating
// point.  The top 32 bits (1.5e-9 rad) are split into a quadrant and a rest of at
// most an eighth of a turn, whose sine and cosine come from their Taylor series
// (remainders 1.8e-9 and 9e-11, below the rounding of the float result).
//
// 8-bit cache.  Each head row (token, kv head, K or V) is stored as e4m3 codes
// and one power-of-two scale 2^(s - 127), s = max(E - 7, 1) with E the exponent
// field of the row's largest finite |x| as a float32, taken before the rotation:
// that value times 2^(127 - s) lies in [128, 256), a turned pair stays below
// 256 sqrt(2) < 448, and s does not depend on the position or on any rounding.
// A power of two makes the scaling exact, here and in the kernels that read the
// cache.
#include <cuda_runtime.h>
#include <math.h>

#include <cmath>

#include "pkv_bsr.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kAxWarps = 8;
constexpr int kAxThreads = kAxWarps * 32;
constexpr int kAxPairs = 64;     // D / 2 for the largest head_dim built (128)
constexpr int kAxIndptr = 1024;  // append_indptr entries staged in shared memory
constexpr int kMaxAxes = 4;

struct AxesArgs {
  const int32_t* append_indptr;  // [batch + 1] new-token rows per request
  const int32_t* kv_indptr;      // [batch + 1] pages per request (new tokens included)
  const int32_t* kv_indices;
  const int32_t* kv_last;        // [batch] valid slots of each last page
  const int32_t* positions;      // [num_axes, nnz], or nullptr: the place in the request, on every axis
  const void* k_new;             // [nnz, Hkv, D]
  const void* v_new;             // [nnz, Hkv, D]
  void* kv;                      // [num_pages, 2, Hkv, P, D], 16-bit values or e4m3 codes
  uint8_t* scales;               // 8-bit cache: [num_pages, 2, Hkv, P] exponent bytes
  const void* q_in;              // [nnz, Hq, D] or nullptr
  void* q_out;                   // [nnz, Hq, D]; may equal q_in
  int32_t* err;                  // device error word or nullptr
  int64_t num_pages;
  int64_t nnz;
  int batch;
  int num_qo_heads;
  int num_kv_heads;
  int page_size;
  int rot_chunks;                // R / 16: lanes of a head row that rotate
  int num_axes;
  int parts;                     // warps that share a token
  int part_passes;               // passes of head rows each of them takes
  uint64_t freq[kAxPairs];       // theta^(-2i/R) / (2 pi) * 2^64
  uint8_t axis[kAxPairs];
};

// Sine and cosine of pos * F turns.
__device__ __forceinline__ void sincos_turn(int32_t pos, uint64_t freq, float& s, float& c) {
  const uint32_t u = static_cast<uint32_t>(pos), fhi = static_cast<uint32_t>(freq >> 32),
                 flo = static_cast<uint32_t>(freq);
  // Bits 32..63 of pos * F: pos = u - 2^32 for a negative one.
  const uint32_t turn = u * fhi + __umulhi(u, flo) - (pos < 0 ? flo : 0u);
  const uint32_t quad = (turn + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(turn - (quad << 30))) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float ps = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  ps = fmaf(z, ps, 1.f / 120.f);
  ps = fmaf(z, ps, -1.f / 6.f);
  const float sx = fmaf(x * z, ps, x);
  float pc = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  pc = fmaf(z, pc, -1.f / 720.f);
  pc = fmaf(z, pc, 1.f / 24.f);
  pc = fmaf(z, pc, -0.5f);
  const float cx = fmaf(z, pc, 1.f);
  const float a = (quad & 1u) ? cx : sx, b = (quad & 1u) ? sx : cx;
  s = (quad & 2u) ? -a : a;
  c = ((quad + 1u) & 2u) ? -b : b;
}

// Two floats to two e4m3 codes, the first in the low byte: round to nearest even,
// past +-448 to +-448, NaN to NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&f)[8]) {
  return make_uint2(pack_e4m3(f[0], f[1]) | (pack_e4m3(f[2], f[3]) << 16),
                    pack_e4m3(f[4], f[5]) | (pack_e4m3(f[6], f[7]) << 16));
}

// One warp takes one token's head rows (keys, then queries, then values), or a
// part of them when there are few tokens, D/16 lanes to a row.  A rotating lane
// holds 8 pairs as 16 bytes of each half of the rotated part, any other lane 32
// bytes in a row, so nothing is shuffled but the 8-bit rows' largest values.
template <int D, typename T, bool OUT8>
__global__ void __launch_bounds__(kAxThreads) append_axes_kernel(const __grid_constant__ AxesArgs a) {
  constexpr int LPH = D / 16;     // lanes per head row
  constexpr int RPP = 32 / LPH;   // head rows per pass
  constexpr int CHUNK = 2;        // passes loaded before the first is used
  __shared__ int32_t s_indptr[kAxIndptr];
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool staged = a.batch < kAxIndptr;
  if (staged)
    for (int i = threadIdx.x; i <= a.batch; i += blockDim.x) s_indptr[i] = a.append_indptr[i];
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPH, hsub = lane / LPH;
  const bool turns = sub < a.rot_chunks;
  // Element offsets of this lane's two 8-element chunks in a head row.
  const int off_a = turns ? sub * 8 : a.rot_chunks * 16 + (sub - a.rot_chunks) * 16;
  const int off_b = turns ? a.rot_chunks * 8 + sub * 8 : off_a + 8;
  uint64_t freq[8];
  uint32_t axes = 0;  // 4 bits per pair
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    freq[j] = turns ? a.freq[sub * 8 + j] : 0;
    axes |= (turns ? static_cast<uint32_t>(a.axis[sub * 8 + j]) : 0u) << (4 * j);
  }
  const int P = a.page_size, Hkv = a.num_kv_heads, Hq = a.q_in ? a.num_qo_heads : 0;
  const int rows = 2 * Hkv + Hq;
  const T* k_new = static_cast<const T*>(a.k_new);
  const T* v_new = static_cast<const T*>(a.v_new);
  const T* q_in = static_cast<const T*>(a.q_in);
  int32_t err = 0;
  const int64_t units = a.nnz * a.parts;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kAxWarps + warp; u < units;
       u += static_cast<int64_t>(gridDim.x) * kAxWarps) {
    const int64_t t = u / a.parts;
    const int part = static_cast<int>(u - t * a.parts);
    // The request holding new row t: the last b with append_indptr[b] <= t.
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      const int v = staged ? s_indptr[mid] : __ldg(a.append_indptr + mid);
      if (v <= t) lo = mid; else hi = mid;
    }
    const int b = lo;
    const int a0 = staged ? s_indptr[b] : __ldg(a.append_indptr + b);
    const int a1 = staged ? s_indptr[b + 1] : __ldg(a.append_indptr + b + 1);
    const int p0 = __ldg(a.kv_indptr + b);
    const int n_pages = __ldg(a.kv_indptr + b + 1) - p0;
    const int last = __ldg(a.kv_last + b);
    const int64_t kv_len = n_pages > 0 ? static_cast<int64_t>(n_pages - 1) * P + last : 0;
    // A request claiming more new tokens than it holds, or more keys than an int
    // counts, is skipped whole.
    if (t < a0 || t >= a1 || a1 - a0 > kv_len || kv_len > INT32_MAX || (n_pages > 0 && (last < 1 || last > P))) {
      err |= kErrAppendLayout;
      continue;
    }
    const int place = static_cast<int>(kv_len - (a1 - a0) + (t - a0));
    const int page = __ldg(a.kv_indices + p0 + place / P);
    if (page < 0 || page >= a.num_pages) {
      err |= kErrPageIndex;
      continue;
    }
    const int slot = place % P;
    float c[8], s[8];
    if (a.rot_chunks > 0) {
      int32_t pos = place;  // lane x: the token's position on axis x
      if (a.positions && lane < a.num_axes) pos = __ldg(a.positions + lane * a.nnz + t);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int32_t pj = __shfl_sync(0xffffffffu, pos, (axes >> (4 * j)) & 15u);
        sincos_turn(pj, freq[j], s[j], c[j]);
      }
    }
    const int64_t head0 = static_cast<int64_t>(page) * 2 * Hkv;  // first (K|V, head) block of the page
    const int r_end = min(rows, (part + 1) * a.part_passes * RPP);
    for (int r0 = part * a.part_passes * RPP; r0 < r_end; r0 += CHUNK * RPP) {
      uint4 xa[CHUNK], xb[CHUNK];
#pragma unroll
      for (int k = 0; k < CHUNK; ++k) {
        const int r = r0 + k * RPP + hsub;
        xa[k] = xb[k] = make_uint4(0u, 0u, 0u, 0u);
        if (r < r_end) {
          const T* src = r < Hkv ? k_new + (t * Hkv + r) * D
                                 : (r < Hkv + Hq ? q_in + (t * Hq + (r - Hkv)) * D
                                                 : v_new + (t * Hkv + (r - Hkv - Hq)) * D);
          xa[k] = *reinterpret_cast<const uint4*>(src + off_a);
          xb[k] = *reinterpret_cast<const uint4*>(src + off_b);
        }
      }
#pragma unroll
      for (int k = 0; k < CHUNK; ++k) {
        const int r = r0 + k * RPP + hsub;
        const bool valid = r < r_end, is_q = r >= Hkv && r < Hkv + Hq, is_v = r >= Hkv + Hq;
        float fa[8], fb[8];
        to_float8<T>(xa[k], fa);
        to_float8<T>(xb[k], fb);
        uint32_t field = 0;
        if constexpr (OUT8) {
          // The row's largest finite |x|, as float bits (ordered like the values).
          uint32_t mx = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t ba = __float_as_uint(fa[j]) & 0x7fffffffu, bb = __float_as_uint(fb[j]) & 0x7fffffffu;
            if (ba < 0x7f800000u) mx = max(mx, ba);
            if (bb < 0x7f800000u) mx = max(mx, bb);
          }
#pragma unroll
          for (int o = LPH / 2; o >= 1; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          field = mx >> 23;
        }
        if (!valid) continue;
        const uint32_t sc = max(static_cast<int>(field) - 7, 1);
        if (OUT8 && !is_q) {
          const float mul = __uint_as_float((254u - sc) << 23);  // 2^(127 - sc)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            fa[j] *= mul;
            fb[j] *= mul;
          }
        }
        if (turns && !is_v) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = fa[j], y = fb[j];
            fa[j] = fmaf(x, c[j], -y * s[j]);
            fb[j] = fmaf(y, c[j], x * s[j]);
          }
        }
        if (is_q) {
          T* dst = static_cast<T*>(a.q_out) + (t * Hq + (r - Hkv)) * D;
          *reinterpret_cast<uint4*>(dst + off_a) = from_float8<T>(fa);
          *reinterpret_cast<uint4*>(dst + off_b) = from_float8<T>(fb);
        } else {
          // K of head h is block h of the page, V of head h block Hkv + h.
          const int64_t row = (head0 + (is_v ? r - Hq : r)) * P + slot;
          if constexpr (OUT8) {
            uint8_t* dst = static_cast<uint8_t*>(a.kv) + row * D;
            *reinterpret_cast<uint2*>(dst + off_a) = pack_e4m3x8(fa);
            *reinterpret_cast<uint2*>(dst + off_b) = pack_e4m3x8(fb);
            if (sub == 0) a.scales[row] = static_cast<uint8_t>(sc);
          } else {
            T* dst = static_cast<T*>(a.kv) + row * D;
            *reinterpret_cast<uint4*>(dst + off_a) = from_float8<T>(fa);
            *reinterpret_cast<uint4*>(dst + off_b) = from_float8<T>(fb);
          }
        }
      }
    }
  }
  if (err && a.err) atomicOr(a.err, err);
}

template <int D, typename T>
cudaError_t launch_t(const AxesArgs& a, int grid, cudaStream_t s) {
  return a.scales ? launch_dependent(append_axes_kernel<D, T, true>, grid, kAxThreads, 0, s, a)
                  : launch_dependent(append_axes_kernel<D, T, false>, grid, kAxThreads, 0, s, a);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Check the rotation and write the pairs' axes and frequencies.
bool set_rotation(AxesArgs& a, const pkv_rope_axes* rope, int head_dim) {
  a.rot_chunks = 0;
  a.num_axes = 1;
  if (!rope) return true;
  if (!(rope->theta > 0.0) || !std::isfinite(rope->theta)) return false;
  if (rope->rotary_dim < 16 || rope->rotary_dim > head_dim || rope->rotary_dim % 16) return false;
  if (rope->num_axes < 1 || rope->num_axes > kMaxAxes) return false;
  const int pairs = rope->rotary_dim / 2;
  int left[kMaxAxes] = {0, 0, 0, 0};
  int64_t sum = 0;
  for (int x = 0; x < rope->num_axes; ++x) {
    if (rope->sections[x] < 0 || rope->sections[x] > pairs) return false;
    left[x] = rope->sections[x];
    sum += left[x];
  }
  if (sum != pairs) return false;
  a.rot_chunks = rope->rotary_dim / 16;
  a.num_axes = rope->num_axes;
  // theta^(-2i/R) as the product of a power by i / 8 and one by i % 8.
  const double step = -2.0 / rope->rotary_dim * std::log2(rope->theta);
  double by8[8], by1[8];
  for (int i = 0; i < 8; ++i) {
    by8[i] = std::exp2(step * (8 * i)) / 6.283185307179586476925286766559;
    by1[i] = std::exp2(step * i);
  }
  for (int i = 0, x = 0; i < pairs; ++i) {
    while (left[x] == 0) x = (x + 1) % rope->num_axes;  // an axis without pairs left is passed over
    a.axis[i] = static_cast<uint8_t>(x);
    --left[x];
    if (rope->interleaved) x = (x + 1) % rope->num_axes;
    // Good to about 2^-50 of its value: the angle of position p to |p| times that.
    const double turn = by8[i / 8] * by1[i % 8];
    a.freq[i] = static_cast<uint64_t>(std::ldexp(turn - std::floor(turn), 64));  // theta < 1: over a turn a step
  }
  return true;
}

pkv_status append_axes(const pkv_params* p, const pkv_rope_axes* rope, int batch, int64_t nnz, int64_t num_pages,
                       const int32_t* append_indptr_d, const int32_t* kv_indptr_d, const int32_t* kv_indices_d,
                       const int32_t* kv_last_page_len_d, const int32_t* positions_d, const void* k_new,
                       const void* v_new, void* kv, uint8_t* scales, bool out8, const void* q_in, void* q_out,
                       int32_t* error_d, void* stream) {
  if (!p || batch < 0 || nnz < 0 || num_pages < 0) return PKV_ERR_INVALID_ARG;
  if (p->num_qo_heads <= 0 || p->num_kv_heads <= 0 || p->page_size <= 0) return PKV_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (p->dtype != PKV_F16 && p->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  AxesArgs a{};
  if (!set_rotation(a, rope, p->head_dim)) return PKV_ERR_INVALID_ARG;
  if (nnz == 0) return PKV_OK;
  if (batch == 0 || nnz > INT32_MAX) return PKV_ERR_INVALID_ARG;
  // A token's head rows are counted in int.
  if (p->num_qo_heads > (1 << 20) || p->num_kv_heads > (1 << 20)) return PKV_ERR_UNSUPPORTED;
  if (!append_indptr_d || !kv_indptr_d || !kv_indices_d || !kv_last_page_len_d || !k_new || !v_new || !kv)
    return PKV_ERR_INVALID_ARG;
  if (out8 && !scales) return PKV_ERR_INVALID_ARG;
  if (!q_in != !q_out) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(kv) || !aligned16(q_in) || !aligned16(q_out) ||
      !aligned4(append_indptr_d) || !aligned4(kv_indptr_d) || !aligned4(kv_indices_d) ||
      !aligned4(kv_last_page_len_d) || !aligned4(positions_d) || !aligned4(error_d) || !aligned4(scales))
    return PKV_ERR_INVALID_ARG;
  a.append_indptr = append_indptr_d;
  a.kv_indptr = kv_indptr_d;
  a.kv_indices = kv_indices_d;
  a.kv_last = kv_last_page_len_d;
  a.positions = positions_d;
  a.k_new = k_new;
  a.v_new = v_new;
  a.kv = kv;
  a.scales = out8 ? scales : nullptr;
  a.q_in = q_in;
  a.q_out = q_out;
  a.err = error_d;
  a.num_pages = num_pages;
  a.nnz = nnz;
  a.batch = batch;
  a.num_qo_heads = p->num_qo_heads;
  a.num_kv_heads = p->num_kv_heads;
  a.page_size = p->page_size;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  // Few tokens are shared by several warps each, down to one pass of head rows a
  // warp, until there are 16 warps for every SM.
  const int rpp = 32 / (p->head_dim / 16);
  const int rows = 2 * p->num_kv_heads + (q_in ? p->num_qo_heads : 0);
  const int passes = (rows + rpp - 1) / rpp;
  const int64_t share = (static_cast<int64_t>(sms) * 16 + nnz - 1) / nnz;
  const int parts = static_cast<int>(share < passes ? share : passes);
  a.part_passes = (passes + parts - 1) / parts;
  a.parts = (passes + a.part_passes - 1) / a.part_passes;
  const int64_t want = (nnz * a.parts + kAxWarps - 1) / kAxWarps;
  const int grid = static_cast<int>(want < static_cast<int64_t>(sms) * 8 ? want : static_cast<int64_t>(sms) * 8);
  auto s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p->head_dim == 128)
    e = p->dtype == PKV_BF16 ? launch_t<128, __nv_bfloat16>(a, grid, s) : launch_t<128, __half>(a, grid, s);
  else
    e = p->dtype == PKV_BF16 ? launch_t<64, __nv_bfloat16>(a, grid, s) : launch_t<64, __half>(a, grid, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_append_paged_kv_axes(const pkv_params* params, const pkv_rope_axes* rope, int batch,
                                               int64_t nnz, int64_t num_pages, const int32_t* append_indptr_d,
                                               const int32_t* kv_indptr_d, const int32_t* kv_indices_d,
                                               const int32_t* kv_last_page_len_d, const int32_t* positions_d,
                                               const void* k_new, const void* v_new, void* kv_data, const void* q_in,
                                               void* q_out, int32_t* error_d, void* stream) {
  return pkv::append_axes(params, rope, batch, nnz, num_pages, append_indptr_d, kv_indptr_d, kv_indices_d,
                          kv_last_page_len_d, positions_d, k_new, v_new, kv_data, nullptr, false, q_in, q_out,
                          error_d, stream);
}

extern "C" pkv_status pkv_append_paged_kv8(const pkv_params* params, const pkv_rope_axes* rope, int batch, int64_t nnz,
                                           int64_t num_pages, const int32_t* append_indptr_d,
                                           const int32_t* kv_indptr_d, const int32_t* kv_indices_d,
                                           const int32_t* kv_last_page_len_d, const int32_t* positions_d,
                                           const void* k_new, const void* v_new, void* kv8, uint8_t* kv8_scales,
                                           const void* q_in, void* q_out, int32_t* error_d, void* stream) {
  return pkv::append_axes(params, rope, batch, nnz, num_pages, append_indptr_d, kv_indptr_d, kv_indices_d,
                          kv_last_page_len_d, positions_d, k_new, v_new, kv8, kv8_scales, true, q_in, q_out, error_d,
                          stream);
}
