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
// (remainders 1.8e-9 and 1.2e-10, below the rounding of the float result).
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

#include <algorithm>
#include <cmath>
#include <type_traits>

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
constexpr int kAhead = 6;        // passes in flight per warp
constexpr int kAxSmem = kAxWarps * kAhead * 2048;

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
  int part_passes;               // passes each of them takes
  uint64_t freq[kAxPairs];       // theta^(-2i/R) / (2 pi) * 2^64
  uint8_t axis[kAxPairs];
};

// pos * F modulo a turn: pos = u - 2^32 for a negative one.
__device__ __forceinline__ uint32_t turn_hi(int32_t pos, uint64_t freq) {  // bits 32 .. 63
  const uint32_t u = static_cast<uint32_t>(pos), flo = static_cast<uint32_t>(freq);
  return u * static_cast<uint32_t>(freq >> 32) + __umulhi(u, flo) - (pos < 0 ? flo : 0u);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}

// Sine and cosine of pos * F turns.
__device__ __forceinline__ void sincos_turn(int32_t pos, uint64_t freq, float& s, float& c) {
  const uint32_t turn = turn_hi(pos, freq);
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

// A pair turned in double precision (quadrant and rest of the 64-bit turn as above, the
// Taylor series to x^17 and x^18: remainders below 2^-60), each element rounded to a
// float by truncation with the lost part in its last bit, so that rounding the float to
// e4m3 rounds the double's value correctly.
__device__ __noinline__ float2 turn_pair_double(float x, float y, int32_t pos, uint64_t freq) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * freq;
  const uint64_t quad = (turn + (uint64_t{1} << 61)) >> 62;
  const double a = static_cast<double>(static_cast<int64_t>(turn - (quad << 62))) * 3.4061215800865545e-19;  // 2 pi / 2^64
  const double z = a * a;
  double ps = 1.0 / 355687428096000.0, pc = -1.0 / 6402373705728000.0;  // 1/17!, 1/18!
  ps = fma(z, ps, -1.0 / 1307674368000.0);
  pc = fma(z, pc, 1.0 / 20922789888000.0);
  ps = fma(z, ps, 1.0 / 6227020800.0);
  pc = fma(z, pc, -1.0 / 87178291200.0);
  ps = fma(z, ps, -1.0 / 39916800.0);
  pc = fma(z, pc, 1.0 / 479001600.0);
  ps = fma(z, ps, 1.0 / 362880.0);
  pc = fma(z, pc, -1.0 / 3628800.0);
  ps = fma(z, ps, -1.0 / 5040.0);
  pc = fma(z, pc, 1.0 / 40320.0);
  ps = fma(z, ps, 1.0 / 120.0);
  pc = fma(z, pc, -1.0 / 720.0);
  ps = fma(z, ps, -1.0 / 6.0);
  pc = fma(z, pc, 1.0 / 24.0);
  pc = fma(z, pc, -0.5);
  const double sa = fma(a * z, ps, a), ca = fma(z, pc, 1.0);
  const double u = (quad & 1) ? ca : sa, v = (quad & 1) ? sa : ca;
  const double s = (quad & 2) ? -u : u, c = ((quad + 1) & 2) ? -v : v;
  const double w[2] = {x * c - y * s, y * c + x * s};
  float r[2];
  for (int i = 0; i < 2; ++i) {
    r[i] = __double2float_rz(w[i]);
    if (static_cast<double>(r[i]) != w[i]) r[i] = __uint_as_float(__float_as_uint(r[i]) | 1u);
  }
  return make_float2(r[0], r[1]);
}

// Two floats to two e4m3 codes, the first in the low byte: round to nearest even,
// past +-448 to +-448, NaN to NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float2 (&f)[4]) {
  return make_uint2(pack_e4m3(f[0].x, f[0].y) | (pack_e4m3(f[1].x, f[1].y) << 16),
                    pack_e4m3(f[2].x, f[2].y) | (pack_e4m3(f[3].x, f[3].y) << 16));
}

// Codes of x (1 - 2^-19) and of x (1 + 2^-19).  Where the two are the same, so is that of
// every value between them.
__device__ __forceinline__ uint2 pack_e4m3x8_both(const float2 (&x)[4], bool& differ) {
  float2 lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo[j] = fmul2(x[j], make_float2(1.f - 0x1p-19f, 1.f - 0x1p-19f));
    hi[j] = fmul2(x[j], make_float2(1.f + 0x1p-19f, 1.f + 0x1p-19f));
  }
  const uint2 a = pack_e4m3x8(lo), b = pack_e4m3x8(hi);
  differ |= a.x != b.x || a.y != b.y;
  return a;
}
__device__ __forceinline__ bool near_border(float x) {
  return pack_e4m3(x * (1.f - 0x1p-19f), 0.f) != pack_e4m3(x * (1.f + 0x1p-19f), 0.f);
}

template <typename T>
__device__ __forceinline__ uint4 pack_16x8(const float2 (&f)[4]) {
  return make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y), pack2<T>(f[2].x, f[2].y), pack2<T>(f[3].x, f[3].y));
}

// The exponent byte of a head row of which each of LPH neighbouring lanes holds 16
// elements: from the largest finite magnitude's float32 exponent field.  Magnitudes of
// a 16-bit type are ordered like their bits, so the row is searched two elements an
// instruction; a row with an infinity or a NaN is searched again without them.
template <typename T, int LPH>
__device__ __forceinline__ uint32_t row_exponent(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kInf = kBf ? 0x7f80u : 0x7c00u;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
#pragma unroll
  for (int o = LPH / 2; o >= 1; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max(m & 0xffffu, m >> 16);
  if (__any_sync(0xffffffffu, m >= kInf)) {
    m = 0;
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
      m = max(m, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
    }
    for (int o = LPH / 2; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  const uint32_t field = kBf ? m >> 7 : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m)))) >> 23;
  return static_cast<uint32_t>(max(static_cast<int>(field) - 7, 1));
}

// One warp takes one token, or some of its passes when there are few tokens.  A pass
// is 4 16-byte loads per lane: RPP keys' and values' head rows, or 2 RPP queries',
// D/16 lanes to a row.  A rotating lane holds 8 pairs as 16 bytes of each half of the
// rotated part, any other lane 16 bytes of each half of the rest, so nothing is shuffled
// but the 8-bit rows' largest magnitudes.  The rows arrive through a ring in shared memory of kAhead
// passes (cp.async; a lane reads back only what it copied itself, so its own wait is the
// only synchronisation), which runs across tokens and ahead of the page lookups.
//
// A key's code depends on which side of a border between two e4m3 values its turned
// element falls.  A float turn is off by about 2^-23 of the pair's length; elements
// within 2^-19 of their size of a border (one in some 20 000) are turned again in double
// precision, so elements of at least an eighth of their pair's length get the code of the
// exact rotation, e4m3's subnormals among them.  (A smaller one may get its second
// nearest, when the two are equally near to within 2^-21 of the pair's length.)
template <int D, typename T, bool OUT8>
__global__ void __launch_bounds__(kAxThreads, 2) append_axes_kernel(const __grid_constant__ AxesArgs a) {
  constexpr int LPH = D / 16;     // lanes per head row
  constexpr int RPP = 32 / LPH;   // head rows per load
  __shared__ int32_t s_indptr[kAxIndptr];
  __shared__ uint64_t s_freq[kAxPairs];
  extern __shared__ __align__(16) uint8_t s_ring[];
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool staged = a.batch < kAxIndptr;
  if (staged)
    for (int i = threadIdx.x; i <= a.batch; i += blockDim.x) s_indptr[i] = a.append_indptr[i];
  if (threadIdx.x < kAxPairs) s_freq[threadIdx.x] = a.freq[threadIdx.x];
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPH, hsub = lane / LPH;
  const bool turns = sub < a.rot_chunks;
  // Element offsets of this lane's two 8-element chunks in a turned head row, and in a
  // value row: neighbouring lanes' chunks are neighbours, so that every copy and store
  // of a warp covers whole sectors.  (Values on their way to the 16-bit cache are one
  // piece of 32 bytes a lane instead: 74.4 against 75.3 us for 16 prompts of 18 000
  // tokens, where the 8-bit cache takes 59.0 against 58.0 us.)
  const int rest = (LPH - a.rot_chunks) * 8;
  const int off_a = turns ? sub * 8 : a.rot_chunks * 16 + (sub - a.rot_chunks) * 8;
  const int off_b = off_a + (turns ? a.rot_chunks * 8 : rest);
  const int voff_a = OUT8 ? sub * 8 : sub * 16, voff_b = OUT8 ? D / 2 + sub * 8 : sub * 16 + 8;
  uint32_t axes = 0;  // 4 bits per pair
  if (turns)
#pragma unroll
    for (int j = 0; j < 8; ++j) axes |= static_cast<uint32_t>(a.axis[sub * 8 + j]) << (4 * j);
  const int P = a.page_size, Hkv = a.num_kv_heads, Hq = a.q_in ? a.num_qo_heads : 0;
  const int kv_passes = (Hkv + RPP - 1) / RPP;
  const int all_passes = kv_passes + (Hq + 2 * RPP - 1) / (2 * RPP);
  const int part = static_cast<int>(blockIdx.x % a.parts);
  const int pass0 = part * a.part_passes, pass1 = min(all_passes, pass0 + a.part_passes);
  const T* k_new = static_cast<const T*>(a.k_new);
  const T* v_new = static_cast<const T*>(a.v_new);
  const T* q_in = static_cast<const T*>(a.q_in);
  const int64_t t_begin = static_cast<int64_t>(blockIdx.x / a.parts) * kAxWarps + warp;
  const int64_t t_step = static_cast<int64_t>(gridDim.x / a.parts) * kAxWarps;
  // The copy side: the next pass to issue, and its place in the ring.  A lane's four
  // chunks of a pass are 512 bytes apart, so a warp's copies and reads are contiguous.
  const uint32_t ring = smem_addr(s_ring) + warp * kAhead * 2048 + lane * 16;
  int64_t next_t = t_begin;
  int next_pass = pass0, next_at = 0;
  auto issue = [&] {
    if (next_t < a.nnz) {
      const uint32_t dst = ring + next_at * 2048;
      if (next_pass < kv_passes) {
        const int r = next_pass * RPP + hsub;
        if (r < Hkv) {
          const int64_t row = (next_t * Hkv + r) * D;
          cp_async_16(dst, k_new + row + off_a, 16);
          cp_async_16(dst + 512, k_new + row + off_b, 16);
          cp_async_16(dst + 1024, v_new + row + voff_a, 16);
          cp_async_16(dst + 1536, v_new + row + voff_b, 16);
        }
      } else {
        const int r = (next_pass - kv_passes) * 2 * RPP + hsub;
        const T* src = q_in + (next_t * Hq + r) * D;
        if (r < Hq) {
          cp_async_16(dst, src + off_a, 16);
          cp_async_16(dst + 512, src + off_b, 16);
        }
        if (r + RPP < Hq) {
          cp_async_16(dst + 1024, src + RPP * D + off_a, 16);
          cp_async_16(dst + 1536, src + RPP * D + off_b, 16);
        }
      }
      next_at = next_at + 1 == kAhead ? 0 : next_at + 1;
      if (++next_pass == pass1) {
        next_pass = pass0;
        next_t += t_step;
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < kAhead - 1; ++i) issue();
  int at = 0;
  // The oldest pass in flight, arrived; its place is free again for the pass issued next.
  auto take = [&](uint4 (&x)[4]) {
    cp_async_wait<kAhead - 2>();
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = ld_shared_v4(ring + at * 2048 + i * 512);
    at = at + 1 == kAhead ? 0 : at + 1;
    issue();
  };
  int32_t err = 0;
  for (int64_t t = t_begin; t < a.nnz; t += t_step) {
    // A token that is skipped leaves its passes in the ring.
    auto skip = [&] {
      uint4 x[4];
      for (int pass = pass0; pass < pass1; ++pass) take(x);
    };
    int32_t pos = 0;  // lane i: the token's position on axis i
    if (a.positions && lane < a.num_axes) pos = __ldg(a.positions + lane * a.nnz + t);
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
    const int64_t n_new = static_cast<int64_t>(a1) - a0;
    // A request claiming more new tokens than it holds, or more keys than an int
    // counts, is skipped whole.
    if (t < a0 || t >= a1 || n_new > kv_len || kv_len > INT32_MAX || (n_pages > 0 && (last < 1 || last > P))) {
      err |= kErrAppendLayout;
      skip();
      continue;
    }
    const int place = static_cast<int>(kv_len - n_new + (t - a0));
    const int page_no = place / P, slot = place - page_no * P;
    const int page = __ldg(a.kv_indices + p0 + page_no);
    if (page < 0 || page >= a.num_pages) {
      err |= kErrPageIndex;
      skip();
      continue;
    }
    if (!a.positions) pos = place;
    float2 c[4], s[4], ns[4];  // cosines, sines and their negatives
    if (a.rot_chunks > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int32_t pj = __shfl_sync(0xffffffffu, pos, (axes >> (4 * j)) & 15u);
        float sj, cj;
        sincos_turn(pj, s_freq[turns ? sub * 8 + j : 0], sj, cj);
        (j & 1 ? s[j >> 1].y : s[j >> 1].x) = sj;
        (j & 1 ? ns[j >> 1].y : ns[j >> 1].x) = -sj;
        (j & 1 ? c[j >> 1].y : c[j >> 1].x) = cj;
      }
    }
    // The turned pair of chunks of a row.
    auto turn = [&](float2 (&fa)[4], float2 (&fb)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = fa[j], v = fb[j];
        fa[j] = ffma2(u, c[j], fmul2(v, ns[j]));
        fb[j] = ffma2(v, c[j], fmul2(u, s[j]));
      }
    };
    const int64_t head0 = static_cast<int64_t>(page) * 2 * Hkv;  // first (K|V, head) block of the page
    for (int pass = pass0; pass < pass1; ++pass) {
      uint4 x[4];
      take(x);
      if (pass < kv_passes) {
        const int r = pass * RPP + hsub;
        // K of head r is block r of the page, V of head r block Hkv + r.
        const int64_t k_row = (head0 + r) * P + slot, v_row = k_row + static_cast<int64_t>(Hkv) * P;
        uint32_t ks = 0, vs = 0;
        if constexpr (OUT8) {
          ks = row_exponent<T, LPH>(x[0], x[1]);
          vs = row_exponent<T, LPH>(x[2], x[3]);
        }
        float2 fa[4], fb[4];
        to_float2x4<T>(x[0], fa);
        to_float2x4<T>(x[1], fb);
        if constexpr (OUT8) {
          const float km = __uint_as_float((254u - ks) << 23), vm = __uint_as_float((254u - vs) << 23);  // 2^(127 - s)
          const float2 km2 = make_float2(km, km), vm2 = make_float2(vm, vm);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fa[j] = fmul2(fa[j], km2);
            fb[j] = fmul2(fb[j], km2);
          }
          uint2 ca, cb;  // the key's codes
          if (!turns) {
            ca = pack_e4m3x8(fa);
            cb = pack_e4m3x8(fb);
          } else {
            turn(fa, fb);
            bool near = false;
            ca = pack_e4m3x8_both(fa, near);
            cb = pack_e4m3x8_both(fb, near);
            if (near) {
              float2 ua[4], ub[4];  // unturned
              to_float2x4<T>(x[0], ua);
              to_float2x4<T>(x[1], ub);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float& ra = j & 1 ? fa[j >> 1].y : fa[j >> 1].x;
                float& rb = j & 1 ? fb[j >> 1].y : fb[j >> 1].x;
                if (near_border(ra) || near_border(rb)) {
                  const int axis = (axes >> (4 * j)) & 15u;
                  const int32_t pj = a.positions ? __ldg(a.positions + axis * a.nnz + t) : place;
                  const float2 d = turn_pair_double((j & 1 ? ua[j >> 1].y : ua[j >> 1].x) * km,
                                                    (j & 1 ? ub[j >> 1].y : ub[j >> 1].x) * km, pj, s_freq[sub * 8 + j]);
                  ra = d.x;
                  rb = d.y;
                }
              }
              ca = pack_e4m3x8(fa);
              cb = pack_e4m3x8(fb);
            }
          }
          if (r < Hkv) {
            uint8_t* dst = static_cast<uint8_t*>(a.kv) + k_row * D;
            *reinterpret_cast<uint2*>(dst + off_a) = ca;
            *reinterpret_cast<uint2*>(dst + off_b) = cb;
            to_float2x4<T>(x[2], fa);
            to_float2x4<T>(x[3], fb);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              fa[j] = fmul2(fa[j], vm2);
              fb[j] = fmul2(fb[j], vm2);
            }
            uint8_t* vd = static_cast<uint8_t*>(a.kv) + v_row * D;
            *reinterpret_cast<uint2*>(vd + voff_a) = pack_e4m3x8(fa);
            *reinterpret_cast<uint2*>(vd + voff_b) = pack_e4m3x8(fb);
            if (sub == 0) {
              a.scales[k_row] = static_cast<uint8_t>(ks);
              a.scales[v_row] = static_cast<uint8_t>(vs);
            }
          }
        } else if (r < Hkv) {
          T* kd = static_cast<T*>(a.kv) + k_row * D;
          T* vd = static_cast<T*>(a.kv) + v_row * D;
          if (turns) {
            turn(fa, fb);
            x[0] = pack_16x8<T>(fa);
            x[1] = pack_16x8<T>(fb);
          }
          *reinterpret_cast<uint4*>(kd + off_a) = x[0];
          *reinterpret_cast<uint4*>(kd + off_b) = x[1];
          *reinterpret_cast<uint4*>(vd + voff_a) = x[2];
          *reinterpret_cast<uint4*>(vd + voff_b) = x[3];
        }
      } else {
        const int r = (pass - kv_passes) * 2 * RPP + hsub;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (turns) {
            float2 fa[4], fb[4];
            to_float2x4<T>(x[2 * h], fa);
            to_float2x4<T>(x[2 * h + 1], fb);
            turn(fa, fb);
            x[2 * h] = pack_16x8<T>(fa);
            x[2 * h + 1] = pack_16x8<T>(fb);
          }
          if (r + h * RPP < Hq) {
            T* dst = static_cast<T*>(a.q_out) + (t * Hq + r + h * RPP) * D;
            *reinterpret_cast<uint4*>(dst + off_a) = x[2 * h];
            *reinterpret_cast<uint4*>(dst + off_b) = x[2 * h + 1];
          }
        }
      }
    }
  }
  if (err && a.err) atomicOr(a.err, err);
}

template <int D, typename T>
cudaError_t launch_t(const AxesArgs& a, int grid, cudaStream_t s) {
  void (*kern)(AxesArgs) = a.scales ? append_axes_kernel<D, T, true> : append_axes_kernel<D, T, false>;
  cudaError_t e = ensure_smem_limit(kern, kAxSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, grid, kAxThreads, kAxSmem, s, a);
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
    if (!(turn < 4503599627370496.0)) return false;  // theta so small that a step's turns fill the double
    a.freq[i] = static_cast<uint64_t>((turn - std::floor(turn)) * 18446744073709551616.0);  // 2^64; theta < 1: over a turn a step
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
  // Rows are read ahead of those that are written, so they turn in place or elsewhere.
  const auto from = reinterpret_cast<uintptr_t>(q_in), to = reinterpret_cast<uintptr_t>(q_out);
  const uint64_t q_bytes = static_cast<uint64_t>(nnz) * p->num_qo_heads * p->head_dim * 2;
  if (from != to && (from < to ? to - from : from - to) < q_bytes) return PKV_ERR_INVALID_ARG;
  a.append_indptr = append_indptr_d;
  a.kv_indptr = kv_indptr_d;
  a.kv_indices = kv_indices_d;
  a.kv_last = kv_last_page_len_d;
  a.positions = rope ? positions_d : nullptr;
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
  // Few tokens are shared by several warps each, down to one pass a warp, as long as all
  // of them run at once (16 warps on every SM).
  const int rpp = 32 / (p->head_dim / 16);
  const int hq = q_in ? p->num_qo_heads : 0;
  const int passes = (p->num_kv_heads + rpp - 1) / rpp + (hq + 2 * rpp - 1) / (2 * rpp);
  const int64_t share = std::max<int64_t>(static_cast<int64_t>(sms) * 16 / nnz, 1);
  const int parts = static_cast<int>(share < passes ? share : passes);
  a.part_passes = (passes + parts - 1) / parts;
  a.parts = (passes + a.part_passes - 1) / a.part_passes;
  const int64_t want = (nnz + kAxWarps - 1) / kAxWarps * a.parts, room = static_cast<int64_t>(sms) * 2 / a.parts * a.parts;
  const int grid = static_cast<int>(want < room ? want : std::max<int64_t>(room, a.parts));
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
