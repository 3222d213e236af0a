// weights.cu -- the attention weight of every cached key, summed over query rows
// (pkv_add_key_weights).
//
// Mathematics.  For key j of a request and kv head h, over the call's rows i of the
// request that see j and the G query heads that share h:
//     w[j, h] = decay * w[j, h] + sum_{i, g} exp(cap(sm_scale q_ig . k_jh) - lse_ig).
// lse comes from the attention call over the same keys, so a probability needs one dot
// product and no second look at the softmax: every key is independent of the others.
// Keys are the M axis of the products throughout (a lane or a fragment row is a key),
// so a key's sum stays in one thread or one quad; no two workers add to the same weight,
// no atomics, and equal calls give equal bits.
//
// Two kernels, both reading K once:
//  - stream: few query rows per request (a decode step).  HBM-bound on K.  A warp takes
//    16 keys at a time straight from global memory into the A fragments of mma.sync
//    m16n8k16 (which dims a k step holds does not matter as long as the query fragments
//    hold the same ones, so a lane's 16-byte chunk of a row serves whole k steps without
//    shared memory), against columns of 8 (row, head) pairs held in registers.  Two tiles
//    are in flight per warp and 16 warps per SM.
//  - tile: many rows per request (prompts, or the last rows of one).  S^T = K Q^T on
//    tcgen05: a CTA owns 128 keys of one kv head in tensor memory and streams 64-column
//    tiles of (row, head) pairs past them by TMA; a thread is a key, and sums its
//    exponentials over the columns in registers.  Few key tiles before many rows are
//    shared by the CTAs of a cluster, which add their sums in rank order through
//    distributed shared memory.
// Both find their work from the device's row pointers alone: request b's tiles start at
//     first(b) = floor(kv_indptr[b] P / K) + b        (K keys a tile),
// which leaves each request room for its ceil(len / K) tiles and at most one unused
// place, so no scan over the batch is needed and a captured graph follows the arrays.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "prefill_kernel.cuh"

namespace pkv {
namespace {

constexpr unsigned kFullMask = 0xffffffffu;

struct WeightArgs {
  const void* q;             // [total_q, Hq, D]
  const void* kv;            // [num_pages, 2, Hkv, P, D] 16-bit values or e4m3 codes
  const uint8_t* scales;     // 8-bit cache: exponent bytes [num_pages, 2, Hkv, P]
  const float* lse;          // [total_q, Hq]
  float* weights;            // [num_pages, Hkv, P]
  const int32_t* qo_indptr;  // nullptr: one row per request
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* kv_last;
  const int32_t* weighed;    // nullptr: every key was there before
  int32_t* err;              // or nullptr
  int64_t num_pages, kv_pages, total_q;
  int batch, hq, hkv, page_size;
  int lg;                    // log2 of the group
  int causal;
  float scale;               // sm_scale (log2(e) sm_scale without a cap)
  float cap, decay;
  uint32_t small_div;        // page_size < 16: ceil(4096 / page_size)
};

__device__ __forceinline__ void flag(const WeightArgs& a, int bits) {
  if (a.err) atomicOr(a.err, bits);
}

// First tile (of K keys) of request b in the numbering above.
template <int K>
__device__ __forceinline__ int64_t first_tile(const WeightArgs& a, int b) {
  return static_cast<int64_t>(__ldg(a.kv_indptr + b)) * a.page_size / K + b;
}

// The last request whose first tile is at or before u, by the whole warp, 32 probes a step.
template <int K>
__device__ __forceinline__ int find_request(const WeightArgs& a, int64_t u, int lane) {
  int lo = 0, n = a.batch;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const unsigned at = __ballot_sync(kFullMask, i < n && first_tile<K>(a, lo + i) <= u);
    const int k = max(__popc(at) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  return lo;
}

struct Request {
  int page0;     // first entry of kv_indices
  int kv_len;
  int row0, rows;
  int weighed;
  bool ok;       // the arrays name a request that exists
};

__device__ __forceinline__ Request load_request(const WeightArgs& a, int b) {
  Request r;
  const int p0 = __ldg(a.kv_indptr + b), p1 = __ldg(a.kv_indptr + b + 1), last = __ldg(a.kv_last + b);
  r.row0 = a.qo_indptr ? __ldg(a.qo_indptr + b) : b;
  const int row1 = a.qo_indptr ? __ldg(a.qo_indptr + b + 1) : b + 1;
  r.weighed = a.weighed ? __ldg(a.weighed + b) : INT_MAX;
  const bool pages = p0 >= 0 && p1 >= p0 && p1 <= a.kv_pages;
  const int64_t len = p1 > p0 ? static_cast<int64_t>(p1 - p0 - 1) * a.page_size + last : 0;
  r.ok = pages && (p1 == p0 || (last >= 1 && last <= a.page_size)) && len <= INT_MAX - 256 && r.row0 >= 0 &&
         row1 >= r.row0 && row1 <= a.total_q;
  r.page0 = p0;
  r.kv_len = r.ok ? static_cast<int>(len) : 0;
  r.rows = row1 - r.row0;
  return r;
}

// ---------------------------------------------------------------------------- stream
__device__ __forceinline__ uint4 ld_stream_v4(const void* p, bool use) {
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"(static_cast<int>(use)));
  return r;
}

template <typename T>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes to two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

constexpr int kStreamKeys = 16;
constexpr int kStreamThreads = 256;

// A tile on its way: lane (g, t) holds 16-byte chunks t, t + 4, ... of keys g and g + 8.
template <int CH>
struct KeyTile {
  uint4 k[2][CH];
  float scale[2];  // 8-bit cache: 2^(s - 127) of the two keys
  float old;       // lanes t = 0, 1: the weight of key g + 8 t before the call, decayed
  float* at;       // and where it goes (nullptr: nowhere)
};

template <int D, typename T, bool KV8, bool CAP>
__global__ void __launch_bounds__(kStreamThreads, 2) key_weights_stream_kernel(const __grid_constant__ WeightArgs a) {
  constexpr int CH = KV8 ? D / 64 : D / 32;  // chunks of a row per lane
  constexpr int ES = KV8 ? 1 : 2;            // bytes per element
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = a.page_size;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * (kStreamThreads / 32) + (threadIdx.x >> 5);
  const int64_t workers = static_cast<int64_t>(gridDim.x) * (kStreamThreads / 32);
  const int64_t listed = min(max(static_cast<int64_t>(__ldg(a.kv_indptr + a.batch)), int64_t{0}), a.kv_pages);
  const int64_t U = listed * P / kStreamKeys + a.batch;  // places of tiles per kv head
  const int64_t run = (U * a.hkv + workers - 1) / workers;
  int64_t f = worker * run;
  const int64_t f_end = min(f + run, U * a.hkv);
  while (f < f_end) {
    const int h = static_cast<int>(f / U);
    const int64_t base = h * U, u = f - base;
    const int b = find_request<kStreamKeys>(a, u, lane);
    const Request rq = load_request(a, b);
    const int64_t c0 = first_tile<kStreamKeys>(a, b), c1 = b + 1 < a.batch ? first_tile<kStreamKeys>(a, b + 1) : U;
    const int64_t stop = min(f_end, base + max(c1, u + 1));
    f = stop;
    if (!rq.ok) {
      if (lane == 0) flag(a, kErrAppendLayout);
      continue;
    }
    const int n_tiles = (rq.kv_len + kStreamKeys - 1) / kStreamKeys;
    const int t_end = static_cast<int>(min(static_cast<int64_t>(n_tiles), stop - base - c0));
    int tile = static_cast<int>(max(u - c0, int64_t{0}));
    if (tile >= t_end) continue;

    const int cols = rq.rows << a.lg;
    const int off = rq.kv_len - rq.rows;  // causal: row i sees keys up to i + off
    // Columns c0 .. c0 + 7: lane (g, t) loads chunk(s) t, t + 4, ... of column c0 + g, and
    // the negated lse of columns c0 + 2 t and c0 + 2 t + 1 (out: such a column adds nothing).
    uint32_t qf[D / 16][2];
    float qs[2] = {1.f, 1.f}, nl[2];
    bool out[2];
    int see[2];  // the last key that the column's row sees
    auto load_columns = [&](int first) {
      const int c = first + g;
      const bool use = c < cols;
      const T* row = static_cast<const T*>(a.q) +
                     (static_cast<int64_t>(rq.row0 + (use ? c >> a.lg : 0)) * a.hq + (h << a.lg) + (use ? c & ((1 << a.lg) - 1) : 0)) * D;
      if constexpr (!KV8) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const uint4 x = use ? ld_nc_v4(row + (t + 4 * i) * 8) : make_uint4(0u, 0u, 0u, 0u);
          qf[2 * i][0] = x.x;
          qf[2 * i][1] = x.y;
          qf[2 * i + 1][0] = x.z;
          qf[2 * i + 1][1] = x.w;
        }
      } else {
        // fp16 of q over the power of two below its row's largest element.
        uint4 raw[CH][2];
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            raw[i][k] = use ? ld_nc_v4(row + (t + 4 * i) * 16 + k * 8) : make_uint4(0u, 0u, 0u, 0u);
            float v[8];
            to_float8<T>(raw[i][k], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
          }
        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 2));
        const uint32_t field = min(max(__float_as_uint(mx) >> 23, 1u), 253u);
        const float mul = __uint_as_float((254u - field) << 23);
        const float back = __uint_as_float(field << 23);
        qs[0] = __shfl_sync(kFullMask, back, 8 * t);
        qs[1] = __shfl_sync(kFullMask, back, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v[8];
            to_float8<T>(raw[i][k], v);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              qf[i * 4 + k * 2 + e][0] = pack2<__half>(v[4 * e] * mul, v[4 * e + 1] * mul);
              qf[i * 4 + k * 2 + e][1] = pack2<__half>(v[4 * e + 2] * mul, v[4 * e + 3] * mul);
            }
          }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int cc = first + 2 * t + k;
        const int i = cc >> a.lg;
        float l = -INFINITY;
        if (cc < cols) l = __ldg(a.lse + static_cast<int64_t>(rq.row0 + i) * a.hq + (h << a.lg) + (cc & ((1 << a.lg) - 1)));
        out[k] = l == -INFINITY;
        nl[k] = -l * kLog2e;
        see[k] = a.causal ? i + off : INT_MAX;
      }
    };

    // The tile whose page ids are being fetched: its first key's page (of the request) and slot.
    int ids_tile = tile, pg = static_cast<int>(static_cast<int64_t>(tile) * kStreamKeys / P);
    int slot = tile * kStreamKeys - pg * P;
    int id[2], at_slot[2];
    auto fetch_ids = [&] {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int x = slot + g + 8 * k;
        const int skip = P < kStreamKeys ? static_cast<int>((static_cast<uint32_t>(x) * a.small_div) >> 12) : 0;
        const bool in = ids_tile * kStreamKeys + g + 8 * k < rq.kv_len;
        id[k] = in ? __ldg(a.kv_indices + rq.page0 + pg + skip) : -1;
        at_slot[k] = in ? x - skip * P : -1;
      }
      ++ids_tile;
      slot += kStreamKeys;
      if (P >= kStreamKeys) {
        if (slot == P) {
          slot = 0;
          ++pg;
        }
      } else {
        const int full = static_cast<int>((static_cast<uint32_t>(slot) * a.small_div) >> 12);
        pg += full;
        slot -= full * P;
      }
    };
    auto fill = [&](KeyTile<CH>& kt, int tile_no) {
      const uint8_t* kv = static_cast<const uint8_t*>(a.kv);
      bool use[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        use[k] = id[k] >= 0 && id[k] < a.num_pages;
        if (!use[k] && at_slot[k] >= 0 && t == 0) flag(a, kErrPageIndex);
        const int64_t row = use[k] ? (static_cast<int64_t>(id[k]) * 2 * a.hkv + h) * P + at_slot[k] : 0;
        const uint8_t* src = kv + row * (D * ES) + t * 16;
#pragma unroll
        for (int i = 0; i < CH; ++i) kt.k[k][i] = ld_stream_v4(src + i * 64, use[k]);
        if constexpr (KV8) kt.scale[k] = __uint_as_float(static_cast<uint32_t>(use[k] ? __ldg(a.scales + row) : 0) << 23);
      }
      const int me = t & 1;
      const bool mine = t < 2 && (me ? use[1] : use[0]);
      kt.at = mine ? a.weights + (static_cast<int64_t>(me ? id[1] : id[0]) * a.hkv + h) * P + (me ? at_slot[1] : at_slot[0])
                   : nullptr;
      const bool before = mine && a.decay != 0.f && tile_no * kStreamKeys + g + 8 * me < rq.weighed;
      kt.old = before ? *kt.at * a.decay : 0.f;
    };
    auto use_tile = [&](const KeyTile<CH>& kt, int tile_no) {
      const int j = tile_no * kStreamKeys + g;
      float sum[2] = {0.f, 0.f};
      for (int first = 0; first < cols; first += 8) {
        if (cols > 8) load_columns(first);
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const uint4 x = kt.k[0][i], z = kt.k[1][i];
          if constexpr (!KV8) {
            mma_16x8x16<T>(sa, x.x, z.x, x.y, z.y, qf[2 * i][0], qf[2 * i][1]);
            mma_16x8x16<T>(sb, x.z, z.z, x.w, z.w, qf[2 * i + 1][0], qf[2 * i + 1][1]);
          } else {
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_half(xw[w], a0, a2);
              e4m3x4_to_half(zw[w], a1, a3);
              mma_16x8x16<__half>((w & 1) ? sb : sa, a0, a1, a2, a3, qf[i * 4 + w][0], qf[i * 4 + w][1]);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // key j + 8 (k / 2), column 2 t + k % 2
          const int c = k & 1, r = k >> 1;
          float s = sa[k] + sb[k];
          if constexpr (KV8) s *= qs[c] * kt.scale[r];
          float y;
          if constexpr (CAP)
            y = fmaf(a.cap * kLog2e, tanh_from_log2(s * (a.scale * 2.f * kLog2e / a.cap)), nl[c]);
          else
            y = fmaf(s, a.scale, nl[c]);
          const float p = fast_exp2(y);
          sum[r] += out[c] || j + 8 * r > see[c] ? 0.f : p;
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(kFullMask, sum[r], 1);
        sum[r] += __shfl_xor_sync(kFullMask, sum[r], 2);
      }
      if (kt.at) *kt.at = kt.old + ((t & 1) ? sum[1] : sum[0]);
    };

    if (cols <= 8) load_columns(0);
    KeyTile<CH> even, odd;
    fetch_ids();
    fill(even, tile);
    fetch_ids();
    for (;;) {
      if (tile + 1 < t_end) {
        fill(odd, tile + 1);
        fetch_ids();
      }
      use_tile(even, tile);
      if (++tile >= t_end) break;
      if (tile + 1 < t_end) {
        fill(even, tile + 1);
        fetch_ids();
      }
      use_tile(odd, tile);
      if (++tile >= t_end) break;
    }
  }
}

// ------------------------------------------------------------------------------ tile
constexpr int kD = prefill_impl::kD;
constexpr int kTileKeys = 128;
constexpr int kTileCols = 64;             // (row, head) pairs of one product
constexpr int kQStages = 5;
constexpr int kSBufs = 3;
constexpr uint32_t kQHalf = kTileCols * 128;  // 64 of the 128 dims of 64 columns
constexpr uint32_t kQTile = 2 * kQHalf;
constexpr int kTileThreads = 320;         // two groups of 4 warps, the Q producer, the MMA issuer
constexpr int kTileSmem = kQStages * kQTile + 1024;
constexpr uint32_t kWTmemCols = 256;      // K 64, then three S^T buffers: two CTAs share an SM's 512
constexpr uint32_t kColSt = 64;

struct TileShared {
  uint64_t q_full[kQStages], q_empty[kQStages], s_full[kSBufs], s_empty[kSBufs], k_full, drain;
  uint32_t tmem;
  int abort;
  alignas(16) float nl[2][2][kTileCols];  // read as float4; [group][buffer]: negated lse in log2 units, -inf for a column that adds nothing
  float part[2][kTileKeys];
  float sum[kTileKeys];
};

// All 128 threads of a group arrive; true where any of them brought true.
__device__ __forceinline__ bool group_any(int group, bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(x)), "r"(group + 1)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.f32 %0, [r];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ void tmem_ld64_sync(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "{\n\t.reg .b32 a1;\n\tadd.u32 a1, %64, 32;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, "
      "%45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [a1];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : PKV_R32(r), PKV_R32((r + 32))
      : "r"(taddr)
      : "memory");
}

// Four e4m3 codes to two pairs of T (exact).
template <typename T>
__device__ __forceinline__ void e4m3x4_to(uint32_t w, uint32_t& lo, uint32_t& hi) {
  e4m3x4_to_half(w, lo, hi);
  if constexpr (!std::is_same<T, __half>::value) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack2<T>(x.x, x.y);
    hi = pack2<T>(y.x, y.y);
  }
}

template <typename T, bool KV8, bool CAP>
__global__ void __launch_bounds__(kTileThreads, 2)
    key_weights_tile_kernel(const __grid_constant__ WeightArgs a, const __grid_constant__ CUtensorMap tq, int share) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ TileShared sh;
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = a.page_size;
  const uint32_t rank = share > 1 ? cluster_rank() : 0u;
  // This cluster's key tile: kv heads of a tile side by side.
  const int64_t item = blockIdx.x / share;
  const int64_t u = item / a.hkv;
  const int h = static_cast<int>(item - u * a.hkv);
  const int b = find_request<kTileKeys>(a, u, lane);
  const Request rq = load_request(a, b);
  const int64_t tile = u - first_tile<kTileKeys>(a, b);
  if (!rq.ok || tile < 0 || tile * kTileKeys >= rq.kv_len) {  // the same for all CTAs of a cluster
    if (!rq.ok && tid == 0) flag(a, kErrAppendLayout);
    return;
  }
  const int k0 = static_cast<int>(tile) * kTileKeys;
  const int off = rq.kv_len - rq.rows;
  const int row_first = a.causal ? min(max(k0 - off, 0), rq.rows) : 0;  // the first row that sees key k0
  const int per = kTileCols >> a.lg;                                    // rows of a column tile
  const int n_all = (rq.rows - row_first + per - 1) / per;
  const int n = n_all > static_cast<int>(rank) ? (n_all - 1 - static_cast<int>(rank)) / share + 1 : 0;  // rank, rank + share, ...

  uint32_t base = smem_addr(smem_raw);
  base = (base + 1023u) & ~1023u;
  auto bar = [](uint64_t& x) { return smem_addr(&x); };
  if (tid == 0) {
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(bar(sh.q_full[i]), 1);
      mbar_init(bar(sh.q_empty[i]), 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(bar(sh.s_full[i]), 1);
      mbar_init(bar(sh.s_empty[i]), 128);
    }
    mbar_init(bar(sh.k_full), 256);
    mbar_init(bar(sh.drain), 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_addr(&sh.tmem), kWTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* give_up = &sh.abort;
  // Bounded wait; false when it ran out (recorded) or another role gave up.
  auto wait = [&](uint64_t& x, uint32_t parity) {
    const uint32_t at = bar(x);
    if (mbar_try_wait(at, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(at, parity)) {
      if (*give_up) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        flag(a, kErrWaitTimeout);
        *give_up = 1;
        return false;
      }
    }
    return true;
  };

  float old = 0.f;
  float* at = nullptr;
  if (warp == 8) {
    // ------------------------------------------------------------ Q producer
    if (lane == 0) {
      int i = 0;
      for (; i < n; ++i) {
        const int s = i % kQStages;
        if (i >= kQStages && !wait(sh.q_empty[s], (i / kQStages - 1) & 1)) break;
        mbar_arrive_expect_tx(bar(sh.q_full[s]), kQTile);
        const int row = rq.row0 + row_first + (static_cast<int>(rank) + i * share) * per;
        for (int x = 0; x < 2; ++x)
          tma_load_3d(base + s * kQTile + x * kQHalf, &tq, x * 64, h << a.lg, row, bar(sh.q_full[s]));
      }
      // The copies in flight land before the CTA may leave.
      for (int k = max(i - kQStages, 0); k < i; ++k) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar(sh.q_full[k % kQStages]), (k / kQStages) & 1))
          if (global_timer_ns() - t0 > kWaitLimitNs) {
            flag(a, kErrWaitTimeout);
            break;
          }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_f16(kFmt, kTileKeys, kTileCols, 0);
      const uint64_t dq = sw128_desc(base, 16, 1024);
      const uint32_t hi = static_cast<uint32_t>(dq >> 32), q_lo = static_cast<uint32_t>(dq);
      bool ok = n == 0 || wait(sh.k_full, 0);
      tc_fence_after();
      for (int i = 0; i < n && ok; ++i) {
        const int s = i % kQStages, d = i % kSBufs;
        if (i >= kSBufs && !(ok = wait(sh.s_empty[d], (i / kSBufs - 1) & 1))) break;
        if (!(ok = wait(sh.q_full[s], (i / kQStages) & 1))) break;
        tc_fence_after();
        const uint32_t dst = tmem + kColSt + d * kTileCols, b0 = q_lo + s * (kQTile >> 4);
        prefill_impl::umma_ts_lo<false>(dst, tmem, b0, hi, idesc);
#pragma unroll
        for (int kk = 1; kk < kD / 16; ++kk)
          prefill_impl::umma_ts_lo<true>(dst, tmem + kk * 8, b0 + (kk / 4) * (kQHalf >> 4) + (kk % 4) * 2, hi, idesc);
        umma_commit(bar(sh.q_empty[s]));
        umma_commit(bar(sh.s_full[d]));
      }
      // Every MMA issued so far must finish before tensor memory is released.
      umma_commit(bar(sh.drain));
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar(sh.drain), 0))
        if (global_timer_ns() - t0 > kWaitLimitNs) {
          flag(a, kErrWaitTimeout);
          break;
        }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ keys, then their sums
    const int x = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane, j = k0 + r;   // this thread's key
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int gt = tid & 127;                        // thread of the group
    bool use = j < rq.kv_len;
    int64_t row = 0;
    if (use) {
      const int pg = j / P, page = __ldg(a.kv_indices + rq.page0 + pg);
      use = page >= 0 && page < a.num_pages;
      if (use) {
        row = (static_cast<int64_t>(page) * 2 * a.hkv + h) * P + (j - pg * P);
        if (x == 0 && rank == 0) {
          at = a.weights + (static_cast<int64_t>(page) * a.hkv + h) * P + (j - pg * P);
          if (a.decay != 0.f && j < rq.weighed) old = *at * a.decay;
        }
      } else if (x == 0) {
        flag(a, kErrPageIndex);
      }
    }
    float mul = a.scale;
    {
      // Group x brings the key's dims 64 x .. 64 x + 63 into its lane of tensor memory, two
      // 16-bit values a column: the A operand.
      uint32_t w[32];
      if constexpr (KV8) {
        const uint8_t* src = static_cast<const uint8_t*>(a.kv) + row * kD + x * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = ld_stream_v4(src + i * 16, use);
          e4m3x4_to<T>(v.x, w[8 * i], w[8 * i + 1]);
          e4m3x4_to<T>(v.y, w[8 * i + 2], w[8 * i + 3]);
          e4m3x4_to<T>(v.z, w[8 * i + 4], w[8 * i + 5]);
          e4m3x4_to<T>(v.w, w[8 * i + 6], w[8 * i + 7]);
        }
        mul *= __uint_as_float(static_cast<uint32_t>(use ? __ldg(a.scales + row) : 0) << 23);
      } else {
        const T* src = static_cast<const T*>(a.kv) + row * kD + x * 64;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = ld_stream_v4(src + i * 8, use);
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
      }
      tmem_st32(tmem + lane_off + x * 32, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(sh.k_full));
    }
    // Column gt (< 64) of a column tile: its negated lse, -inf where it adds nothing.
    auto load_nl = [&](int i) {
      float v = -INFINITY;
      if (i < n && gt < kTileCols) {
        const int q_row = row_first + (static_cast<int>(rank) + i * share) * per + (gt >> a.lg);
        if (q_row < rq.rows) {
          const float l =
              __ldg(a.lse + static_cast<int64_t>(rq.row0 + q_row) * a.hq + (h << a.lg) + (gt & ((1 << a.lg) - 1)));
          v = l == -INFINITY ? -INFINITY : -l * kLog2e;
        }
      }
      return v;
    };
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    float next_nl = load_nl(x);
    bool ok = true;
    for (int i = x, k = 0; i < n; i += 2, ++k) {  // every warp meets the group's barrier n times, come what may
      float* nl = sh.nl[x][k & 1];
      if (gt < kTileCols) nl[gt] = next_nl;
      const bool some_out = group_any(x, gt < kTileCols && next_nl == -INFINITY);
      next_nl = load_nl(i + 2);
      const int d = i % kSBufs;
      if (ok) ok = __all_sync(kFullMask, wait(sh.s_full[d], (i / kSBufs) & 1));
      if (!ok) continue;
      tc_fence_after();
      uint32_t sr[64];
      tmem_ld64_sync(tmem + lane_off + kColSt + d * kTileCols, sr);
      tc_fence_before();
      mbar_arrive(bar(sh.s_empty[d]));
      const int q_row = row_first + (static_cast<int>(rank) + i * share) * per;
      // The first column whose row sees this key.
      const int c_min = a.causal ? max(j - off - q_row, 0) << a.lg : 0;
      const bool masked = some_out || (a.causal && k0 + kTileKeys - 1 - off > q_row);
      const float2 mul2 = make_float2(mul, mul);
      float k_in = 0.f, k_out = 0.f;
      if constexpr (CAP) {
        k_in = mul * 2.f * kLog2e / a.cap;
        k_out = a.cap * kLog2e;
      }
#pragma unroll
      for (int c = 0; c < kTileCols; c += 4) {
        const float4 l4 = *reinterpret_cast<const float4*>(nl + c);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 s = make_float2(__uint_as_float(sr[c + 2 * e]), __uint_as_float(sr[c + 2 * e + 1]));
          const float2 l = e ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
          float2 y;
          if constexpr (CAP) {
            // cap tanh(y) = k_out - 2 k_out / (e^(2y) + 1), e^(2y) = 2^(s k_in)
            float2 z = fmul2(s, make_float2(k_in, k_in));
            z.x = fast_exp2(z.x);
            z.y = fast_exp2(z.y);
            z = fadd2(z, make_float2(1.f, 1.f));
            z.x = fast_rcp(z.x);
            z.y = fast_rcp(z.y);
            y = fadd2(ffma2(z, make_float2(-2.f * k_out, -2.f * k_out), make_float2(k_out, k_out)), l);
          } else {
            y = ffma2(s, mul2, l);
          }
          float2 p = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          if (masked) {
            if (c + 2 * e < c_min || l.x == -INFINITY) p.x = 0.f;
            if (c + 2 * e + 1 < c_min || l.y == -INFINITY) p.y = 0.f;
          }
          acc[e] = fadd2(acc[e], p);
        }
      }
    }
    const float2 s2 = fadd2(acc[0], acc[1]);
    sh.part[x][r] = s2.x + s2.y;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, kWTmemCols);
  if (sh.abort) at = nullptr;  // sums that a wait left incomplete
  if (share > 1) {
    if (tid < kTileKeys) sh.sum[tid] = sh.part[0][tid] + sh.part[1][tid];
    __syncwarp();
    cluster_sync_all();
    if (rank == 0 && at) {
      float v = 0.f;
      for (int k = 0; k < share; ++k) v += ld_cluster_f32(smem_addr(&sh.sum[tid]), k);
      *at = old + v;
    }
    __syncwarp();
    cluster_sync_all();  // a CTA's sums stay until they have been read
  } else if (at) {
    *at = old + (sh.part[0][tid] + sh.part[1][tid]);
  }
}

template <int D, typename T>
cudaError_t launch_stream(const WeightArgs& a, bool cap, int grid, cudaStream_t s) {
  void (*kern)(WeightArgs) = nullptr;
  if (a.scales)
    kern = cap ? key_weights_stream_kernel<D, T, true, true> : key_weights_stream_kernel<D, T, true, false>;
  else
    kern = cap ? key_weights_stream_kernel<D, T, false, true> : key_weights_stream_kernel<D, T, false, false>;
  return launch_dependent(kern, grid, kStreamThreads, 0, s, a);
}

template <typename T>
cudaError_t launch_tile(const WeightArgs& a, bool cap, int64_t items, int share, const CUtensorMap& tq, cudaStream_t s) {
  void (*kern)(WeightArgs, CUtensorMap, int) = nullptr;
  if (a.scales)
    kern = cap ? key_weights_tile_kernel<T, true, true> : key_weights_tile_kernel<T, true, false>;
  else
    kern = cap ? key_weights_tile_kernel<T, false, true> : key_weights_tile_kernel<T, false, false>;
  cudaError_t e = ensure_smem_limit(kern, kTileSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * share));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(share);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = share > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a, tq, share);
}

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

pkv_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return PKV_OK;
  cudaGetLastError();
  return e == cudaErrorInvalidValue ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_add_key_weights(const pkv_params* p, int batch, int64_t total_q, int64_t num_pages,
                                          int64_t kv_pages, const int32_t* qo_indptr_d, const int32_t* kv_indptr_d,
                                          const int32_t* kv_indices_d, const int32_t* kv_last_page_len_d,
                                          const int32_t* weighed_len_d, const void* q, const void* kv,
                                          const uint8_t* kv8_scales, const float* lse, float* weights, float decay,
                                          int32_t* error_d, void* stream) {
  using namespace pkv;
  if (!p || batch < 0 || total_q < 0 || num_pages < 0 || kv_pages < 0) return PKV_ERR_INVALID_ARG;
  if (p->num_qo_heads <= 0 || p->num_kv_heads <= 0 || p->num_qo_heads % p->num_kv_heads) return PKV_ERR_INVALID_ARG;
  if (!(p->sm_scale > 0.f) || !(decay >= 0.f) || !(decay <= 1.f)) return PKV_ERR_INVALID_ARG;
  if (p->page_size <= 0 || (p->page_size > 16 && p->page_size % 16)) return PKV_ERR_UNSUPPORTED;
  if (p->dtype != PKV_F16 && p->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  const int g = p->num_qo_heads / p->num_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8) return PKV_ERR_UNSUPPORTED;
  if (p->num_qo_heads > (1 << 20) || p->page_size > (1 << 20)) return PKV_ERR_UNSUPPORTED;
  if (total_q > (INT32_MAX - 256) / 8 || num_pages > INT32_MAX || kv_pages > INT32_MAX) return PKV_ERR_INVALID_ARG;
  if (!qo_indptr_d && total_q != batch) return PKV_ERR_INVALID_ARG;
  if (batch == 0 || kv_pages == 0) return PKV_OK;  // no keys
  if (!kv_indptr_d || !kv_indices_d || !kv_last_page_len_d || !kv || !weights) return PKV_ERR_INVALID_ARG;
  if (total_q > 0 && (!q || !lse)) return PKV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(lse, 4) || !aligned(weights, 4) || !aligned(qo_indptr_d, 4) ||
      !aligned(kv_indptr_d, 4) || !aligned(kv_indices_d, 4) || !aligned(kv_last_page_len_d, 4) ||
      !aligned(weighed_len_d, 4) || !aligned(error_d, 4))
    return PKV_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  const bool cap = p->logits_cap > 0.f;
  WeightArgs a{};
  a.q = q;
  a.kv = kv;
  a.scales = kv8_scales;
  a.lse = lse;
  a.weights = weights;
  a.qo_indptr = qo_indptr_d;
  a.kv_indptr = kv_indptr_d;
  a.kv_indices = kv_indices_d;
  a.kv_last = kv_last_page_len_d;
  a.weighed = weighed_len_d;
  a.err = error_d;
  a.num_pages = num_pages;
  a.kv_pages = kv_pages;
  a.total_q = total_q;
  a.batch = batch;
  a.hq = p->num_qo_heads;
  a.hkv = p->num_kv_heads;
  a.page_size = p->page_size;
  a.lg = g == 1 ? 0 : g == 2 ? 1 : g == 4 ? 2 : 3;
  a.causal = p->causal != 0 && qo_indptr_d;
  a.scale = cap ? p->sm_scale : p->sm_scale * kLog2e;
  a.cap = cap ? p->logits_cap : 0.f;
  a.decay = decay;
  a.small_div = p->page_size < 16 ? (4096 + p->page_size - 1) / p->page_size : 0;
  auto s = static_cast<cudaStream_t>(stream);
  const int64_t tokens = kv_pages * p->page_size;
  // Many columns per request: the tensor-core tiles.
  const int64_t items = (tokens / kTileKeys + batch) * p->num_kv_heads;
  if (p->head_dim == kD && total_q * g > int64_t{32} * batch && items <= INT32_MAX / 8) {
    // Key tiles too few for the chip are shared by a cluster, as long as each of its CTAs
    // has a column tile.
    int share = 1;
    while (share < 8 && items * share * 2 <= 2 * sms && total_q * g >= int64_t{kTileCols} * batch * share * 2) share *= 2;
    CUtensorMap tq;
    cudaError_t e = prefill_impl::make_rows_map(q, p->dtype, a.hq, total_q, static_cast<int64_t>(a.hq) * kD, g, kTileCols / g, tq);
    if (e == cudaSuccess)
      e = p->dtype == PKV_BF16 ? launch_tile<__nv_bfloat16>(a, cap, items, share, tq, s)
                               : launch_tile<__half>(a, cap, items, share, tq, s);
    return status_of(e);
  }
  const int64_t tiles = (tokens / kStreamKeys + batch) * p->num_kv_heads, ctas = (tiles + 7) / 8;
  const int grid = static_cast<int>(std::min<int64_t>(ctas, 2 * sms));
  cudaError_t e;
  if (p->head_dim == 128)
    e = p->dtype == PKV_BF16 ? launch_stream<128, __nv_bfloat16>(a, cap, grid, s) : launch_stream<128, __half>(a, cap, grid, s);
  else
    e = p->dtype == PKV_BF16 ? launch_stream<64, __nv_bfloat16>(a, cap, grid, s) : launch_stream<64, __half>(a, cap, grid, s);
  return status_of(e);
}
