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
//  - stream: few query rows per request (a decode step).  HBM-bound on K.  Every warp streams
//    keys through its own ring of shared memory by cp.async and multiplies 16 keys at a
//    time with mma.sync m16n8k16, against columns of 8 (row, head) pairs (which dims a k
//    step holds does not matter as long as the query fragments hold the same ones, so a
//    lane's 16-byte chunk of a row serves whole k steps).  Measured: 64 requests of 512 to
//    4096 keys, group 4, 49.3 us, 95 % of measured HBM bandwidth; two of 10^5 in the 8-bit
//    cache, group 8, 48.1 us, 80 % (issue slots: a key row is 128 bytes there).
//  - tile: many rows per request (prompts, or the last rows of one).  S^T = K Q^T on
//    tcgen05: a CTA holds 128 keys of one kv head in tensor memory and streams 64-column
//    tiles of (row, head) pairs past them by TMA; a thread is a key, and sums its
//    exponentials over the columns in registers.  Four CTAs share an SM, so that one's
//    start and waits are another's products.  Many columns before few keys are shared by
//    the CTAs of a cluster, which add their sums in rank order through distributed shared
//    memory.  10 prompts of 128 to 1500 rows, 8 kv heads, group 4, take 64 us: 18064 column
//    tiles, 1100 cycles each on an SM, where the product takes 432, the exponentials 256 and
//    the queries' copies (296 MB) half of what TMA brings from L2.  No unit is the limit;
//    what is left (counted, not timed apart) is what the key warps do around a tile: its lse
//    through shared memory, their barrier, the wait for the one S.  Few columns pay for a key
//    tile's start (tensor memory, page ids, staging): the last 32 to 64 rows of 7 prompts of
//    2000 to 9000 keys, group 2, capped, 40 us.
// The choice between them goes by the batch's average rows, which the host knows: a request
// of many rows among few-row ones is right but slow on the stream kernel, whose warps share
// keys and never columns (63 decode rows over 2000 keys beside a prompt of 400 rows, 8 kv
// heads, group 4: 1290 us in one call, 75 us in two).
// Both find their work from the device's row pointers alone: request b's tiles start at
//     first(b) = floor(kv_indptr[b] P / K) + b        (K keys a tile),
// which leaves each request room for its ceil(len / K) tiles and at most one unused
// place, so no scan over the batch is needed and a captured graph follows the arrays.
// (Prompts take the same places in another order: all first tiles, then all second ones.)
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pkv_join.h"
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
  float scale;               // log2(e) sm_scale
  float scale_lo;            // tile kernel: what `scale` lacks, relative to it
  float cap, decay;
  uint32_t small_div;        // page_size < 16: ceil(4096 / page_size)
  int by_level;              // tile kernel: all requests' first key tiles first
};

// tanh(u) = u + u t h(t), t = u^2, for |u| <= 1: h of degree 6, a least-maximum fit (5.3e-9 of tanh).  A logit
// y within the cap is then y + (y t) h(t): its first term is exact up to one rounding of the sum with
// the lse, the correction is small.  By e^(2u) an error of 2^-23 in the exponential is one of cap 2^-24
// in every logit (at a cap of 30, 2e-6 of a weight; so 6e-7).
constexpr float kTanhIn = 1.f;
__device__ __forceinline__ constexpr float tanh_term(int i) {
  return i == 0 ? -0.33333296f : i == 1 ? 0.13332345f : i == 2 ? -0.0538798f : i == 3 ? 0.021486657f
       : i == 4 ? -0.0079461057f : i == 5 ? 0.002301364f : -0.00035845183f;
}
__device__ __forceinline__ float tanh_correction(float t) {  // t h(t)
  float h = tanh_term(6);
#pragma unroll
  for (int i = 5; i >= 0; --i) h = fmaf(h, t, tanh_term(i));
  return t * h;
}

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

// Records request b if its arrays do not fit.  Every request is looked at by one thread: a tile finds
// its request by a search that takes the row pointers to ascend, and where they do not it may meet
// neither a request that does not fit nor one that does.
__device__ __forceinline__ void check_request(const WeightArgs& a, int b) {
  if (!load_request(a, b).ok) flag(a, kErrAppendLayout);
}

// ---------------------------------------------------------------------------- stream
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

// A warp's ring of tiles of 16 keys (rows of 256 bytes) or 32 (shorter ones: what goes with a
// tile, its page ids and addresses, is as many instructions for 16 keys of the 8-bit cache as
// their products).  Behind a tile's rows: the keys' weights before the call, the rows of the
// weights they go to (kNoRow: none) and, for the 8-bit cache, the aligned word around each
// exponent byte and the byte's place in it.  Two 10^5-token contexts of the 8-bit cache: 16
// keys a tile 54 us; 32 keys with 16 warps of 3 tiles 69 us (128 registers do not hold two
// products' fragments), with 8 of 6 58 us, with 12 of 4 48 us.
template <int D, bool KV8>
struct StreamShape {
  static constexpr int kRow = D * (KV8 ? 1 : 2);
  static constexpr int kKeys = kRow == 256 ? 16 : 32;
  static constexpr int kTile = kKeys * kRow;
  static constexpr int kStage = kTile + kKeys * (KV8 ? 16 : 8);
  static constexpr int kWarps = kKeys == 16 ? 16 : 12;
  static constexpr int kStages = kKeys == 16 ? 3 : kTile == 4096 ? 4 : 6;
  static constexpr int kSmem = kWarps * kStages * kStage;
  static_assert(kSmem <= 232448 - 1024, "stream rings exceed shared memory");
};
constexpr uint32_t kNoRow = 0xffffffffu;

// Byte offset of 16-byte chunk c of row r inside a tile: a fragment load reads 2 rows x 4
// chunks at a time, in different banks.
template <int ROW>
__device__ __forceinline__ uint32_t key_off(int r, int c) {
  return r * ROW + ((ROW >= 128 ? c ^ ((r & 1) << 2) : c) << 4);
}

__device__ __forceinline__ void cp_async_16_hint(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes),
               "l"(policy)
               : "memory");
}
// Four bytes, both addresses 4-byte aligned; bytes past src_bytes are filled with zeros.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// MULTI: more than 8 columns a request on average.  Two tiles' fragments stay in registers
// while the columns pass by (from L1), 8 at a time; without it the first 8 columns stay.
template <int D, typename T, bool KV8, bool MULTI>
__global__ void __launch_bounds__(StreamShape<D, KV8>::kWarps * 32, 1) key_weights_stream_kernel(const __grid_constant__ WeightArgs a) {
  using S = StreamShape<D, KV8>;
  using O = std::conditional_t<KV8, __half, T>;  // operands: e4m3 codes are exact in fp16
  constexpr int KS = D / 16;                     // k steps
  constexpr int CH = S::kRow / 64;               // 16-byte chunks of a row per lane
  constexpr int K = S::kKeys;
  constexpr int SPS = MULTI && K == 16 ? 2 : 1;  // tiles of the ring a step
  constexpr int NS = K / 16, NT = SPS * NS;      // products of 16 keys: of a tile, of a step
  constexpr int CPR = S::kRow / 16, RPI = 32 / CPR;  // chunks per row, rows per copy instruction
  extern __shared__ __align__(128) uint8_t smem[];
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * (S::kStages * S::kStage);
  const int P = a.page_size;
  const bool whole = P % 16 == 0;  // 16 keys lie in one page
  const bool cap = a.cap > 0.f;
  const float cap_out = a.cap * kLog2e, cap_in = cap ? a.scale / cap_out : 0.f;
  const uint32_t vdist = static_cast<uint32_t>(a.hkv) * P;  // rows from a K row to its V row
  const uint8_t* kv = static_cast<const uint8_t*>(a.kv);
  const uint64_t policy = l2_policy_evict_first();
  const int64_t worker = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  const int64_t workers = static_cast<int64_t>(gridDim.x) * S::kWarps;
  const int64_t listed = min(max(static_cast<int64_t>(__ldg(a.kv_indptr + a.batch)), int64_t{0}), a.kv_pages);
  const int64_t U = listed * P / K + a.batch;  // places of tiles per kv head
  const int64_t run = (U * a.hkv + workers - 1) / workers;
  for (int64_t r = (workers - 1 - worker) * 32 + lane; r < a.batch; r += workers * 32)  // (the last workers have the least to do)
    check_request(a, static_cast<int>(r));
  int64_t f = worker * run;
  const int64_t f_end = min(f + run, U * a.hkv);
  while (f < f_end) {
    const int h = static_cast<int>(f / U);
    const int64_t base = h * U, u = f - base;
    const int b = find_request<K>(a, u, lane);
    const Request rq = load_request(a, b);
    const int64_t c0 = first_tile<K>(a, b), c1 = b + 1 < a.batch ? first_tile<K>(a, b + 1) : U;
    const int64_t stop = min(f_end, base + max(c1, u + 1));
    f = stop;
    if (!rq.ok) continue;
    const int n_tiles = (rq.kv_len - 1 + K) / K;
    const int t_end = static_cast<int>(min(static_cast<int64_t>(n_tiles), stop - base - c0));
    const int t_begin = static_cast<int>(max(u - c0, int64_t{0}));
    if (t_begin >= t_end) continue;

    // The copy side.  Lane i (of 16, or of 32) looks after key i of a tile: its page id is fetched a
    // tile ahead, its row counted over the pool's rows.
    int feed = t_begin, stage_in = 0;
    int pg = static_cast<int>(static_cast<int64_t>(t_begin) * K / P);
    int slot = t_begin * K - pg * P;
    int id, my_slot;
    auto fetch_id = [&] {
      const bool in = lane < K && feed < t_end && feed * K + lane < rq.kv_len;
      int skip = 0, x = slot + lane;
      if (!whole)
        skip = static_cast<int>((static_cast<uint32_t>(x) * a.small_div) >> 12);
      else if (x >= P)  // the second 16 keys' page
        skip = 1;
      id = in ? __ldg(a.kv_indices + rq.page0 + pg + skip) : -1;
      my_slot = in ? x - skip * P : -1;
      slot += K;
      if (whole) {
        while (slot >= P) {
          slot -= P;
          ++pg;
        }
      } else {
        const int full = static_cast<int>((static_cast<uint32_t>(slot) * a.small_div) >> 12);
        pg += full;
        slot -= full * P;
      }
    };
    // Start the next tile's copies as one cp.async group (an empty one past the last tile).
    auto issue = [&] {
      if (feed < t_end) {
        const uint32_t dst = ring + stage_in * S::kStage;
        stage_in = stage_in + 1 == S::kStages ? 0 : stage_in + 1;
        const bool use = id >= 0 && id < a.num_pages;
        if (!use && my_slot >= 0) flag(a, kErrPageIndex);
        const uint32_t row = use ? (static_cast<uint32_t>(id) * 2u * a.hkv + h) * P + my_slot : kNoRow;
        if (whole) {
          // 16 rows are contiguous: chunk it * 32 + lane.
          const int left = rq.kv_len - feed * K;
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            const uint32_t first = __shfl_sync(kFullMask, row, 16 * n);
            const int valid = first == kNoRow ? 0 : left - 16 * n;
            const uint8_t* src = kv + static_cast<uint64_t>(first == kNoRow ? 0u : first) * S::kRow + lane * 16;
#pragma unroll
            for (int it = 0; it < 16 / RPI; ++it) {
              const int r = it * RPI + lane / CPR;
              cp_async_16_hint(dst + key_off<S::kRow>(16 * n + r, lane % CPR), r < valid ? src + it * 512 : kv,
                               r < valid ? 16u : 0u, policy);
            }
          }
        } else {
#pragma unroll
          for (int it = 0; it < K / RPI; ++it) {
            const int r = it * RPI + lane / CPR;
            const uint32_t at = __shfl_sync(kFullMask, row, r);
            const uint8_t* src = kv + static_cast<uint64_t>(at == kNoRow ? 0u : at) * S::kRow + (lane % CPR) * 16;
            cp_async_16_hint(dst + key_off<S::kRow>(r, lane % CPR), src, at == kNoRow ? 0u : 16u, policy);
          }
        }
        if (lane < K) {
          const uint32_t at = dst + S::kTile + lane * 4;
          const uint32_t w_row = use ? row - static_cast<uint32_t>(id) * vdist : kNoRow;
          const bool before = use && a.decay != 0.f && feed * K + lane < rq.weighed;
          cp_async_4(at, before ? a.weights + w_row : a.weights, before ? 4u : 0u);
          sts32(at + 4 * K, w_row);
          if constexpr (KV8) {
            const uint32_t byte = use ? row : 0u, word = byte & ~3u;
            const uint64_t rest = static_cast<uint64_t>(a.num_pages) * 2 * vdist - word;  // bytes of the pool from this word on
            cp_async_4(at + 8 * K, a.scales + word, use ? static_cast<uint32_t>(rest < 4 ? rest : 4) : 0u);
            sts32(at + 12 * K, (byte - word) * 8);
          }
        }
        ++feed;
        fetch_id();
      }
      cp_async_commit();
    };
    fetch_id();
#pragma unroll 1
    for (int i = 0; i < S::kStages - 1; ++i) issue();

    const int cols = rq.rows << a.lg;
    const int off = rq.kv_len - rq.rows;  // causal: row i sees keys up to i + off
    // Columns first .. first + 7: lane (g, t) loads chunk(s) t, t + 4, ... of column first + g, and
    // the negated lse of columns first + 2 t and first + 2 t + 1.
    uint32_t qf[KS][2];
    float qs[2] = {1.f, 1.f}, nl[2];
    int see[2];  // the last key that the column's row sees; -1: the column adds nothing
    auto load_columns = [&](int first) {
      const int c = first + g;
      const bool use = c < cols;
      const T* row = static_cast<const T*>(a.q) +
                     (static_cast<int64_t>(rq.row0 + (use ? c >> a.lg : 0)) * a.hq + (h << a.lg) + (use ? c & ((1 << a.lg) - 1) : 0)) * D;
      if constexpr (!KV8) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const uint4 v = use ? ld_nc_v4(row + (t + 4 * i) * 8) : make_uint4(0u, 0u, 0u, 0u);
          qf[2 * i][0] = v.x;
          qf[2 * i][1] = v.y;
          qf[2 * i + 1][0] = v.z;
          qf[2 * i + 1][1] = v.w;
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
        const int cc = first + 2 * t + k, i = cc >> a.lg;
        float l = -INFINITY;
        if (cc < cols) l = __ldg(a.lse + static_cast<int64_t>(rq.row0 + i) * a.hq + (h << a.lg) + (cc & ((1 << a.lg) - 1)));
        nl[k] = -l * kLog2e;
        see[k] = l == -INFINITY ? -1 : a.causal ? i + off : INT_MAX;
      }
    };
    load_columns(0);

    int stage_out = 0;
    for (int tile = t_begin; tile < t_end; tile += SPS) {
      // Of the kStages - 1 groups ahead the first SPS must have landed.
      cp_async_wait<S::kStages - 1 - SPS>();
      __syncwarp();
      uint32_t fr[NT][KS][4];  // A fragments: keys g and g + 8
      float ksc[NT][2], sum[NT][2];
      uint32_t meta[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t at = ring + stage_out * S::kStage;
        if (n % NS == NS - 1) stage_out = stage_out + 1 == S::kStages ? 0 : stage_out + 1;
        const int r0 = 16 * (n % NS);  // first row of the 16
        meta[n] = at + S::kTile + r0 * 4;
        sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const uint4 v = lds128(at + key_off<S::kRow>(r0 + g, t + 4 * i)), z = lds128(at + key_off<S::kRow>(r0 + g + 8, t + 4 * i));
          if constexpr (KV8) {
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              e4m3x4_to_half(vw[w], fr[n][4 * i + w][0], fr[n][4 * i + w][2]);
              e4m3x4_to_half(zw[w], fr[n][4 * i + w][1], fr[n][4 * i + w][3]);
            }
          } else {
            fr[n][2 * i][0] = v.x; fr[n][2 * i][2] = v.y;
            fr[n][2 * i + 1][0] = v.z; fr[n][2 * i + 1][2] = v.w;
            fr[n][2 * i][1] = z.x; fr[n][2 * i][3] = z.y;
            fr[n][2 * i + 1][1] = z.z; fr[n][2 * i + 1][3] = z.w;
          }
        }
        if constexpr (KV8) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t k = (g + 8 * r) * 4;
            ksc[n][r] = __uint_as_float(((lds32(meta[n] + 8 * K + k) >> lds32(meta[n] + 12 * K + k)) & 255u) << 23);
          }
        }
      }
      for (int first = 0;;) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < KS; i += 2) {
            mma_16x8x16<O>(sa, fr[n][i][0], fr[n][i][1], fr[n][i][2], fr[n][i][3], qf[i][0], qf[i][1]);
            mma_16x8x16<O>(sb, fr[n][i + 1][0], fr[n][i + 1][1], fr[n][i + 1][2], fr[n][i + 1][3], qf[i + 1][0], qf[i + 1][1]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // key g + 8 (k / 2) of the tile, column 2 t + k % 2
            const int c = k & 1, r = k >> 1, j = tile * K + 16 * n + g + 8 * r;
            float s = sa[k] + sb[k];
            if constexpr (KV8) s *= qs[c] * ksc[n][r];
            float y = fmaf(s, a.scale, nl[c]);
            if (cap) {
              const float u = s * cap_in;
              y = fabsf(u) <= kTanhIn ? fmaf(s * a.scale, tanh_correction(u * u), y)
                                      : fmaf(cap_out, tanh_from_log2(u * (2.f * kLog2e)), nl[c]);
            }
            const float p = fast_exp2(y);
            sum[n][r] += j > see[c] ? 0.f : p;
          }
        }
        first += 8;
        if (first >= cols) break;
        load_columns(first);
      }
      if (cols > 8) load_columns(0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sum[n][r] += __shfl_xor_sync(kFullMask, sum[n][r], 1);
          sum[n][r] += __shfl_xor_sync(kFullMask, sum[n][r], 2);
        }
        // Lane t = 0 has key g, t = 1 key g + 8.
        if (t < 2 && tile + n / NS < t_end) {
          const uint32_t k = (g + 8 * t) * 4, w_row = lds32(meta[n] + 4 * K + k);
          if (w_row != kNoRow) a.weights[w_row] = fmaf(__uint_as_float(lds32(meta[n] + k)), a.decay, t ? sum[n][1] : sum[n][0]);
        }
      }
      __syncwarp();  // every lane has read the stages before they are filled again
#pragma unroll 1
      for (int n = 0; n < SPS; ++n) issue();
    }
    cp_async_wait<0>();
    __syncwarp();
  }
}

// ------------------------------------------------------------------------------ tile
constexpr int kD = prefill_impl::kD;
constexpr int kTileKeys = 128;
constexpr int kLevelBatch = 128;              // requests whose key tiles may be taken longest first
constexpr int kTileCols = 64;                 // (row, head) pairs of one product
constexpr int kQStages = 3;                   // the last two bring the keys first
constexpr uint32_t kQHalf = kTileCols * 128;  // 64 of the 128 dims of 64 columns
constexpr uint32_t kQTile = 2 * kQHalf;
constexpr int kTileThreads = 192;             // four warps of keys, the Q producer, the MMA issuer
constexpr int kTileCtas = 4;                  // per SM
constexpr int kTileSmem = kQStages * kQTile + 1024;
constexpr uint32_t kWTmemCols = 128;          // K 64, S^T 64
constexpr uint32_t kColSt = 64;

struct TileShared {
  uint64_t q_full[kQStages], q_empty[kQStages], s_full, s_empty, k_full, drain;
  alignas(16) float nl[2][kTileCols];  // read as float4; negated lse in log2 units, -inf for a column that adds nothing
  float sum[kTileKeys];
  uint32_t tmem;
  int abort;
};

// All 128 threads with keys arrive; true where any of them brought true.
__device__ __forceinline__ bool keys_any(bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(x))
      : "memory");
  return r != 0;
}

// The u-th key tile in the order of their places in their requests (all first tiles, then all
// second ones, ...): under a causal mask the first tiles have the most columns, so the longest
// work starts first.  By the whole warp; false past the last tile.
__device__ __forceinline__ bool tile_by_level(const WeightArgs& a, int64_t u, int lane, int& b, int64_t& tile) {
  auto tiles_of = [&](int r) -> int {
    if (r >= a.batch) return 0;
    const Request q = load_request(a, r);
    return q.ok ? (q.kv_len + kTileKeys - 1) / kTileKeys : 0;
  };
  // Tiles of the first kOwn * 32 requests stay in registers: lane l has requests l, l + 32, ...
  constexpr int kOwn = kLevelBatch / 32;
  int mine[kOwn], most = 0;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    mine[k] = k * 32 < a.batch ? tiles_of(k * 32 + lane) : 0;
    most = max(most, mine[k]);
  }
  most = __reduce_max_sync(kFullMask, most);
  auto below = [&](int level) {  // tiles of levels before `level`
    int64_t sum = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      if (k * 32 < a.batch) sum += static_cast<uint32_t>(__reduce_add_sync(kFullMask, static_cast<uint32_t>(min(mine[k], level))));
    return sum;
  };
  if (u >= below(most)) return false;
  int lo = 0, hi = most;  // below(lo) <= u < below(hi)
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (below(mid) <= u) lo = mid; else hi = mid;
  }
  int left = static_cast<int>(u - below(lo));  // the left-th request that has a tile `lo`
  tile = lo;
  b = 0;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const unsigned at = __ballot_sync(kFullMask, mine[k] > lo);
    const int c = __popc(at);
    if (left >= 0 && left < c) b = k * 32 + __fns(at, 0, left + 1);
    left -= c;
    if (left < 0) left = INT_MIN / 2;
  }
  return true;
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
__global__ void __launch_bounds__(kTileThreads, kTileCtas)
    key_weights_tile_kernel(const __grid_constant__ WeightArgs a, const __grid_constant__ CUtensorMap tq, int share) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ TileShared sh;
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = a.page_size;
  const int rank = share > 1 ? static_cast<int>(cluster_rank()) : 0;
  // This cluster's key tile: kv heads of a tile side by side.
  const int64_t item = blockIdx.x / share;
  const int64_t u = item / a.hkv;
  const int h = static_cast<int>(item - u * a.hkv);
  int b = 0;
  int64_t tile = 0;
  const uint32_t back = gridDim.x - 1 - blockIdx.x;  // the last CTAs have the least to do; there is one a request at least
  if (back <= static_cast<uint32_t>(a.batch) / kTileThreads && back * kTileThreads + tid < static_cast<uint32_t>(a.batch))
    check_request(a, back * kTileThreads + tid);
  if (a.by_level) {
    if (!tile_by_level(a, u, lane, b, tile)) return;  // the same for all CTAs of a cluster
  } else {
    b = find_request<kTileKeys>(a, u, lane);
    tile = u - first_tile<kTileKeys>(a, b);
  }
  const Request rq = load_request(a, b);
  if (!rq.ok || tile < 0 || tile * kTileKeys >= rq.kv_len) return;  // the same for all CTAs of a cluster
  const int k0 = static_cast<int>(tile) * kTileKeys;
  const int off = rq.kv_len - rq.rows;
  const int row_first = a.causal ? min(max(k0 - off, 0), rq.rows) : 0;  // the first row that sees key k0
  const int per = kTileCols >> a.lg;                                    // rows of a column tile
  const int n_all = (rq.rows - row_first + per - 1) / per;
  const int n = n_all > rank ? (n_all - 1 - rank) / share + 1 : 0;      // column tiles rank, rank + share, ...

  uint32_t base = smem_addr(smem_raw);
  base = (base + 1023u) & ~1023u;
  auto bar = [](uint64_t& x) { return smem_addr(&x); };
  if (tid == 0) {
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(bar(sh.q_full[i]), 1);
      mbar_init(bar(sh.q_empty[i]), 1);
    }
    mbar_init(bar(sh.s_full), 1);
    mbar_init(bar(sh.s_empty), 128);
    mbar_init(bar(sh.k_full), 128);
    mbar_init(bar(sh.drain), 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
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

  float old = 0.f, total = 0.f;
  float* at = nullptr;
  if (warp == 4) {
    // ------------------------------------------------------------ Q producer
    if (elect_one()) {
      int i = 0;
      for (; i < n; ++i) {
        const int s = i % kQStages;
        if (i == 1 && !wait(sh.k_full, 0)) break;  // the keys have left the room of stages 1 and 2
        if (i >= kQStages && !wait(sh.q_empty[s], (i / kQStages - 1) & 1)) break;
        mbar_arrive_expect_tx(bar(sh.q_full[s]), kQTile);
        const int row = rq.row0 + row_first + (rank + i * share) * per;
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
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      const uint32_t idesc = umma_idesc_f16(kFmt, kTileKeys, kTileCols, 0);
      const uint64_t dq = sw128_desc(base, 16, 1024);
      const uint32_t hi = static_cast<uint32_t>(dq >> 32), q_lo = static_cast<uint32_t>(dq);
      bool ok = n == 0 || wait(sh.k_full, 0);
      tc_fence_after();
      for (int i = 0; i < n && ok; ++i) {
        const int s = i % kQStages;
        if (!(ok = wait(sh.q_full[s], (i / kQStages) & 1))) break;
        if (i > 0 && !(ok = wait(sh.s_empty, (i - 1) & 1))) break;
        tc_fence_after();
        const uint32_t dst = tmem + kColSt, b0 = q_lo + s * (kQTile >> 4);
        prefill_impl::umma_ts_lo<false>(dst, tmem, b0, hi, idesc);
#pragma unroll
        for (int kk = 1; kk < kD / 16; ++kk)
          prefill_impl::umma_ts_lo<true>(dst, tmem + kk * 8, b0 + (kk / 4) * (kQHalf >> 4) + (kk % 4) * 2, hi, idesc);
        umma_commit(bar(sh.s_full));
        umma_commit(bar(sh.q_empty[s]));
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
    const int j = k0 + tid;  // this thread's key: its lane of tensor memory
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    uint32_t row = kNoRow;
    float mul = a.scale;
    if (j < rq.kv_len) {
      const int pg = j / P, page = __ldg(a.kv_indices + rq.page0 + pg);
      if (page >= 0 && page < a.num_pages) {
        row = (static_cast<uint32_t>(page) * 2u * a.hkv + h) * P + (j - pg * P);
        if (rank == 0) {
          at = a.weights + (static_cast<int64_t>(page) * a.hkv + h) * P + (j - pg * P);
          if (a.decay != 0.f && j < rq.weighed) old = *at * a.decay;
        }
      } else {
        flag(a, kErrPageIndex);
      }
    }
    __syncwarp();
    // The key's values, two to a column: the A operand.  A warp brings its 32 rows, whole
    // segments a copy, through the later Q stages' room; then a lane reads its own row.
    {
      constexpr int kRow = KV8 ? kD : 2 * kD, kCpr = kRow / 16, kRpi = 32 / kCpr;
      const uint32_t room = base + kQTile + warp * 32 * kRow;
      const uint8_t* kv = static_cast<const uint8_t*>(a.kv) + (lane % kCpr) * 16;
#pragma unroll
      for (int it = 0; it < 32 / kRpi; ++it) {
        const int r = it * kRpi + lane / kCpr;
        const uint32_t from = __shfl_sync(kFullMask, row, r);
        cp_async_16(room + r * kRow + (((lane % kCpr) ^ (r & 7)) << 4), kv + static_cast<uint64_t>(from == kNoRow ? 0u : from) * kRow,
                    from == kNoRow ? 0u : 16u);
      }
      cp_async_commit();
      if constexpr (KV8) mul *= __uint_as_float(static_cast<uint32_t>(row != kNoRow ? __ldg(a.scales + row) : 0) << 23);
      cp_async_wait<0>();
      __syncwarp();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < kCpr / 2; ++i) {
          const uint4 v = lds128(room + lane * kRow + (((x * (kCpr / 2) + i) ^ (lane & 7)) << 4));
          if constexpr (KV8) {
            e4m3x4_to<T>(v.x, w[8 * i], w[8 * i + 1]);
            e4m3x4_to<T>(v.y, w[8 * i + 2], w[8 * i + 3]);
            e4m3x4_to<T>(v.z, w[8 * i + 4], w[8 * i + 5]);
            e4m3x4_to<T>(v.w, w[8 * i + 6], w[8 * i + 7]);
          } else {
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
          }
        }
        tmem_st32(tmem + lane_off + x * 32, w);
      }
      fence_proxy_async_smem();  // the room is the Q copies' from here on
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(bar(sh.k_full));
    // Column tid (< 64) of column tile i: its negated lse, -inf where it adds nothing.
    auto load_nl = [&](int i) {
      float v = -INFINITY;
      if (i < n && tid < kTileCols) {
        const int q_row = row_first + (rank + i * share) * per + (tid >> a.lg);
        if (q_row < rq.rows) {
          const float l =
              __ldg(a.lse + static_cast<int64_t>(rq.row0 + q_row) * a.hq + (h << a.lg) + (tid & ((1 << a.lg) - 1)));
          v = l == -INFINITY ? -INFINITY : -l * kLog2e;
        }
      }
      return v;
    };
    float2 all = make_float2(0.f, 0.f);  // of the halves' sums, so that an error grows with the root of their number
    float next_nl = load_nl(0);
    float u_in = 0.f, k_out = 0.f;  // the cap's argument is u_in times the product
    if constexpr (CAP) {
      k_out = a.cap * kLog2e;
      u_in = mul / k_out;
    }
    bool ok = true;
    for (int i = 0; i < n; ++i) {  // every warp meets the barrier n times, come what may
      float* nl = sh.nl[i & 1];
      if (tid < kTileCols) nl[tid] = next_nl;
      const bool some_out = keys_any(tid < kTileCols && next_nl == -INFINITY);
      next_nl = load_nl(i + 1);
      if (ok) ok = __all_sync(kFullMask, wait(sh.s_full, i & 1));
      if (!ok) continue;
      tc_fence_after();
      const int q_row = row_first + (rank + i * share) * per;
      const int cols = min((rq.rows - q_row) << a.lg, kTileCols);  // (no overflow: at most 64 are asked for)
      // The first column whose row sees this key.
      const int c_min = a.causal ? max(j - off - q_row, 0) << a.lg : 0;
      const bool masked = some_out || (a.causal && k0 + kTileKeys - 1 - off > q_row);
      const float2 mul2 = make_float2(mul, mul), mul_lo2 = make_float2(mul * a.scale_lo, mul * a.scale_lo);
#pragma unroll(CAP ? 1 : 2)
      for (int half = 0; half < 2; ++half) {
        uint32_t sr[32];
        const bool any = half * 32 < cols;
        if (any) tmem_ld32_sync(tmem + lane_off + kColSt + half * 32, sr);
        if (half == 1) {  // S^T is free for the next column tile
          tc_fence_before();
          mbar_arrive(bar(sh.s_empty));
        }
        if (!any) break;
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // CAP: kSmall, every argument of the warp's 32 columns is within [-1, 1].
        auto add = [&](auto masked_c, auto small_c) {
          constexpr bool kMasked = decltype(masked_c)::value, kSmall = decltype(small_c)::value;
          const int c_from = c_min - half * 32;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(nl + half * 32 + c);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 s = make_float2(__uint_as_float(sr[c + 2 * e]), __uint_as_float(sr[c + 2 * e + 1]));
              const float2 l = e ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
              // Which of the two do not count (always known to be false without kMasked).
              const bool out0 = kMasked && (c + 2 * e < c_from || l.x == -INFINITY);
              const bool out1 = kMasked && (c + 2 * e + 1 < c_from || l.y == -INFINITY);
              float2 y;
              if constexpr (CAP && kSmall) {
                auto two = [](float x) { return make_float2(x, x); };
                float2 t = fmul2(s, two(u_in));
                t = fmul2(t, t);
                float2 f = two(tanh_term(6));
#pragma unroll
                for (int i = 5; i >= 0; --i) f = ffma2(f, t, two(tanh_term(i)));
                y = ffma2(fmul2(s, mul2), ffma2(f, t, two(a.scale_lo)), ffma2(s, mul2, l));
              } else if constexpr (CAP) {
                // cap tanh(u) = k_out - 2 k_out / (e^(2u) + 1), with one reciprocal for both:
                // 1 / a = b (1 / ab).  2^60 is infinity here, so that ab stays finite; NaN stays
                // NaN, and one that does not count is kept from the other.
                float2 z = fmul2(s, make_float2(u_in * (2.f * kLog2e), u_in * (2.f * kLog2e)));
                z.x = out0 ? 0.f : min_nan(z.x, 60.f);
                z.y = out1 ? 0.f : min_nan(z.y, 60.f);
                z = fadd2(make_float2(fast_exp2(z.x), fast_exp2(z.y)), make_float2(1.f, 1.f));
                const float r = fast_rcp(z.x * z.y);
                z = fmul2(make_float2(z.y, z.x), make_float2(r, r));
                y = fadd2(ffma2(z, make_float2(-2.f * k_out, -2.f * k_out), make_float2(k_out, k_out)), l);
              } else {
                y = ffma2(s, mul_lo2, ffma2(s, mul2, l));
              }
              const float p0 = fast_exp2(y.x), p1 = fast_exp2(y.y);
              acc[e] = fadd2(acc[e], make_float2(out0 ? 0.f : p0, out1 ? 0.f : p1));
            }
          }
        };
        bool small = true;
        if constexpr (CAP) {
          float most = 0.f;  // (NaN gives NaN by either formula)
#pragma unroll
          for (int c = 0; c < 32; ++c) most = fmaxf(most, fabsf(__uint_as_float(sr[c])));
          small = __all_sync(kFullMask, most * u_in <= kTanhIn);
        }
        if (!small)
          add(std::true_type{}, std::false_type{});
        else if (masked)
          add(std::true_type{}, std::true_type{});
        else
          add(std::false_type{}, std::true_type{});
        all = fadd2(all, fadd2(acc[0], acc[1]));
      }
    }
    total = all.x + all.y;
    sh.sum[tid] = total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kWTmemCols);
  // Where a wait ran out on any of the tile's CTAs its weights stay as they were.
  if (share > 1) {
    cluster_sync_all();
    if (at && !join_ranks(share, [&](int k) { return __uint_as_float(ld_cluster_u32(&sh.sum[tid], k)); },
                          [&](int k) { return ld_cluster_u32(&sh.abort, k) != 0u; }, total))
      at = nullptr;      // (rank 0's keys)
    cluster_sync_all();  // a CTA's sums stay until they have been read
  } else if (sh.abort) {
    at = nullptr;
  }
  if (at) *at = old + total;
}

template <int D, typename T>
cudaError_t launch_stream(const WeightArgs& a, bool multi, int grid, cudaStream_t s) {
  void (*kern)(WeightArgs) = nullptr;
  if (a.scales)
    kern = multi ? key_weights_stream_kernel<D, T, true, true> : key_weights_stream_kernel<D, T, true, false>;
  else
    kern = multi ? key_weights_stream_kernel<D, T, false, true> : key_weights_stream_kernel<D, T, false, false>;
  const int smem = a.scales ? StreamShape<D, true>::kSmem : StreamShape<D, false>::kSmem;
  const int warps = a.scales ? StreamShape<D, true>::kWarps : StreamShape<D, false>::kWarps;
  cudaError_t e = ensure_smem_limit(kern, smem);
  return e == cudaSuccess ? launch_dependent(kern, grid, warps * 32, smem, s, a) : e;
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
  // Rows of the pool are counted in 32 bits, with the last value for none.
  if (static_cast<double>(num_pages) * 2 * p->num_kv_heads * p->page_size >= 4294967295.0) return PKV_ERR_UNSUPPORTED;
  if (!aligned(kv8_scales, 4)) return PKV_ERR_INVALID_ARG;  // exponent bytes are copied in fours
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
  // The tensor core cuts its partial sums off: of 400000 products over 128 dims, those within one standard
  // deviation of 0 were 0.7e-7 of themselves nearer to 0 than the exact ones, those past three 1.4e-7.  The tile
  // kernel adds 1e-7, and what the rounding of the scale took, by a second product (3 us of 65 on 10 prompts of
  // 128 to 1500 rows).  What it brings and costs, as errors of the weights: prompts over keys of unlike sizes
  // (logits to 20) 1.7e-7, without it 1.3e-6; sums that lose nothing (one nonzero element a row), where it is the
  // error itself, 1.6e-6 at logits to 22 and 6.5e-6 at 90, without it 1e-7 and 3e-7.  Rows of queries and keys are
  // dense, so the first counts, and the second is two roundings of the logit in fp32 (2^-24 each).  The branch for
  // arguments past the cap's polynomial and the stream kernel do without.
  const double scale = static_cast<double>(p->sm_scale) * 1.4426950408889634;
  a.scale = static_cast<float>(scale);
  a.scale_lo = static_cast<float>(scale / a.scale * (1 + 1e-7) - 1);
  a.cap = cap ? p->logits_cap : 0.f;
  a.decay = decay;
  a.small_div = p->page_size < 16 ? (4096 + p->page_size - 1) / p->page_size : 0;
  auto s = static_cast<cudaStream_t>(stream);
  const int64_t tokens = kv_pages * p->page_size;
  // Many columns per request: the tensor-core tiles.
  const int64_t places = tokens / kTileKeys + batch, items = places * p->num_kv_heads;
  if (p->head_dim == kD && total_q * g > int64_t{32} * batch && items <= INT32_MAX / 8) {
    // Causal prompts' key tiles differ in their columns, up to all of a request's for the first
    // one: clusters share the columns of a tile until there are six CTAs an SM, as long as each
    // has eight column tiles of a request of average length.  (Prompts of 128 to 1500 rows, 8 kv
    // heads, before the second product below: alone 92 us, two CTAs a tile 62 us, four 75 us.)
    int share = 1;
    while (share < 8 && items * share < 6 * sms && total_q * g >= int64_t{16 * kTileCols} * batch * share) share *= 2;
    // A causal call whose rows are most of its keys: a request's first key tile has columns of
    // all its rows, its last one of 128 rows.  The longest start first then, or the last CTAs
    // run alone (12 us of those prompts' 74).  Where keys are many
    // times the rows all tiles are alike, and the longer search only costs.
    a.by_level = a.causal && batch <= kLevelBatch && tokens <= 4 * total_q;
    CUtensorMap tq;
    cudaError_t e = prefill_impl::make_rows_map(q, p->dtype, a.hq, total_q, static_cast<int64_t>(a.hq) * kD, g, kTileCols / g, tq);
    if (e == cudaSuccess)
      e = p->dtype == PKV_BF16 ? launch_tile<__nv_bfloat16>(a, cap, items, share, tq, s)
                               : launch_tile<__half>(a, cap, items, share, tq, s);
    return status_of(e);
  }
  const int64_t tiles = (tokens / 16 + batch) * p->num_kv_heads;  // (of 32 keys: half as many)
  const int grid = static_cast<int>(std::min<int64_t>(tiles, sms));
  const bool multi = total_q * g > int64_t{8} * batch;
  cudaError_t e;
  if (p->head_dim == 128)
    e = p->dtype == PKV_BF16 ? launch_stream<128, __nv_bfloat16>(a, multi, grid, s) : launch_stream<128, __half>(a, multi, grid, s);
  else
    e = p->dtype == PKV_BF16 ? launch_stream<64, __nv_bfloat16>(a, multi, grid, s) : launch_stream<64, __half>(a, multi, grid, s);
  return status_of(e);
}
