// decode8.cu -- batch decode over the 8-bit paged KV cache (e4m3 codes with one
// power-of-two scale per head row), split-KV, on the same plan tables as
// decode_kernel.cuh.
//
// Mathematics.  For a query row q of head h, key codes k_j with scale 2^a_j and
// value codes v_j with scale 2^b_j:
//     y_j = (q . k_j) sm_scale log2(e) 2^a_j          (logit, in log2 units)
//     l   = sum_j 2^(y_j - m)                          m: running reference of y
//     O   = sum_j 2^((y_j - m) + b_j - R + 7) v_j      R: running reference of (y - m) + b
//     o   = O 2^(R - 7) / l,   lse = (m + log2 l) ln 2.
// The value's scale joins its probability's exponent, so no value is multiplied by
// it; with a reference of its own, values of any scale keep the probabilities in
// fp16's normal range: they are at most 2^15 (a reference is raised when a term
// passes it by 2^8) and lose bits only 2^-21 below the largest term.  b joins the
// difference y - m, not y, whose last bit may be larger than b.
//
// GB300 design.  The cache's bytes are read once: HBM-bound, two bytes of K and V for
// 4 G flops.  On the CUDA cores a group of 4 would need 27 Tfma/s of the 37 the
// chip has, next to the conversions, so both products run on the tensor cores as
// mma.sync m16n8k16 (fp16 operands, fp32 sums): 16 keys x 8 heads of the group
// (padded), then 16 dims x 8 heads.  Keys and dims are the M axis, so a group of 8
// wastes nothing, and the padding of a smaller one costs no bandwidth.
//  - One CTA per SM holds kDecodeWarps independent warps, each with the plan's
//    list of (request, kv head, page range) segments and a ring of 16-token tiles in
//    shared memory, filled by its own 16-byte cp.async copies kStages - 1 tiles
//    ahead (any page size, zeros past the request: nothing unread is ever in a
//    product).  Chunks are XOR-swizzled so that both fragment reads are free of bank
//    conflicts.
//  - e4m3 becomes fp16 exactly, in registers (cvt of a pair).  K is the A operand of
//    Q K^T: a lane's 32-bit word of a row is one k step (which dims a k step holds
//    does not matter as long as Q's fragments hold the same ones).  V is the A operand
//    of V^T P: two tokens' bytes of the same dim are paired by one byte permute.
//  - The scores leave the first product with the token on the lane's row; a transposing
//    register move (movmatrix) makes them the second product's B operand.
//  - A tile raises the references only when a score passes one by 2^8, so most tiles
//    have no shuffle at all.
#include <cuda_runtime.h>
#include <math.h>

#include "decode_kernel.cuh"

namespace pkv {
namespace {

using decode_impl::kFull;
using decode_impl::load_seg;
using decode_impl::seg_tokens;
using decode_impl::SegInfo;

constexpr int kRows = kDecodeTileRows;  // tokens of a tile

template <int D>
struct Shape8 {
  static constexpr int kTile = kRows * D;               // bytes of K (or V) of one tile
  static constexpr int kStages = D == 128 ? 6 : 12;     // 24 KB of rows in flight per warp
  static constexpr int kScales = 2 * kRows;             // exponent bytes of one tile
  static constexpr int kWarpBytes = kStages * (2 * kTile + kScales);
};

// Byte offset of 16-byte chunk c of row r inside a tile, swizzled within each
// 128-byte line.  K is read 8 rows x 4 chunks at a time, V 4 row pairs x 2 chunks.
template <int D>
__device__ __forceinline__ uint32_t k_off(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
  return r * 64 + (c << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_off(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return (r >> 1) * 128 + (((((r & 1) << 2) + c) ^ (r & 6)) << 4);
}

__device__ __forceinline__ void cp_async_16_hint(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes),
               "l"(policy)
               : "memory");
}

// Four bytes, both addresses 4-byte aligned; src_bytes = 0 fills them with zeros.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Four e4m3 codes to two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose an 8x8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 2^(s - 127) of an exponent byte.
__device__ __forceinline__ float exp_byte(uint32_t s) { return __uint_as_float(s << 23); }

// The copy side of a warp's ring, ahead of the compute side in the same (segment,
// tile) sequence.  `row` is the tile's first slot in page `page` of the segment.
struct Feed {
  int seg, seg_end;
  int tok, n_tok;
  int idx_begin, n_pages, kvh;
  int page, row;
  int win_base, win;   // 32 page ids from entry win_base of the segment, one per lane
  int issued;
  int scale, scale_stage;  // this lane's exponent byte of the tile issued last, and its stage
};

__device__ __forceinline__ void feed_enter(Feed& p, const DecodeArgs& a, int lane) {
  const SegInfo s = load_seg(a.segs, p.seg, lane);
  p.idx_begin = s.idx_begin;
  p.n_pages = s.n_pages;
  p.n_tok = seg_tokens(s.n_pages, s.last_rows, a.page_size);
  p.kvh = s.kvh;
  p.tok = p.page = p.row = p.win_base = 0;
  p.win = lane < s.n_pages ? __ldg(a.kv_indices + p.idx_begin + lane) : 0;
}

// How a tile lies in its pages: kOne, pages of a multiple of 16 rows, so that it lies in
// one; kFours, pages of 4, 8 or 12 rows; kAny, the other sizes below 16.
enum PageMode { kOne, kFours, kAny };

// Issue the next tile's copies as one cp.async group (an empty one when the list has
// ended).  Its exponent bytes are copied in fours (which may take in slots past
// kv_last_page_len: their scores are masked).  Where a page does not hold whole fours
// (kAny) they come as one plain load per lane (K's tokens on lanes 0-15, V's on
// 16-31), put into shared memory at the next call, when they have arrived: the
// compute side reads a tile's bytes two calls later at the earliest.
template <int D, PageMode MODE>
__device__ __forceinline__ void feed_issue(Feed& p, const DecodeArgs& a, const uint8_t* scales, uint32_t rows0,
                                           uint32_t scales0, int lane, int64_t num_pages, uint32_t small_div,
                                           uint64_t policy) {
  using S = Shape8<D>;
  constexpr bool ONE = MODE == kOne;
  constexpr int CPR = D / 16;          // 16-byte chunks per row
  constexpr int RPI = 32 / CPR;        // rows per copy instruction
  if constexpr (MODE == kAny) {
    if (p.scale_stage >= 0) sts8(scales0 + p.scale_stage * S::kScales + lane, p.scale);
    p.scale_stage = -1;
  }
  while (p.seg < p.seg_end && p.tok >= p.n_tok) {
    ++p.seg;
    if (p.seg < p.seg_end) feed_enter(p, a, lane);
  }
  if (p.seg < p.seg_end) {
    const int P = a.page_size;
    const int rows = min(kRows, p.n_tok - p.tok);
    const int stage = p.issued % S::kStages;
    const uint32_t dst = rows0 + stage * 2 * S::kTile;
    const uint8_t* kv = static_cast<const uint8_t*>(a.kv);
    const int64_t vdist = static_cast<int64_t>(a.num_kv_heads) * P;  // rows from a K row to its V row
    const int span = ONE ? 1 : static_cast<int>((static_cast<uint32_t>(p.row + kRows - 1) * small_div) >> 12) + 1;
    if (p.page + span - p.win_base > 32) {
      p.win_base = p.page;
      p.win = p.page + lane < p.n_pages ? __ldg(a.kv_indices + p.idx_begin + p.page + lane) : 0;
    }
    bool bad = false;
    // Row (counted over the pool's (page, head) blocks of K) of row r of the tile, or
    // -1 past the tile's rows or in a page outside the pool.
    auto place = [&](int r) -> int64_t {
      const int x = p.row + r;
      const int k = ONE ? 0 : static_cast<int>((static_cast<uint32_t>(x) * small_div) >> 12);  // x / P
      const int id = __shfl_sync(kFull, p.win, (p.page + k - p.win_base) & 31);
      if (r >= rows) return -1;
      if (id < 0 || id >= num_pages) {
        bad = true;
        return -1;
      }
      return (static_cast<int64_t>(id) * 2 * a.num_kv_heads + p.kvh) * P + (ONE ? x : x - k * P);
    };
#pragma unroll
    for (int it = 0; it < kRows / RPI; ++it) {
      const int r = it * RPI + lane / CPR, c = lane % CPR;
      const int64_t at = place(r);
      const uint8_t* src = kv + (at < 0 ? 0 : at * D) + c * 16;
      const uint32_t n = at < 0 ? 0u : 16u;
      cp_async_16_hint(dst + k_off<D>(r, c), src, n, policy);
      cp_async_16_hint(dst + S::kTile + v_off<D>(r, c), at < 0 ? src : src + vdist * D, n, policy);
    }
    if constexpr (MODE == kAny) {
      const int64_t at = place(lane & 15);
      p.scale = 127;
      if (at >= 0) p.scale = __ldg(scales + at + (lane < 16 ? 0 : vdist));
      p.scale_stage = stage;
    } else {
      const int64_t at = place((lane & 3) * 4);
      if (lane < 8)
        cp_async_4(scales0 + stage * S::kScales + lane * 4, scales + (at < 0 ? 0 : at + (lane < 4 ? 0 : vdist)),
                   at < 0 ? 0u : 4u);
    }
    if (bad) atomicOr(a.err, kErrPageIndex);
    ++p.issued;
    p.tok += rows;
    p.row += kRows;
    if constexpr (ONE) {
      if (p.row == P) {
        p.row = 0;
        ++p.page;
      }
    } else {
      const int k = static_cast<int>((static_cast<uint32_t>(p.row) * small_div) >> 12);
      p.page += k;
      p.row -= k * P;
    }
  }
  cp_async_commit();
}

struct Decode8Args {
  DecodeArgs d;            // kv: the e4m3 codes; q_scale unused
  const uint8_t* scales;
  float sm_scale;
  uint32_t small_div;      // page_size < 16: ceil(4096 / page_size)
};

template <int D, typename T, bool CAP, PageMode MODE>
__device__ __forceinline__ void decode8_worker(const Decode8Args& a8, int worker, uint32_t rows0, uint32_t scales0) {
  using S = Shape8<D>;
  constexpr int ST = S::kStages;
  constexpr int KC = D / 64;     // 16-byte chunks of a K row per lane (and of a 16-bit Q row, pairs of them)
  constexpr int KS = D / 16;     // k steps of Q K^T, and 16-dim blocks of V^T P
  const DecodeArgs& a = a8.d;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const PlanHeader* hdr = a.hdr;
  if (worker >= hdr->num_workers) return;
  const int64_t num_pages = hdr->num_pages;
  const int seg_begin = a.worker_ptr[worker], seg_end = a.worker_ptr[worker + 1];
  if (seg_begin >= seg_end) return;
  const uint64_t policy = l2_policy_evict_first();
  const int G = a.num_qo_heads / a.num_kv_heads;

  Feed feed;
  feed.seg = seg_begin;
  feed.seg_end = seg_end;
  feed.issued = 0;
  feed.scale_stage = -1;
  feed_enter(feed, a, lane);
  auto issue = [&] {
    feed_issue<D, MODE>(feed, a, a8.scales, rows0, scales0, lane, num_pages, a8.small_div, policy);
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue();

  int consumed = 0;
  for (int si = seg_begin; si < seg_end; ++si) {
    const SegInfo sg = load_seg(a.segs, si, lane);
    const int hq0 = sg.kvh * G;
    if (lane == 0 && __ldg(a.kv_indptr + sg.b) != sg.idx_begin - sg.page_begin) atomicOr(a.err, kErrIndptrMismatch);

    // Q fragments: lane (g, t) holds head g's dims of K chunks t (and t + 4), as fp16
    // of q over the power of two below its row's largest element (heads past the
    // group are zero).
    uint32_t qf[KS][2];
    float qs;  // the logits' factor of head g
    {
      uint4 raw[KC][2];
      float mx = 0.f;
      const T* qrow = static_cast<const T*>(a.q) + (static_cast<int64_t>(sg.q_row) * a.num_qo_heads + hq0 + g) * D;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          raw[c][h] = g < G ? ld_nc_v4(qrow + (t + 4 * c) * 16 + h * 8) : make_uint4(0u, 0u, 0u, 0u);
          float f[8];
          to_float8<T>(raw[c][h], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
        }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const uint32_t field = min(max(__float_as_uint(mx) >> 23, 1u), 253u);
      const float mul = __uint_as_float((254u - field) << 23);
      qs = a8.sm_scale * exp_byte(field) * (CAP ? 1.f : kLog2e);
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[8];
          to_float8<T>(raw[c][h], f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qf[c * 4 + h * 2 + e][0] = pack2<__half>(f[4 * e] * mul, f[4 * e + 1] * mul);
            qf[c * 4 + h * 2 + e][1] = pack2<__half>(f[4 * e + 2] * mul, f[4 * e + 3] * mul);
          }
        }
    }
    // From here on a lane's two heads are 2t and 2t + 1.
    const float qs0 = __shfl_sync(kFull, qs, 8 * t), qs1 = __shfl_sync(kFull, qs, 8 * t + 4);
    float m[2] = {-INFINITY, -INFINITY}, R[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float acc[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;

    const int n_tok = seg_tokens(sg.n_pages, sg.last_rows, a.page_size);
    for (int tok0 = 0; tok0 < n_tok; tok0 += kRows) {
      const int rows = min(kRows, n_tok - tok0);
      const int stage = consumed % ST;
      cp_async_wait<ST - 2>();
      __syncwarp();
      const uint32_t sK = rows0 + stage * 2 * S::kTile, sV = sK + S::kTile, sS = scales0 + stage * S::kScales;
      const uint32_t ka0 = lds8(sS + g), ka1 = lds8(sS + g + 8), vb0 = lds8(sS + 16 + g), vb1 = lds8(sS + 24 + g);

      // S = K Q^T: rows g and g + 8 of the tile, heads 2t and 2t + 1.
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 x = lds128(sK + k_off<D>(g, t + 4 * c)), y = lds128(sK + k_off<D>(g + 8, t + 4 * c));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_half(xw[w], a0, a2);
          e4m3x4_to_half(yw[w], a1, a3);
          mma16816((w & 1) ? sb : sa, a0, a1, a2, a3, qf[c * 4 + w][0], qf[c * 4 + w][1]);
        }
      }
      const float k0 = exp_byte(ka0), k1 = exp_byte(ka1);
      float y[4] = {(sa[0] + sb[0]) * (qs0 * k0), (sa[1] + sb[1]) * (qs1 * k0), (sa[2] + sb[2]) * (qs0 * k1),
                    (sa[3] + sb[3]) * (qs1 * k1)};
      if constexpr (CAP) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = a.cap * kLog2e * tanh_from_log2(y[e] * (2.f * kLog2e / a.cap));
      }
      if (rows < kRows) {
        if (g >= rows) y[0] = y[1] = -INFINITY;
        if (g + 8 >= rows) y[2] = y[3] = -INFINITY;
      }
      const float b0 = static_cast<float>(vb0) - 127.f, b1 = static_cast<float>(vb1) - 127.f;
      // d = y - m and e = d + b, against the references (-inf before the first tile,
      // whose first token is valid: d is then +inf and raises them).
      float d[4], e[4];
      bool up = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] = y[i] - m[i & 1];
        e[i] = d[i] + (i < 2 ? b0 : b1);
        up |= d[i] > 8.f || e[i] > R[i & 1] + 8.f;
      }
      if (__any_sync(kFull, up)) {
        float beta[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float my = warp_max(fmaxf(y[h], y[2 + h]), 16, 4);
          const float m_new = my - m[h] > 8.f ? my : m[h];
          const float shift = m[h] - m_new;  // 0, or by how much every earlier term falls
          if (m_new != m[h]) l[h] *= fast_exp2(shift);
          d[h] = y[h] - m_new;
          d[2 + h] = y[2 + h] - m_new;
          e[h] = d[h] + b0;
          e[2 + h] = d[2 + h] + b1;
          const float r_old = m_new != m[h] ? R[h] + shift : R[h];
          const float me = warp_max(fmaxf(e[h], e[2 + h]), 16, 4);
          const float r_new = me > r_old + 8.f ? me : r_old;
          beta[h] = r_new != r_old ? fast_exp2(r_old - r_new) : 1.f;
          m[h] = m_new;
          R[h] = r_new;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][k] *= beta[k & 1];
      }
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l[i & 1] += fast_exp2(d[i]);
        p[i] = fast_exp2(e[i] - R[i & 1] + 7.f);
      }
      const uint32_t pb0 = movmatrix_trans(pack2<__half>(p[0], p[1])), pb1 = movmatrix_trans(pack2<__half>(p[2], p[3]));

      // O += V^T P: lane (g, t) pairs tokens 2t, 2t + 1 (and + 8) of dims D/8 g ...
      if constexpr (D == 128) {
        const uint4 v0 = lds128(sV + v_off<D>(2 * t, g)), v1 = lds128(sV + v_off<D>(2 * t + 1, g)),
                    v2 = lds128(sV + v_off<D>(2 * t + 8, g)), v3 = lds128(sV + v_off<D>(2 * t + 9, g));
        const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w},
                       w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_half(__byte_perm(w0[i / 2], w1[i / 2], sel), a0, a1);
          e4m3x4_to_half(__byte_perm(w2[i / 2], w3[i / 2], sel), a2, a3);
          mma16816(acc[i], a0, a1, a2, a3, pb0, pb1);
        }
      } else {
        const uint32_t h8 = (g & 1) * 8;
        const uint2 v0 = lds64(sV + v_off<D>(2 * t, g >> 1) + h8), v1 = lds64(sV + v_off<D>(2 * t + 1, g >> 1) + h8),
                    v2 = lds64(sV + v_off<D>(2 * t + 8, g >> 1) + h8), v3 = lds64(sV + v_off<D>(2 * t + 9, g >> 1) + h8);
        const uint32_t w0[2] = {v0.x, v0.y}, w1[2] = {v1.x, v1.y}, w2[2] = {v2.x, v2.y}, w3[2] = {v3.x, v3.y};
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_half(__byte_perm(w0[i / 2], w1[i / 2], sel), a0, a1);
          e4m3x4_to_half(__byte_perm(w2[i / 2], w3[i / 2], sel), a2, a3);
          mma16816(acc[i], a0, a1, a2, a3, pb0, pb1);
        }
      }
      ++consumed;
      __syncwarp();  // every lane has read the stage before it is filled again
      issue();
    }

    // acc[i][h] and acc[i][2 + h] are dims D/8 g + 2i and + 2i + 1 of head 2t + h.
    const bool empty = sg.n_pages == 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float lh = l[h];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) lh += __shfl_xor_sync(kFull, lh, o);
      const int head = 2 * t + h;
      if (head >= G) continue;
      const float f = empty ? 0.f : exp2f(R[h] - 7.f) / lh;
      const float lse_v = empty ? -INFINITY : (m[h] + log2f(lh)) * kLn2;
      if (sg.slot < 0) {
        const int64_t orow = static_cast<int64_t>(sg.q_row) * a.num_qo_heads + hq0 + head;
        T* dst = static_cast<T*>(a.o) + orow * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < KS; i += 4) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = acc[i + e][h] * f;
            v[2 * e + 1] = acc[i + e][2 + h] * f;
          }
          *reinterpret_cast<uint4*>(dst + 2 * i) = from_float8<T>(v);
        }
        if (g == 0 && a.lse) a.lse[orow] = lse_v;
      } else {
        const int64_t prow = static_cast<int64_t>(sg.slot) * G + head;
        float* dst = a.part_o + prow * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < KS; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(acc[i][h] * f, acc[i][2 + h] * f, acc[i + 1][h] * f, acc[i + 1][2 + h] * f);
        if (g == 0) a.part_lse[prow] = lse_v;
      }
    }
  }
}

template <int D, typename T, bool CAP, PageMode MODE>
__global__ void __launch_bounds__(kDecodeWarps * 32, 1) decode8_kernel(const __grid_constant__ Decode8Args a) {
  using S = Shape8<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const uint32_t base = smem_addr(smem);
  decode8_worker<D, T, CAP, MODE>(a, blockIdx.x * kDecodeWarps + warp, base + warp * (S::kStages * 2 * S::kTile),
                                 base + kDecodeWarps * (S::kStages * 2 * S::kTile) + warp * (S::kStages * S::kScales));
}

template <int D, typename T>
cudaError_t launch_t(const Decode8Args& a, bool cap, int grid, cudaStream_t s) {
  const int P = a.d.page_size;
  void (*kern)(Decode8Args) = nullptr;
  if (P % kRows == 0)
    kern = cap ? decode8_kernel<D, T, true, kOne> : decode8_kernel<D, T, false, kOne>;
  else if (P % 4 == 0)
    kern = cap ? decode8_kernel<D, T, true, kFours> : decode8_kernel<D, T, false, kFours>;
  else
    kern = cap ? decode8_kernel<D, T, true, kAny> : decode8_kernel<D, T, false, kAny>;
  constexpr int smem = kDecodeWarps * Shape8<D>::kWarpBytes;
  static_assert(smem <= 232448, "decode ring exceeds shared memory");
  cudaError_t e = ensure_smem_limit(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, grid, kDecodeWarps * 32, smem, s, a);
}

}  // namespace

cudaError_t launch_decode8(const DecodeArgs& d, const uint8_t* scales, float sm_scale, int head_dim, int dtype, bool cap,
                           int grid, cudaStream_t stream) {
  Decode8Args a{d, scales, sm_scale, 0};
  if (d.page_size < kRows) a.small_div = (4096 + d.page_size - 1) / d.page_size;
  if (head_dim == 128)
    return dtype == PKV_BF16 ? launch_t<128, __nv_bfloat16>(a, cap, grid, stream) : launch_t<128, __half>(a, cap, grid, stream);
  if (head_dim == 64)
    return dtype == PKV_BF16 ? launch_t<64, __nv_bfloat16>(a, cap, grid, stream) : launch_t<64, __half>(a, cap, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
