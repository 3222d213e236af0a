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
// wastes nothing, and the padding of a smaller one costs no bandwidth.  (tcgen05 tiles
// would tie a CTA's warps together over 128 keys, with the codes expanded into shared
// memory first; here every warp streams on its own, and the tensor pipe is 16 % busy.)
//  - One CTA per SM holds 8 (head_dim 64: 16) independent warps, each with the plan's
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
//  - Short page lists are shared by the warps of one CTA, which join their states
//    through shared memory; longer ones are split over the card and merged by a second
//    kernel (the plan decides, see compute_decode_shared and compute_decode_heads).
// Measured (head_dim 128, 8 kv heads, page 16, call with its merge): 64 requests of 8192
// tokens 163, 165 and 169 us at groups 1, 4 and 8, 99, 98 and 96 % of measured HBM bandwidth;
// of 512 to 4096 tokens 48.5 us, 82 %, where about 8 us go to the launches, the chain of
// table reads before the first tile and the merge.
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

// How a tile lies in its pages: kOne, pages of a multiple of 16 rows, so that it lies in
// one; kFours, pages of 4, 8 or 12 rows; kAny, the other sizes below 16.
enum PageMode { kOne, kFours, kAny };

template <int D, PageMode MODE>
struct Shape8 {
  static constexpr int kTile = kRows * D;               // bytes of K (or V) of one tile
  // Exponent bytes of one tile: 16 of K and 16 of V, or (kAny) the aligned word
  // around each, with the byte's place in it behind the words.
  static constexpr int kScales = MODE == kAny ? 32 * 5 : 32;
  // 200 - 230 KB of rows and exponents per CTA.
  static constexpr int kStages = D == 128 ? (MODE == kAny ? 6 : 7) : 6;
  static constexpr int kWarps = decode8_warps(D);
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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, const float4& v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
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
  int win_base;        // 64 page ids from entry win_base of the segment, two per lane; the
  int win, win_next;   // second half is loaded half a window before its first use
  int stage;
};

__device__ __forceinline__ int feed_ids(const Feed& p, const DecodeArgs& a, int at) {
  return at < p.n_pages ? __ldg(a.kv_indices + p.idx_begin + at) : 0;
}

__device__ __forceinline__ void feed_enter(Feed& p, const DecodeArgs& a, int lane) {
  const SegInfo s = load_seg(a.segs, p.seg, lane);
  p.idx_begin = s.idx_begin;
  p.n_pages = s.n_pages;
  p.n_tok = seg_tokens(s.n_pages, s.last_rows, a.page_size);
  p.kvh = s.kvh;
  p.tok = p.page = p.row = p.win_base = 0;
  p.win = feed_ids(p, a, lane);
  p.win_next = feed_ids(p, a, lane + 32);
}

// Issue the next tile's copies as one cp.async group (an empty one when the list has
// ended).  Rows past the request, and of a page id outside the pool, arrive as zeros.
// Exponent bytes are copied in aligned fours (which may take in slots past
// kv_last_page_len: their scores are masked).
template <int D, PageMode MODE>
__device__ __forceinline__ void feed_issue(Feed& p, const DecodeArgs& a, const uint8_t* scales, uint32_t rows0,
                                           uint32_t scales0, int lane, int64_t num_pages, uint32_t small_div,
                                           uint64_t policy) {
  using S = Shape8<D, MODE>;
  constexpr int CPR = D / 16;          // 16-byte chunks per row
  constexpr int RPI = 32 / CPR;        // rows per copy instruction
  while (p.seg < p.seg_end && p.tok >= p.n_tok) {
    ++p.seg;
    if (p.seg < p.seg_end) feed_enter(p, a, lane);
  }
  if (p.seg < p.seg_end) {
    const int P = a.page_size;
    const int rows = min(kRows, p.n_tok - p.tok);
    const uint32_t dst = rows0 + p.stage * 2 * S::kTile, dst_s = scales0 + p.stage * S::kScales;
    p.stage = p.stage + 1 == S::kStages ? 0 : p.stage + 1;
    const uint8_t* kv = static_cast<const uint8_t*>(a.kv);
    const uint32_t vdist = static_cast<uint32_t>(a.num_kv_heads) * P;  // rows from a K row to its V row
    const uint8_t* kv_v = kv + static_cast<uint64_t>(vdist) * D;
    if (p.page - p.win_base >= 32) {
      p.win_base += 32;
      p.win = p.win_next;
      p.win_next = feed_ids(p, a, p.win_base + 32 + lane);
    }
    const int w0 = p.page - p.win_base;
    if constexpr (MODE == kOne) {
      const int id = __shfl_sync(kFull, p.win, w0);
      const bool bad = id < 0 || id >= num_pages;
      const uint32_t at = bad ? 0u : (static_cast<uint32_t>(id) * 2u * a.num_kv_heads + p.kvh) * P + p.row;
      const int valid = bad ? 0 : rows;
      // The tile's rows are contiguous: chunk it * 32 + lane of K, and of V.
      const uint64_t off = static_cast<uint64_t>(at) * D + lane * 16;
#pragma unroll
      for (int it = 0; it < kRows / RPI; ++it) {
        const int r = it * RPI + lane / CPR, c = lane % CPR;
        const uint32_t n = r < valid ? 16u : 0u;
        cp_async_16_hint(dst + k_off<D>(r, c), kv + off + it * 512, n, policy);
        cp_async_16_hint(dst + S::kTile + v_off<D>(r, c), kv_v + off + it * 512, n, policy);
      }
      if (lane < 8)
        cp_async_4(dst_s + lane * 4, scales + (at + (lane & 3) * 4 + (lane < 4 ? 0u : vdist)), bad ? 0u : 4u);
      if (bad && lane == 0) atomicOr(a.err, kErrPageIndex);
      p.row += kRows;
      if (p.row == P) {
        p.row = 0;
        ++p.page;
      }
    } else {
      // Lanes i and 16 + i find K row i of the tile: its row counted over the pool's
      // (page, head) blocks, or kNone past the tile's rows or in a page outside the pool.
      constexpr uint32_t kNone = 0xffffffffu;
      const int i = lane & 15, x = p.row + i;
      const int k = static_cast<int>((static_cast<uint32_t>(x) * small_div) >> 12);  // x / P
      const int id0 = __shfl_sync(kFull, p.win, (w0 + k) & 31), id1 = __shfl_sync(kFull, p.win_next, (w0 + k) & 31);
      const int id = w0 + k < 32 ? id0 : id1;
      const bool bad = i < rows && (id < 0 || id >= num_pages);
      uint32_t at = (static_cast<uint32_t>(id) * 2u * a.num_kv_heads + p.kvh) * P + (x - k * P);
      if (bad || i >= rows) at = kNone;
      if (bad) atomicOr(a.err, kErrPageIndex);
#pragma unroll
      for (int it = 0; it < kRows / RPI; ++it) {
        const int r = it * RPI + lane / CPR, c = lane % CPR;
        const uint32_t row = __shfl_sync(kFull, at, r);
        const uint64_t off = row == kNone ? 0u : static_cast<uint64_t>(row) * D + c * 16;
        const uint32_t n = row == kNone ? 0u : 16u;
        cp_async_16_hint(dst + k_off<D>(r, c), kv + off, n, policy);
        cp_async_16_hint(dst + S::kTile + v_off<D>(r, c), row == kNone ? kv : kv_v + off, n, policy);
      }
      if constexpr (MODE == kFours) {
        const uint32_t row = __shfl_sync(kFull, at, (lane & 3) * 4);
        if (lane < 8)
          cp_async_4(dst_s + lane * 4, scales + (row == kNone ? 0u : row + (lane < 4 ? 0u : vdist)), row == kNone ? 0u : 4u);
      } else {
        // Lane i < 16: K's byte of token i, lane 16 + i: V's.
        const uint32_t byte = at == kNone ? 0u : at + (lane < 16 ? 0u : vdist), word = byte & ~3u;
        const uint64_t left = static_cast<uint64_t>(num_pages) * 2 * vdist - word;  // bytes of the pool from this word on
        cp_async_4(dst_s + lane * 4, scales + word, at == kNone ? 0u : static_cast<uint32_t>(left < 4 ? left : 4));
        sts8(dst_s + 128 + lane, (byte - word) * 8);
      }
      p.row += kRows;
      const int full = static_cast<int>((static_cast<uint32_t>(p.row) * small_div) >> 12);
      p.page += full;
      p.row -= full * P;
    }
    p.tok += rows;
  }
  cp_async_commit();
}

struct Decode8Args {
  DecodeArgs d;            // kv: the e4m3 codes; q_scale unused
  const uint8_t* scales;
  float sm_scale;
  uint32_t small_div;      // page_size < 16: ceil(4096 / page_size)
};

// A lane's running state of one segment: heads 2t and 2t + 1 of its quad position t.
template <int KS>
struct Acc8 {
  float m[2], R[2], l[2];
  float o[KS][4];  // o[i][h], o[i][2 + h]: dims D/8 g + 2i and + 2i + 1 of head 2t + h
};

// NT consecutive tiles in shared memory (the last of `rows` valid rows, 1 .. 16).
template <int D, bool CAP, PageMode MODE, int NT>
__device__ __forceinline__ void tiles_step(const DecodeArgs& a, const uint32_t (&sK)[NT], const uint32_t (&sS)[NT],
                                           int rows, int g, int t, const uint32_t (&qf)[D / 16][2], float qs0,
                                           float qs1, Acc8<D / 16>& st) {
  using S = Shape8<D, MODE>;
  constexpr int KC = D / 64, KS = D / 16;
  float y[NT][4], b[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // Exponent bytes of K and V, tokens g and g + 8.
    uint32_t kb[2], vb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (MODE == kAny) {
        const uint32_t i = g + 8 * h;
        kb[h] = (lds32(sS[n] + 4 * i) >> lds8(sS[n] + 128 + i)) & 255u;
        vb[h] = (lds32(sS[n] + 64 + 4 * i) >> lds8(sS[n] + 144 + i)) & 255u;
      } else {
        kb[h] = lds8(sS[n] + g + 8 * h);
        vb[h] = lds8(sS[n] + 16 + g + 8 * h);
      }
      b[n][h] = static_cast<float>(vb[h]) - 127.f;
    }
    // S = K Q^T: rows g and g + 8 of the tile, heads 2t and 2t + 1.
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const uint4 x = lds128(sK[n] + k_off<D>(g, t + 4 * c)), z = lds128(sK[n] + k_off<D>(g + 8, t + 4 * c));
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_half(xw[w], a0, a2);
        e4m3x4_to_half(zw[w], a1, a3);
        mma16816((w & 1) ? sb : sa, a0, a1, a2, a3, qf[c * 4 + w][0], qf[c * 4 + w][1]);
      }
    }
    const float k0 = exp_byte(kb[0]), k1 = exp_byte(kb[1]);
    y[n][0] = (sa[0] + sb[0]) * (qs0 * k0);
    y[n][1] = (sa[1] + sb[1]) * (qs1 * k0);
    y[n][2] = (sa[2] + sb[2]) * (qs0 * k1);
    y[n][3] = (sa[3] + sb[3]) * (qs1 * k1);
    if constexpr (CAP) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[n][i] = a.cap * kLog2e * tanh_from_log2(y[n][i] * (2.f * kLog2e / a.cap));
    }
  }
  if (rows < kRows) {
    if (g >= rows) y[NT - 1][0] = y[NT - 1][1] = -INFINITY;
    if (g + 8 >= rows) y[NT - 1][2] = y[NT - 1][3] = -INFINITY;
  }
  // d = y - m and e = d + b, against the references (-inf before the first tile,
  // whose first token is valid: d is then +inf and raises them).
  float d[NT][4], e[NT][4];
  bool up = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[n][i] = y[n][i] - st.m[i & 1];
      e[n][i] = d[n][i] + b[n][i >> 1];
      up |= d[n][i] > 8.f || e[n][i] > st.R[i & 1] + 8.f;
    }
  if (__any_sync(kFull, up)) {
    float beta[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float my = fmaxf(y[0][h], y[0][2 + h]);
#pragma unroll
      for (int n = 1; n < NT; ++n) my = fmaxf(my, fmaxf(y[n][h], y[n][2 + h]));
      my = warp_max(my, 16, 4);
      const float m_new = my - st.m[h] > 8.f ? my : st.m[h];
      const float shift = st.m[h] - m_new;  // 0, or by how much every earlier term falls
      if (m_new != st.m[h]) st.l[h] *= fast_exp2(shift);
      float me = -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          d[n][2 * k + h] = y[n][2 * k + h] - m_new;
          e[n][2 * k + h] = d[n][2 * k + h] + b[n][k];
          me = fmaxf(me, e[n][2 * k + h]);
        }
      me = warp_max(me, 16, 4);
      const float r_old = m_new != st.m[h] ? st.R[h] + shift : st.R[h];
      const float r_new = me > r_old + 8.f ? me : r_old;
      beta[h] = r_new != r_old ? fast_exp2(r_old - r_new) : 1.f;
      st.m[h] = m_new;
      st.R[h] = r_new;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) st.o[i][k] *= beta[k & 1];
  }
  const float r7[2] = {7.f - st.R[0], 7.f - st.R[1]};
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      st.l[i & 1] += fast_exp2(d[n][i]);
      p[i] = fast_exp2(e[n][i] + r7[i & 1]);
    }
    const uint32_t pb0 = movmatrix_trans(pack2<__half>(p[0], p[1])), pb1 = movmatrix_trans(pack2<__half>(p[2], p[3]));
    // O += V^T P: lane (g, t) pairs tokens 2t, 2t + 1 (and + 8) of dims D/8 g ...
    const uint32_t sV = sK[n] + S::kTile;
    constexpr int W = KS / 2;  // 32-bit words of the lane's dims per row
    uint32_t w0[W], w1[W], w2[W], w3[W];
    if constexpr (D == 128) {
      const uint4 v0 = lds128(sV + v_off<D>(2 * t, g)), v1 = lds128(sV + v_off<D>(2 * t + 1, g)),
                  v2 = lds128(sV + v_off<D>(2 * t + 8, g)), v3 = lds128(sV + v_off<D>(2 * t + 9, g));
      w0[0] = v0.x; w0[1] = v0.y; w0[2] = v0.z; w0[3] = v0.w;
      w1[0] = v1.x; w1[1] = v1.y; w1[2] = v1.z; w1[3] = v1.w;
      w2[0] = v2.x; w2[1] = v2.y; w2[2] = v2.z; w2[3] = v2.w;
      w3[0] = v3.x; w3[1] = v3.y; w3[2] = v3.z; w3[3] = v3.w;
    } else {
      const uint32_t h8 = (g & 1) * 8;
      const uint2 v0 = lds64(sV + v_off<D>(2 * t, g >> 1) + h8), v1 = lds64(sV + v_off<D>(2 * t + 1, g >> 1) + h8),
                  v2 = lds64(sV + v_off<D>(2 * t + 8, g >> 1) + h8), v3 = lds64(sV + v_off<D>(2 * t + 9, g >> 1) + h8);
      w0[0] = v0.x; w0[1] = v0.y;
      w1[0] = v1.x; w1[1] = v1.y;
      w2[0] = v2.x; w2[1] = v2.y;
      w3[0] = v3.x; w3[1] = v3.y;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
      uint32_t a0, a1, a2, a3;
      e4m3x4_to_half(__byte_perm(w0[i / 2], w1[i / 2], sel), a0, a1);
      e4m3x4_to_half(__byte_perm(w2[i / 2], w3[i / 2], sel), a2, a3);
      mma16816(st.o[i], a0, a1, a2, a3, pb0, pb1);
    }
  }
}

// What a warp leaves for its CTA of a shared list's piece; its outputs are at the start
// of its ring, [head][dim] in fp32.
struct Shared8 {
  float lse[8];  // -inf without a piece
  int row, kvh;  // row: -1 without one
};

template <int D, typename T, bool CAP, PageMode MODE>
__device__ __forceinline__ void decode8_worker(const Decode8Args& a8, int worker, uint32_t rows0, uint32_t scales0,
                                               Shared8& mine) {
  using S = Shape8<D, MODE>;
  constexpr int ST = S::kStages;
  constexpr int KC = D / 64;     // 16-byte chunks of a K row per lane (and of a 16-bit Q row, pairs of them)
  constexpr int KS = D / 16;     // k steps of Q K^T, and 16-dim blocks of V^T P
  const DecodeArgs& a = a8.d;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const PlanHeader* hdr = a.hdr;
  // The table has an entry for every worker of the grid: read beside the header, used
  // where the plan gave this worker work.
  const int seg_begin = a.worker_ptr[worker], seg_end = a.worker_ptr[worker + 1];
  const int64_t num_pages = hdr->num_pages;
  if (worker >= hdr->num_workers || seg_begin >= seg_end) return;
  const uint64_t policy = l2_policy_evict_first();
  const int G = a.num_qo_heads / a.num_kv_heads;

  Feed feed;
  feed.seg = seg_begin;
  feed.seg_end = seg_end;
  feed.stage = 0;
  feed_enter(feed, a, lane);
  auto issue = [&] {
    feed_issue<D, MODE>(feed, a, a8.scales, rows0, scales0, lane, num_pages, a8.small_div, policy);
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue();

  int stage = 0;
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
    Acc8<KS> st;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      st.m[h] = st.R[h] = -INFINITY;
      st.l[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) st.o[i][k] = 0.f;

    const int n_tok = seg_tokens(sg.n_pages, sg.last_rows, a.page_size);
    auto next_stage = [&](uint32_t& sK, uint32_t& sS) {
      sK = rows0 + stage * 2 * S::kTile;
      sS = scales0 + stage * S::kScales;
      stage = stage + 1 == ST ? 0 : stage + 1;
    };
    // NT tiles a step (more independent work for the warp between its waits), and one a
    // step where fewer are left.  Of the ST - 1 groups ahead
    // of the compute side the first NT (or one) must have landed.
    constexpr int NT = 2;
    int tok = 0;
    for (; tok + (NT - 1) * kRows < n_tok; tok += NT * kRows) {
      cp_async_wait<ST - 1 - NT>();
      __syncwarp();
      uint32_t sK[NT], sS[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) next_stage(sK[n], sS[n]);
      tiles_step<D, CAP, MODE, NT>(a, sK, sS, min(kRows, n_tok - tok - (NT - 1) * kRows), g, t, qf, qs0, qs1, st);
      __syncwarp();  // every lane has read the stages before they are filled again
#pragma unroll 1
      for (int n = 0; n < NT; ++n) issue();
    }
    for (; tok < n_tok; tok += kRows) {
      cp_async_wait<ST - 2>();
      __syncwarp();
      uint32_t sK[1], sS[1];
      next_stage(sK[0], sS[0]);
      tiles_step<D, CAP, MODE, 1>(a, sK, sS, min(kRows, n_tok - tok), g, t, qf, qs0, qs1, st);
      __syncwarp();
      issue();
    }

    const bool empty = sg.n_pages == 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float lh = st.l[h];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) lh += __shfl_xor_sync(kFull, lh, o);
      const int head = 2 * t + h;
      if (head >= G) continue;
      const float f = empty ? 0.f : exp2f(st.R[h] - 7.f) / lh;
      const float lse_v = empty ? -INFINITY : (st.m[h] + log2f(lh)) * kLn2;
      if (sg.slot == -1) {
        const int64_t orow = static_cast<int64_t>(sg.q_row) * a.num_qo_heads + hq0 + head;
        T* dst = static_cast<T*>(a.o) + orow * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < KS; i += 4) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = st.o[i + e][h] * f;
            v[2 * e + 1] = st.o[i + e][2 + h] * f;
          }
          *reinterpret_cast<uint4*>(dst + 2 * i) = from_float8<T>(v);
        }
        if (g == 0 && a.lse) a.lse[orow] = lse_v;
      } else if (sg.slot == kSharedSlot) {
        // The warp's copies have all arrived and been read: its ring is free.
        const uint32_t dst = rows0 + (head * D + g * (D / 8)) * 4;
#pragma unroll
        for (int i = 0; i < KS; i += 2)
          sts128(dst + 8 * i, make_float4(st.o[i][h] * f, st.o[i][2 + h] * f, st.o[i + 1][h] * f, st.o[i + 1][2 + h] * f));
        if (g == 0) mine.lse[head] = lse_v;
        if (g == 0 && head == 0) {
          mine.row = sg.q_row;
          mine.kvh = sg.kvh;
        }
      } else {
        const int64_t prow = static_cast<int64_t>(sg.slot) * G + head;
        float* dst = a.part_o + prow * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < KS; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(st.o[i][h] * f, st.o[i][2 + h] * f, st.o[i + 1][h] * f, st.o[i + 1][2 + h] * f);
        if (g == 0) a.part_lse[prow] = lse_v;
      }
    }
  }
}

template <int D, typename T, bool CAP, PageMode MODE>
__global__ void __launch_bounds__(decode8_warps(D) * 32, 1) decode8_kernel(const __grid_constant__ Decode8Args a) {
  using S = Shape8<D, MODE>;
  extern __shared__ __align__(128) uint8_t smem[];
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int W = S::kWarps;
  __shared__ Shared8 shared[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int share = a.d.hdr->share;
  if (lane < 8) shared[warp].lse[lane] = -INFINITY;
  if (lane == 0) shared[warp].row = -1;
  __syncwarp();
  const uint32_t base = smem_addr(smem);
  constexpr uint32_t kRing = S::kStages * 2 * S::kTile;
  decode8_worker<D, T, CAP, MODE>(a, blockIdx.x * W + warp, base + warp * kRing,
                                  base + W * kRing + warp * (S::kStages * S::kScales), shared[warp]);
  if (share <= 1) return;
  // Lists shared by `share` neighbouring warps: each of them joins some of the heads.
  __syncthreads();
  constexpr int PER = D / 32;  // dims per lane
  const int first = warp / share * share;
  const int row = shared[first].row;  // the first piece exists where any does
  if (row < 0) return;
  const int G = a.d.num_qo_heads / a.d.num_kv_heads;
  for (int head = warp - first; head < G; head += share) {
    float m = -INFINITY;
    for (int k = 0; k < share; ++k) m = fmaxf(m, shared[first + k].lse[head]);
    float l = 0.f, acc[PER];
#pragma unroll
    for (int v = 0; v < PER; ++v) acc[v] = 0.f;
    for (int k = 0; k < share; ++k) {
      if (shared[first + k].lse[head] == -INFINITY) continue;  // no piece: its ring holds anything
      const float w = fast_exp2((shared[first + k].lse[head] - m) * kLog2e);
      l += w;
      const float* o = reinterpret_cast<const float*>(smem + (first + k) * kRing) + head * D + lane * PER;
#pragma unroll
      for (int v = 0; v < PER; ++v) acc[v] = fmaf(w, o[v], acc[v]);
    }
    const int64_t orow = static_cast<int64_t>(row) * a.d.num_qo_heads + shared[first].kvh * G + head;
    T* dst = static_cast<T*>(a.d.o) + orow * D + lane * PER;
    const float inv = 1.f / l;
#pragma unroll
    for (int v = 0; v < PER; v += 2) *reinterpret_cast<uint32_t*>(dst + v) = pack2<T>(acc[v] * inv, acc[v + 1] * inv);
    if (lane == 0 && a.d.lse) a.d.lse[orow] = m + logf(l);
  }
}

// The merge of split sequences, as decode_merge_pair computes it, with the slots of one
// (item, head) dealt to as many warps of a CTA as the grid has to spare and the slots
// fill (a power of two up to all of them): a request of 8192 tokens alone leaves 32 such
// pairs of 152 slots, which take one warp each 10 us to read and eight warps 2.5 us; the
// serving batch leaves 2016 pairs of 3 slots, a warp each.  The warps' states are
// combined in their order, so the result does not depend on timing.  A slot whose lse
// is NaN counts like any other (fmaxf passes over a NaN, so m may stay -inf beside it):
// its weight is NaN, and so are o and lse, as where one warp holds the whole list.
template <int D, typename T>
__global__ void __launch_bounds__(kMergeThreads) decode8_merge_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int PER = D / 32;           // dims per lane
  constexpr int W = kMergeThreads / 32;
  constexpr int U = 8;                  // slots in flight per lane
  __shared__ float s_o[W][D];
  __shared__ float s_m[W], s_l[W];
  // Launched as a programmatic dependent of the decode kernel: wait until that grid
  // has finished and its partial states are visible.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.num_qo_heads / a.num_kv_heads;
  const int n_items = a.hdr->num_merge, n_slots = a.hdr->num_slots;
  const int pairs = n_items * G;
  int wpp = W;  // warps per pair
  while (wpp > 1 && (static_cast<int64_t>(pairs) * wpp > static_cast<int64_t>(gridDim.x) * W ||
                     static_cast<int64_t>(n_items) * wpp * 4 > n_slots))
    wpp >>= 1;
  const int per_cta = W / wpp, part = warp % wpp;
  for (int p0 = blockIdx.x * per_cta; p0 < pairs; p0 += gridDim.x * per_cta) {
    const int pair = p0 + warp / wpp;
    const bool have = pair < pairs;
    float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
    for (int v = 0; v < PER; ++v) acc[v] = 0.f;
    MergeItem it{};
    const int g = pair % G;
    if (have) {
      it = a.merge[pair / G];
      const int lo = static_cast<int>(static_cast<int64_t>(it.n_slots) * part / wpp),
                hi = static_cast<int>(static_cast<int64_t>(it.n_slots) * (part + 1) / wpp);
      const float* lse_p = a.part_lse + static_cast<int64_t>(it.slot_begin) * G + g;
      const float* o_p = a.part_o + (static_cast<int64_t>(it.slot_begin) * G + g) * D + lane * PER;
      for (int i0 = lo; i0 < hi; i0 += U) {
        // U slots' lse and rows together, then folded into the running state.
        float vals[U][PER], lse[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          lse[u] = -INFINITY;
#pragma unroll
          for (int v = 0; v < PER; ++v) vals[u][v] = 0.f;
          if (i0 + u < hi) {
            const int64_t row = static_cast<int64_t>(i0 + u) * G;
            lse[u] = lse_p[row];
#pragma unroll
            for (int v = 0; v < PER; v += 2) {
              const float2 x = *reinterpret_cast<const float2*>(o_p + row * D + v);
              vals[u][v] = x.x;
              vals[u][v + 1] = x.y;
            }
          }
        }
        float top = m;
        bool any = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          top = fmaxf(top, lse[u]);
          any |= lse[u] != -INFINITY;
        }
        if (!any) continue;
        const float w0 = m == top ? 1.f : fast_exp2((m - top) * kLog2e);  // 0 while m alone is -inf
        l *= w0;
#pragma unroll
        for (int v = 0; v < PER; ++v) acc[v] *= w0;
        m = top;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float w = lse[u] == -INFINITY ? 0.f : fast_exp2((lse[u] - m) * kLog2e);  // 0 for a slot past hi
          l += w;
#pragma unroll
          for (int v = 0; v < PER; ++v) acc[v] = fmaf(w, vals[u][v], acc[v]);
        }
      }
    }
    if (wpp > 1) {
      __syncthreads();  // the round before has been read
      if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
      }
#pragma unroll
      for (int v = 0; v < PER; ++v) s_o[warp][lane * PER + v] = acc[v];
      __syncthreads();
      if (part == 0) {
        float top = m;
        for (int k = 1; k < wpp; ++k) top = fmaxf(top, s_m[warp + k]);
        const float w0 = m == top ? 1.f : fast_exp2((m - top) * kLog2e);
        l *= w0;
#pragma unroll
        for (int v = 0; v < PER; ++v) acc[v] *= w0;
        for (int k = 1; k < wpp; ++k) {
          if (s_l[warp + k] == 0.f) continue;  // no slots
          const float w = fast_exp2((s_m[warp + k] - top) * kLog2e);
          l = fmaf(w, s_l[warp + k], l);
#pragma unroll
          for (int v = 0; v < PER; ++v) acc[v] = fmaf(w, s_o[warp + k][lane * PER + v], acc[v]);
        }
        m = top;
      }
    }
    if (have && part == 0) {
      const int64_t row = static_cast<int64_t>(it.row) * a.num_qo_heads + it.kvh * G + g;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T* dst = static_cast<T*>(a.o) + row * D + lane * PER;
#pragma unroll
      for (int v = 0; v < PER; v += 2)
        *reinterpret_cast<uint32_t*>(dst + v) = pack2<T>(acc[v] * inv, acc[v + 1] * inv);
      if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
    }
  }
}

template <int D, typename T>
cudaError_t launch_t(const Decode8Args& a, bool cap, int grid, cudaStream_t s) {
  const int P = a.d.page_size;
  void (*kern)(Decode8Args) = nullptr;
  constexpr int W = decode8_warps(D);
  int smem = W * Shape8<D, kOne>::kWarpBytes;
  static_assert(W * Shape8<D, kOne>::kWarpBytes <= 232448 && W * Shape8<D, kAny>::kWarpBytes <= 232448 &&
                    Shape8<D, kFours>::kWarpBytes == Shape8<D, kOne>::kWarpBytes,
                "decode ring exceeds shared memory");
  if (P % kRows == 0) {
    kern = cap ? decode8_kernel<D, T, true, kOne> : decode8_kernel<D, T, false, kOne>;
  } else if (P % 4 == 0) {
    kern = cap ? decode8_kernel<D, T, true, kFours> : decode8_kernel<D, T, false, kFours>;
  } else {
    kern = cap ? decode8_kernel<D, T, true, kAny> : decode8_kernel<D, T, false, kAny>;
    smem = W * Shape8<D, kAny>::kWarpBytes;
  }
  cudaError_t e = ensure_smem_limit(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, grid, W * 32, smem, s, a);
}

}  // namespace

cudaError_t launch_decode8(const DecodeArgs& d, const uint8_t* scales, float sm_scale, int head_dim, int dtype, bool cap,
                           int grid, int64_t num_pages, cudaStream_t stream) {
  // Rows of the pool are counted in 32 bits, with the last value for none.
  if (static_cast<double>(num_pages) * 2 * d.num_kv_heads * d.page_size >= 4294967295.0) return cudaErrorInvalidValue;
  Decode8Args a{d, scales, sm_scale, 0};
  if (d.page_size < kRows) a.small_div = (4096 + d.page_size - 1) / d.page_size;
  if (head_dim == 128)
    return dtype == PKV_BF16 ? launch_t<128, __nv_bfloat16>(a, cap, grid, stream) : launch_t<128, __half>(a, cap, grid, stream);
  if (head_dim == 64)
    return dtype == PKV_BF16 ? launch_t<64, __nv_bfloat16>(a, cap, grid, stream) : launch_t<64, __half>(a, cap, grid, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode8_merge(const DecodeArgs& a, int head_dim, int dtype, int grid, cudaStream_t stream) {
  void (*kern)(DecodeArgs) = nullptr;
  if (head_dim == 128)
    kern = dtype == PKV_BF16 ? decode8_merge_kernel<128, __nv_bfloat16> : decode8_merge_kernel<128, __half>;
  else if (head_dim == 64)
    kern = dtype == PKV_BF16 ? decode8_merge_kernel<64, __nv_bfloat16> : decode8_merge_kernel<64, __half>;
  if (!kern) return cudaErrorInvalidValue;
  return launch_dependent(kern, grid, kMergeThreads, 0, stream, a);
}

}  // namespace pkv
