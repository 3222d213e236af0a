// evict.cu -- which keys of a cache stay, and their move to the front of a page list
// (pkv_select_keys, pkv_compact_paged_kv).
//
// Select.  For each (request, kv head) the last `window` keys stay, then the first `sink`
// ones, then those of the largest weight (equal weights: the lower index), up to the
// request's budget.  A radix select on the weights' bits in order of their values: passes of
// 12, 10 and 10 bits find the weight T of the last key that stays and how many keys of
// weight T stay; one more pass writes the indices in ascending order, places counted by
// ballots.  (The first digit holds the exponent and three bits of the mantissa.)  The weights
// are read from global memory once and kept in shared memory as ordered 32-bit integers
// (what does not fit is read again).  The CTAs of a cluster share a long list, each a
// contiguous slice; they add their digit counts through distributed shared memory.  Each of
// five passes looks at every key (issue slots 57 % busy on average, 74 % on the busiest SM,
// on the batch below) and ends at a barrier; loops are unrolled over independent keys, and
// a digit is found by 64 threads that each add up the counts above one (a chain of shuffles
// took 4800 of a list's 36000 cycles).  Measured, 8 kv heads: 64 requests of 512 to 4096 keys 15.4 us (20.7 us with
// digits of 8 bits and a key at a time), 2 requests of 10^5 keys 25.4 us (50.3 us).  CTAs
// and shared memory a list go by the average length, which the host knows: one request of
// 10^5 keys among 63 of 500 takes 1000 us, most of its keys being read again in each pass.
//
// Compact.  A kept key moves from its token index s to its place i <= s in the list of
// kept keys.  In place, a CTA owns a column slice of one (request, kv head, K or V) and
// moves the rows in order, 128 to 1024 at a time: every thread has read its part of a round before
// any writes it, and what a round writes lies before everything later rounds read
// (s >= i), so the next round is read ahead of the writes.  Slices of 32 bytes or more
// give a list up to 16 CTAs (8 in the 8-bit cache at head_dim 128), and one more moves scales
// and weights; into other pages rounds are independent, and go to as many CTAs as the chip
// holds.  A batch is HBM-bound, each kept row read once and written once: 64 requests of 512
// to 4096 keys, half kept, 118 us, 80 % of measured bandwidth.  One request alone is not: of
// 10^5 keys, 8 kv heads, half kept, 237 us (8-bit cache 226) against 62 (32) for its bytes.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "pkv_bsr.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr unsigned kFullMask = 0xffffffffu;
// Keys of a request: indices are 32-bit and run ahead of the last key by up to a page (2^20 slots)
// or a few thousand keys.
constexpr int kMaxKeys = INT_MAX - (1 << 21);

// Where the keys of a batch are.
struct Table {
  const int32_t* indptr;
  const int32_t* indices;
  const int32_t* last;
  int64_t num_pages, kv_pages;
  int batch, hkv, page_size;
  int32_t* err;
};

__device__ __forceinline__ void flag(const Table& t, int bits) {
  if (t.err) atomicOr(t.err, bits);
}

// Request b's first entry of kv_indices and its keys; false where the arrays do not fit.
__device__ __forceinline__ bool keys_of(const Table& t, int b, int& page0, int& len) {
  const int p0 = __ldg(t.indptr + b), p1 = __ldg(t.indptr + b + 1), last = __ldg(t.last + b);
  page0 = p0;
  len = 0;
  if (p0 < 0 || p1 < p0 || p1 > t.kv_pages) return false;
  if (p1 == p0) return true;
  const int64_t n = static_cast<int64_t>(p1 - p0 - 1) * t.page_size + last;
  if (last < 1 || last > t.page_size || n > kMaxKeys) return false;
  len = static_cast<int>(n);
  return true;
}

// ---------------------------------------------------------------------------- select
constexpr int kMaxHeld = 48 * 1024;  // weights in shared memory

struct SelectArgs {
  Table t;
  const float* weights;   // [num_pages, Hkv, P]
  const int32_t* budget;
  int sink, window, max_keep;
  int32_t* keep;          // [batch, Hkv, max_keep]
  int32_t* kept_len;      // [batch]
  int share;              // CTAs of a cluster
  int held;               // weights a CTA keeps in shared memory, a multiple of 4
  uint32_t page_mul;      // ceil(2^32 / page_size) (page_size > 1)
  int fours;              // four keys' weights are one aligned load
};

// Digits of the three passes, in one array of counters behind one another.
__device__ constexpr int digit_bits(int pass) { return pass == 0 ? 12 : 10; }
__device__ constexpr int digit_shift(int pass) { return 20 - 10 * pass; }
__device__ constexpr int first_bin(int pass) { return pass == 0 ? 0 : 4096 + 1024 * (pass - 1); }
constexpr int kBins = 6144, kGroup = 64;  // bins that are first counted together

template <int THREADS>
struct SelectShared {
  alignas(16) uint32_t hist[kBins];
  alignas(16) uint32_t group[3][kGroup];
  alignas(16) uint32_t all[2][kGroup];  // counts of 64 groups, then of the 64 bins of one, over the cluster
  uint32_t warp_gt[THREADS / 32], warp_eq[THREADS / 32];
  uint32_t total[2];      // this CTA's keys above T, and of weight T
  uint32_t digit, left, group_at, group_left;
};

// Of 64 counts in shared memory, the one that holds the left-th key from above: thread i of 64
// adds up those above count i (no chain of shuffles).
__device__ __forceinline__ void find_count(const uint32_t* counts, int i, uint32_t left, int base, uint32_t& digit,
                                           uint32_t& rest) {
  uint32_t above = 0;
#pragma unroll
  for (int k = 0; k < kGroup; k += 4) {
    const uint4 c = *reinterpret_cast<const uint4*>(counts + k);
    above += (k > i ? c.x : 0u) + (k + 1 > i ? c.y : 0u) + (k + 2 > i ? c.z : 0u) + (k + 3 > i ? c.w : 0u);
  }
  if (above < left && above + counts[i] >= left) {
    digit = base + i;
    rest = left - above;
  }
}

// The weight's bits in order of its value: NaN lowest (1), -0 equal to +0.  0 stands for no key.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t v = __float_as_uint(x + 0.f);
  if (x != x) return 1u;
  return v & 0x80000000u ? ~v : v | 0x80000000u;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) select_keys_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kWarps = THREADS / 32;
  extern __shared__ __align__(16) uint32_t held[];
  __shared__ SelectShared<THREADS> sh;
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int share = a.share, rank = share > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int list = blockIdx.x / share, b = list / a.t.hkv, h = list - b * a.t.hkv;
  int page0, len;
  const int asked = __ldg(a.budget + b);
  const bool ok = keys_of(a.t, b, page0, len);
  if (!ok && tid == 0) flag(a.t, kErrAppendLayout);
  const int n = min(min(max(asked, 0), len), a.max_keep);
  const int tail = min(a.window, n), front = min(a.sink, n - tail);
  const int pick = n - tail - front, mid = len - tail - front;  // pick of keys front .. front + mid - 1
  const int P = a.t.page_size;
  // The keys between in aligned groups of four, a run of groups for each CTA: entry e is key j0 + e.
  const int first4 = front & ~3, end = front + mid, groups = (end - first4 + 3) / 4;
  const int slice = (groups + share - 1) / share;
  const int g0 = min(rank * slice, groups), count = (min(g0 + slice, groups) - g0) * 4, j0 = first4 + g0 * 4;
  auto page_of = [&](int j) { return P == 1 ? j : [&] { const int q = __umulhi(j, a.page_mul); return q * P > j ? q - 1 : q; }(); };
  auto row_of = [&](int j, int pg) -> int64_t {  // the weight of key j, or -1
    const int page = __ldg(a.t.indices + page0 + pg);
    if (page < 0 || page >= a.t.num_pages) {
      flag(a.t, kErrPageIndex);
      return -1;
    }
    return (static_cast<int64_t>(page) * a.t.hkv + h) * P + (j - pg * P);
  };
  auto fetch = [&](int e) -> uint32_t {
    const int j = j0 + e;
    if (j < front || j >= end) return 0u;
    const int64_t at = row_of(j, page_of(j));
    return at < 0 ? 1u : ordered(__ldg(a.weights + at));
  };
  const int in_smem = min(count, a.held);
  if (pick > 0 && pick < mid) {
    // Page ids of kAhead loads first, then the loads, then what they brought.
    constexpr int kAhead = 4;
    const int width = a.fours ? 4 : 1;
    bool bad = false;
    for (int e0 = tid * width; e0 < in_smem; e0 += kAhead * THREADS * width) {
      int page[kAhead], at_slot[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int e = e0 + k * THREADS * width, j = j0 + e;  // fours: key j's page holds all four
        const bool in = e < in_smem && (a.fours || (j >= front && j < end));
        const int pg = in ? page_of(j) : 0;
        at_slot[k] = j - pg * P;
        page[k] = in ? __ldg(a.t.indices + page0 + pg) : -1;
        if (!in) at_slot[k] = -1;
      }
      float4 w[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const bool use = page[k] >= 0 && page[k] < a.t.num_pages;
        bad |= !use && at_slot[k] >= 0;
        const float* at = a.weights + (use ? (static_cast<int64_t>(page[k]) * a.t.hkv + h) * P + at_slot[k] : 0);
        const float nan = __int_as_float(0x7fffffff);  // a key in no page: one of the lowest
        w[k] = make_float4(nan, nan, nan, nan);
        if (a.fours) {
          if (use) w[k] = __ldg(reinterpret_cast<const float4*>(at));
        } else if (use) {
          w[k].x = __ldg(at);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int e = e0 + k * THREADS * width, j = j0 + e;
        if (e >= in_smem) continue;
        if (a.fours) {
          *reinterpret_cast<uint4*>(held + e) =
              make_uint4(j < front || j >= end ? 0u : ordered(w[k].x), j + 1 < front || j + 1 >= end ? 0u : ordered(w[k].y),
                         j + 2 < front || j + 2 >= end ? 0u : ordered(w[k].z), j + 3 < front || j + 3 >= end ? 0u : ordered(w[k].w));
        } else {
          held[e] = j < front || j >= end ? 0u : ordered(w[k].x);
        }
      }
    }
    if (bad) flag(a.t, kErrPageIndex);
  }
  int32_t* out = a.keep + static_cast<int64_t>(list) * a.max_keep;
  if (h == 0 && rank == 0 && tid == 0) a.kept_len[b] = n;
  // The keys that stay anyway, and what is past the list.
  const uint32_t step = share * THREADS;  // (unsigned: the last step may pass 2^31)
  for (uint32_t at = rank * THREADS + tid; at < static_cast<uint32_t>(a.max_keep); at += step) {
    const int i = static_cast<int>(at);
    if (i >= front && i < n - tail && pick < mid) {
      at += (n - tail - 1 - i) / step * step;  // the chosen ones are written below
      continue;
    }
    out[i] = i >= n ? -1 : i >= n - tail ? len - (n - i) : i;
  }
  if (pick == 0 || pick == mid) return;  // the same for all CTAs of a cluster
  for (int i = tid * 4; i < kBins; i += THREADS * 4) *reinterpret_cast<uint4*>(sh.hist + i) = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  uint32_t prefix = 0;
  int left = pick;  // keys still to find among those whose upper digits are prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = digit_shift(pass), bits = digit_bits(pass);
    uint32_t* hist = sh.hist + first_bin(pass);
    auto count_key = [&](uint32_t v) {
      if (v != 0u && (pass == 0 || v >> ((shift + bits) & 31) == prefix)) atomicAdd(hist + (v >> shift & ((1u << bits) - 1)), 1u);
    };
    for (int e0 = tid; e0 < in_smem; e0 += 4 * THREADS) {
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = e0 + k * THREADS < in_smem ? held[e0 + k * THREADS] : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) count_key(v[k]);
    }
    for (int e = in_smem + tid; e < count; e += THREADS) count_key(fetch(e));
    __syncthreads();
    // Groups of 64 bins are counted first: the group, then the bin, each over the cluster.
    const int n_groups = (1 << bits) / kGroup;
    for (int g = warp; g < kGroup; g += kWarps) {
      const uint32_t c = g < n_groups ? __reduce_add_sync(kFullMask, hist[g * kGroup + lane] + hist[g * kGroup + 32 + lane]) : 0u;
      if (lane == 0) sh.group[pass][g] = c;
    }
    auto over_cluster = [&](const uint32_t* x, uint32_t* sum) {  // 64 threads
      uint32_t c[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) c[r] = r < share ? ld_cluster_u32(x + tid, r) : 0u;
      sum[tid] = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
    };
    const uint32_t* counts = sh.group[pass];
    if (share > 1) {
      cluster_sync_all();
      if (tid < kGroup) over_cluster(counts, sh.all[0]);
      counts = sh.all[0];
    }
    __syncthreads();
    if (tid < kGroup) find_count(counts, tid, left, 0, sh.group_at, sh.group_left);
    __syncthreads();
    const int g = static_cast<int>(sh.group_at);
    counts = hist + g * kGroup;
    if (share > 1) {
      if (tid < kGroup) over_cluster(counts, sh.all[1]);
      counts = sh.all[1];
      __syncthreads();
    }
    if (tid < kGroup) find_count(counts, tid, sh.group_left, g * kGroup, sh.digit, sh.left);
    __syncthreads();
    prefix = prefix << bits | sh.digit;
    left = static_cast<int>(sh.left);
  }
  // prefix is T; left of the keys of weight T stay, those of the lowest index.  Each warp has a
  // contiguous run of the slice.
  const int per_warp = ((count + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int w0 = min(warp * per_warp, count), w1 = min(w0 + per_warp, count);
  uint32_t gt = 0, eq = 0;
  // Four neighbouring chunks of 32 keys of a run.
  auto load4 = [&](int e0, uint32_t (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = e0 + k * 32 + lane < min(w1, in_smem) ? held[e0 + k * 32 + lane] : 0u;
    if (e0 + 128 > in_smem && in_smem < w1) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int e = e0 + k * 32 + lane;
        const uint32_t x = e >= in_smem && e < w1 ? fetch(e) : 0u;
        if (k == 0) v[0] |= x;
        if (k == 1) v[1] |= x;
        if (k == 2) v[2] |= x;
        if (k == 3) v[3] |= x;
      }
    }
  };
  for (int e0 = w0; e0 < w1; e0 += 128) {
    uint32_t v[4];
    load4(e0, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      gt += v[k] > prefix;
      eq += v[k] == prefix;
    }
  }
  gt = __reduce_add_sync(kFullMask, gt);
  eq = __reduce_add_sync(kFullMask, eq);
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  // Before this warp's run.
  uint32_t gt0 = __reduce_add_sync(kFullMask, lane < warp ? sh.warp_gt[lane] : 0u);
  uint32_t eq0 = __reduce_add_sync(kFullMask, lane < warp ? sh.warp_eq[lane] : 0u);
  if (share > 1) {
    if (tid == THREADS - 1) {  // the last warp's end is the slice's
      sh.total[0] = gt0 + sh.warp_gt[kWarps - 1];
      sh.total[1] = eq0 + sh.warp_eq[kWarps - 1];
    }
    cluster_sync_all();
    uint32_t g[8], q[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      g[r] = r < rank ? ld_cluster_u32(&sh.total[0], r) : 0u;
      q[r] = r < rank ? ld_cluster_u32(&sh.total[1], r) : 0u;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      gt0 += g[r];
      eq0 += q[r];
    }
  }
  const uint32_t below = (1u << lane) - 1;
  for (int e0 = w0; e0 < w1; e0 += 128) {
    uint32_t v[4];
    load4(e0, v);
    unsigned mg[4], mq[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mg[k] = __ballot_sync(kFullMask, v[k] > prefix);
      mq[k] = __ballot_sync(kFullMask, v[k] == prefix);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t q_at = eq0 + __popc(mq[k] & below), g_at = gt0 + __popc(mg[k] & below);
      if (v[k] > prefix || (v[k] == prefix && q_at < static_cast<uint32_t>(left)))
        out[front + g_at + min(q_at, static_cast<uint32_t>(left))] = j0 + e0 + k * 32 + lane;
      gt0 += __popc(mg[k]);
      eq0 += __popc(mq[k]);
    }
  }
  if (share > 1) cluster_sync_all();  // a CTA's counts stay until they have been read
}

// --------------------------------------------------------------------------- compact
constexpr int kCmpThreads = 256;
constexpr int kSteps = 8;                // 16-byte pieces of a round per thread
constexpr uint32_t kNoRow = 0xffffffffu;

struct CompactArgs {
  Table t;
  const int32_t* keep;       // [batch, Hkv, max_keep], ascending
  const int32_t* kept_len;   // [batch]
  int max_keep;
  const int32_t* dst_indptr;   // nullptr: in place
  const int32_t* dst_indices;
  int64_t dst_pages;
  uint8_t* kv;               // [num_pages, 2, Hkv, P] rows
  uint8_t* scales;           // [num_pages, 2, Hkv, P] or nullptr
  float* weights;            // [num_pages, Hkv, P] or nullptr
  int split;                 // column slices of a row
  int parts;                 // CTAs that share a slice's rounds (in place: 1)
  int roles;                 // CTAs per list: 2 split parts, and one for scales and weights
};

// Rows of a (request, head): where kept key i comes from and goes to, counted over the
// pool's rows (the K row), or kNoRow where it stays or cannot move.
struct Moves {
  int page0, len, n;
  const int32_t* dst;        // page table of the destination
  const int32_t* keep;
};

__device__ __forceinline__ bool moves_of(const CompactArgs& a, int b, int h, Moves& m) {
  m.n = __ldg(a.kept_len + b);
  m.keep = a.keep + (static_cast<int64_t>(b) * a.t.hkv + h) * a.max_keep;
  bool ok = keys_of(a.t, b, m.page0, m.len) && m.n >= 0 && m.n <= m.len && m.n <= a.max_keep;
  if (a.dst_indptr) {
    const int d0 = __ldg(a.dst_indptr + b), d1 = __ldg(a.dst_indptr + b + 1);
    ok = ok && d0 >= 0 && d1 >= d0 && d1 <= a.dst_pages && (static_cast<int64_t>(d1) - d0) * a.t.page_size >= m.n;
    m.dst = a.dst_indices + d0;
  } else {
    m.dst = a.t.indices + m.page0;
  }
  return ok;
}

__device__ __forceinline__ uint2 move_of(const CompactArgs& a, const Moves& m, int i, int h, int& err) {
  uint2 r = make_uint2(kNoRow, kNoRow);
  if (i >= m.n) return r;
  const int P = a.t.page_size;
  const int s = __ldg(m.keep + i);
  if (s < 0 || s >= m.len) {
    err |= kErrAppendLayout;
    return r;
  }
  if (s == i && !a.dst_indptr) return r;  // stays where it is
  const int sp = s / P, dp = i / P;
  const int from = __ldg(a.t.indices + m.page0 + sp), to = __ldg(m.dst + dp);
  if (from < 0 || from >= a.t.num_pages || to < 0 || to >= a.t.num_pages) {
    err |= kErrPageIndex;
    return r;
  }
  r.x = (static_cast<uint32_t>(from) * 2u * a.t.hkv + h) * P + (s - sp * P);
  r.y = (static_cast<uint32_t>(to) * 2u * a.t.hkv + h) * P + (i - dp * P);
  return r;
}

// ROW: bytes of a head row.
template <int ROW>
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ uint2 moves[4][kCmpThreads * kSteps / 2];  // two pieces of 16 bytes a row at least
  // Launched as a programmatic dependent of the kernel before it on the stream:
  // nothing global is touched before that grid has finished.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int list = blockIdx.x / a.roles, role = blockIdx.x - list * a.roles;
  const int b = list / a.t.hkv, h = list - b * a.t.hkv;
  Moves m;
  if (!moves_of(a, b, h, m)) {
    if (tid == 0) flag(a.t, kErrAppendLayout);
    return;
  }
  int err = 0;
  const uint32_t v_dist = static_cast<uint32_t>(a.t.hkv) * a.t.page_size;  // rows from a K row to its V row
  if (role < 2 * a.split * a.parts) {
    const int part = role % a.parts, piece = role / a.parts, which = piece / a.split, col = piece % a.split;
    const int width = ROW / a.split, per_row = width / 16, rows_step = kCmpThreads / per_row, round = rows_step * kSteps;
    const int my_row = tid / per_row, my_off = col * width + (tid % per_row) * 16;
    uint8_t* base = a.kv + (which ? static_cast<uint64_t>(v_dist) * ROW : 0) + my_off;
    const int rounds = (m.n + round - 1) / round;
    // Rounds part, part + parts, ...; the k-th of them uses moves[k % 4]
    // (round k + 2 is planned while slower threads still store round k - 1).
    auto plan = [&](int k) {
      const int64_t first = (part + static_cast<int64_t>(k) * a.parts) * round;
      for (int i = tid; i < round; i += kCmpThreads)
        moves[k % 4][i] = first + i < m.n ? move_of(a, m, static_cast<int>(first) + i, h, err) : make_uint2(kNoRow, kNoRow);
    };
    auto load = [&](int k, uint4 (&x)[kSteps]) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint32_t from = moves[k % 4][s * rows_step + my_row].x;
        if (from != kNoRow) x[s] = *reinterpret_cast<const uint4*>(base + static_cast<uint64_t>(from) * ROW);
      }
    };
    auto store = [&](int k, const uint4 (&x)[kSteps]) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint32_t to = moves[k % 4][s * rows_step + my_row].y;
        if (to != kNoRow) *reinterpret_cast<uint4*>(base + static_cast<uint64_t>(to) * ROW) = x[s];
      }
    };
    const int mine = rounds > part ? (rounds - part + a.parts - 1) / a.parts : 0;
    uint4 x[2][kSteps];
    if (mine > 0) plan(0);
    if (mine > 1) plan(1);
    __syncthreads();
    if (mine > 0) load(0, x[0]);
    for (int k = 0; k < mine; k += 2) {
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        if (k + o >= mine) break;
        if (k + o + 1 < mine) load(k + o + 1, x[(o + 1) & 1]);
        if (k + o + 2 < mine) plan(k + o + 2);
        // Every thread has read round k + o (and what the next round moves) before any writes it.
        __syncthreads();
        store(k + o, x[o]);
      }
    }
  } else {
    // Scales and weights: a thread is a row, kSteps rows a round.
    constexpr int kRound = kCmpThreads * kSteps;
    for (int64_t first = 0; first < m.n; first += kRound) {
      uint2 mv[kSteps];
      float w[kSteps];
      uint8_t ks[kSteps], vs[kSteps];
      uint32_t to_w[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int64_t i = first + s * kCmpThreads + tid;
        mv[s] = i < m.n ? move_of(a, m, static_cast<int>(i), h, err) : make_uint2(kNoRow, kNoRow);
        if (mv[s].x == kNoRow) continue;
        // A K row ((page 2 + 0) Hkv + h) P + slot is row (page Hkv + h) P + slot of the weights.
        const uint32_t sp = mv[s].x / (2 * v_dist), dp = mv[s].y / (2 * v_dist);
        to_w[s] = mv[s].y - dp * v_dist;
        if (a.weights) w[s] = a.weights[mv[s].x - sp * v_dist];
        if (a.scales) {
          ks[s] = a.scales[mv[s].x];
          vs[s] = a.scales[static_cast<uint64_t>(mv[s].x) + v_dist];
        }
      }
      __syncthreads();  // the round is read before any of it is written
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (mv[s].x == kNoRow) continue;
        if (a.weights) a.weights[to_w[s]] = w[s];
        if (a.scales) {
          a.scales[mv[s].y] = ks[s];
          a.scales[static_cast<uint64_t>(mv[s].y) + v_dist] = vs[s];
        }
      }
    }
  }
  if (err) flag(a.t, err);
}

template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kern)(Params...), int64_t clusters, int share, int block, int smem, cudaStream_t s,
                            const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * share));
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(share);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = share > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

pkv_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return PKV_OK;
  cudaGetLastError();
  return e == cudaErrorInvalidValue ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
}

bool sm_count(int& sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    return true;
  cudaGetLastError();
  return false;
}

// Sizes that both calls share.
pkv_status check_table(int batch, int hkv, int page_size, int64_t num_pages, int64_t kv_pages, int max_keep) {
  if (batch < 0 || hkv <= 0 || num_pages < 0 || kv_pages < 0 || max_keep < 0) return PKV_ERR_INVALID_ARG;
  if (page_size <= 0 || (page_size > 16 && page_size % 16)) return PKV_ERR_UNSUPPORTED;
  if (num_pages > INT32_MAX || kv_pages > INT32_MAX) return PKV_ERR_INVALID_ARG;
  if (hkv > (1 << 20) || page_size > (1 << 20)) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * hkv > INT32_MAX / 64) return PKV_ERR_UNSUPPORTED;  // CTAs of a grid
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_select_keys(int batch, int num_kv_heads, int page_size, int64_t num_pages, int64_t kv_pages,
                                      const int32_t* kv_indptr_d, const int32_t* kv_indices_d,
                                      const int32_t* kv_last_page_len_d, const float* weights, const int32_t* budget_d,
                                      int sink, int window, int max_keep, int32_t* keep, int32_t* kept_len_d,
                                      int32_t* error_d, void* stream) {
  using namespace pkv;
  pkv_status st = check_table(batch, num_kv_heads, page_size, num_pages, kv_pages, max_keep);
  if (st != PKV_OK) return st;
  if (sink < 0 || window < 0) return PKV_ERR_INVALID_ARG;
  if (batch == 0) return PKV_OK;
  if (!kv_indptr_d || !kv_last_page_len_d || !budget_d || !kept_len_d || (max_keep > 0 && !keep)) return PKV_ERR_INVALID_ARG;
  if (kv_pages > 0 && (!kv_indices_d || !weights)) return PKV_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(kv_indptr_d), static_cast<const void*>(kv_indices_d),
                        static_cast<const void*>(kv_last_page_len_d), static_cast<const void*>(weights),
                        static_cast<const void*>(budget_d), static_cast<const void*>(keep),
                        static_cast<const void*>(kept_len_d), static_cast<const void*>(error_d)})
    if (!aligned(p, 4)) return PKV_ERR_INVALID_ARG;
  int sms = 0;
  if (!sm_count(sms)) return PKV_ERR_CUDA;
  SelectArgs a{};
  a.t = Table{kv_indptr_d, kv_indices_d, kv_last_page_len_d, num_pages, kv_pages, batch, num_kv_heads, page_size, error_d};
  a.weights = weights;
  a.budget = budget_d;
  a.sink = sink;
  a.window = window;
  a.max_keep = max_keep;
  a.keep = keep;
  a.kept_len = kept_len_d;
  // Lists too few for the chip are shared by clusters, as long as a CTA has 1024 keys of a
  // list of average length.  Shared memory for twice that length, as far as it goes: longer
  // lists read the rest again.  256 threads where that is 6144 keys or fewer, so that the
  // lists of a serving batch run at once.
  const int64_t lists = static_cast<int64_t>(batch) * num_kv_heads, avg = kv_pages * page_size / batch;
  a.share = 1;
  while (a.share < 8 && lists * a.share * 2 <= 2 * sms && avg / (a.share * 2) >= 1024) a.share *= 2;
  const int64_t room = std::max<int64_t>(5 * avg / 4 / a.share, 20 * 1024);  // two CTAs an SM, or a quarter more than the average
  a.held = static_cast<int>(std::min<int64_t>(kMaxHeld, (std::max<int64_t>(std::min(2 * avg / a.share, room), 1024) + 35) & ~int64_t{31}));
  a.page_mul = page_size > 1 ? static_cast<uint32_t>(((int64_t{1} << 32) + page_size - 1) / page_size) : 0u;
  a.fours = page_size % 4 == 0 && aligned(weights, 16);
  auto s = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto kern, int threads) {
    cudaError_t e = ensure_smem_limit(kern, kMaxHeld * 4);
    return e == cudaSuccess ? launch_clusters(kern, lists, a.share, threads, a.held * 4, s, a) : e;
  };
  return status_of(a.held <= 6144 ? launch(select_keys_kernel<256>, 256) : launch(select_keys_kernel<512>, 512));
}

extern "C" pkv_status pkv_compact_paged_kv(const pkv_params* p, int batch, int64_t num_pages, int64_t kv_pages,
                                           const int32_t* kv_indptr_d, const int32_t* kv_indices_d,
                                           const int32_t* kv_last_page_len_d, int max_keep, const int32_t* keep,
                                           const int32_t* kept_len_d, int64_t dst_pages, const int32_t* dst_indptr_d,
                                           const int32_t* dst_indices_d, void* kv, uint8_t* kv8_scales, float* weights,
                                           int32_t* error_d, void* stream) {
  using namespace pkv;
  if (!p) return PKV_ERR_INVALID_ARG;
  pkv_status st = check_table(batch, p->num_kv_heads, p->page_size, num_pages, kv_pages, max_keep);
  if (st != PKV_OK) return st;
  if (p->head_dim != 64 && p->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (p->dtype != PKV_F16 && p->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (dst_pages < 0 || dst_pages > INT32_MAX || !dst_indptr_d != !dst_indices_d) return PKV_ERR_INVALID_ARG;
  // Rows of the pool are counted in 32 bits, with the last value for none.
  if (static_cast<double>(num_pages) * 2 * p->num_kv_heads * p->page_size >= 4294967295.0) return PKV_ERR_UNSUPPORTED;
  if (batch == 0 || max_keep == 0 || kv_pages == 0) return PKV_OK;
  if (!kv_indptr_d || !kv_indices_d || !kv_last_page_len_d || !keep || !kept_len_d || !kv) return PKV_ERR_INVALID_ARG;
  if (!aligned(kv, 16)) return PKV_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(kv_indptr_d), static_cast<const void*>(kv_indices_d),
                        static_cast<const void*>(kv_last_page_len_d), static_cast<const void*>(weights),
                        static_cast<const void*>(keep), static_cast<const void*>(kept_len_d),
                        static_cast<const void*>(dst_indptr_d), static_cast<const void*>(dst_indices_d),
                        static_cast<const void*>(error_d)})
    if (!aligned(x, 4)) return PKV_ERR_INVALID_ARG;
  int sms = 0;
  if (!sm_count(sms)) return PKV_ERR_CUDA;
  CompactArgs a{};
  a.t = Table{kv_indptr_d, kv_indices_d, kv_last_page_len_d, num_pages, kv_pages, batch, p->num_kv_heads, p->page_size, error_d};
  a.keep = keep;
  a.kept_len = kept_len_d;
  a.max_keep = max_keep;
  a.dst_indptr = dst_indptr_d;
  a.dst_indices = dst_indices_d;
  a.dst_pages = dst_pages;
  a.kv = static_cast<uint8_t*>(kv);
  a.scales = kv8_scales;
  a.weights = weights;
  const int row = p->head_dim * (kv8_scales ? 1 : 2);
  const int64_t lists = static_cast<int64_t>(batch) * p->num_kv_heads;
  // CTAs for the chip, two an SM at least: column slices in place, rounds of whole rows elsewhere.
  a.split = a.parts = 1;
  if (!dst_indptr_d) {
    while (a.split < row / 32 && lists * 2 * a.split < 2 * sms) a.split *= 2;
  } else {
    const int per_round = kCmpThreads * kSteps / (row / 16), rounds = max_keep / per_round + (max_keep % per_round != 0);
    while (a.parts < 16 && a.parts * 2 <= rounds && lists * 2 * a.parts < 4 * sms) a.parts *= 2;
  }
  a.roles = 2 * a.split * a.parts + (kv8_scales || weights ? 1 : 0);
  if (lists * a.roles > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const int grid = static_cast<int>(lists * a.roles);
  auto s = static_cast<cudaStream_t>(stream);
  cudaError_t e = row == 256   ? launch_dependent(compact_kernel<256>, grid, kCmpThreads, 0, s, a)
                  : row == 128 ? launch_dependent(compact_kernel<128>, grid, kCmpThreads, 0, s, a)
                               : launch_dependent(compact_kernel<64>, grid, kCmpThreads, 0, s, a);
  return status_of(e);
}
