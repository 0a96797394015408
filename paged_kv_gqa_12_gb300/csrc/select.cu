// Page selection: which pages of its context a query attends to.
//
// For query row r, kv head g, page p with key bounds lo, hi:
//   u(h, p) = sum_d max(q_d lo_d, q_d hi_d) = sum_{q_d > 0} q_d hi_d + sum_{q_d < 0} q_d lo_d
//   score(p) = max over the group's heads h of u(h, p)
// (no key of the page has a larger q . k), and the row takes its first and last
// pages and the best of the others.  With q+ = max(q, 0), q- = min(q, 0) the sums
// are a matrix product [lo | hi] . [q- | q+] over 2 D, which is what the score
// kernel computes; the bounds are its only large input and are read once per
// kv head and block of query rows.
//
// The chosen pages are those of the exact sums.  The tensor cores sum in 32
// bits: products of bf16 are exact there, each of the 2 D additions is off by at
// most 2^-22 of the largest partial sum (a factor of two above one truncated
// 24-bit addition), and every partial sum is at most |q|_1 A, A the largest
// bound in magnitude.  So |s - u| <= eps = D 2^-21 |q|_1 A, and against the K-th
// largest s, t, pages above t + 2 eps are in, pages below t - 2 eps are out, and
// only those between are summed again, in 64 bits.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "ptx.cuh"
#include "sparse.h"

namespace pa {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kListCap = 512;          // undecided pages ranked in shared memory

struct SelectParams {
  const uint16_t* q;
  int64_t q_stride_tok, q_stride_head;
  const uint16_t* bounds;
  int64_t bounds_stride_page, bounds_stride_head;
  int num_pages;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  const int32_t* qsl;
  int batch, num_kv_heads, group, cols, ps_log2;   // cols: score columns per token (>= group)
  int64_t max_len;
  int top, first, last;
  int row0, rows;             // query rows of this pass
  int block_rows;             // rows per score CTA
  int chunk_pages, n_chunks;  // pages per score CTA; chunk maxima per (row, kv head)
  float* scores;              // [rows of the pass, Hkv, row_pages]
  int row_pages;
  float* amax;                // [rows of the pass, Hkv, n_chunks]
  int32_t* pages;             // [rows, Hkv, top]
  uint32_t* err;
};

__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {   // magnitudes; signs are not meant
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float finite_or_inf(float s) { return fabsf(s) <= FLT_MAX ? s : INFINITY; }

// ---- scores -------------------------------------------------------------------
// One CTA = (page chunk, kv head, block of query rows).  A warp takes 16 pages as
// the M rows of its MMAs, their 2 D bounds loaded straight from global memory
// into A fragments: thread (g, c) of the fragment holds any four k-pairs of rows
// g and g + 8 as long as B agrees, so it takes 16 contiguous bytes for two
// k-steps, and the query coefficients in shared memory are read the same way.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const SelectParams p) {
  constexpr int K2 = 2 * D;
  constexpr int NP = K2 / 32;                 // 16-byte pieces per thread and row
  constexpr int QROW = K2 * 2 + 64;           // bytes of a query column: rows 64 bytes apart in the banks
  extern __shared__ __align__(16) uint8_t qs[];
  __shared__ float s_a[kScoreWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int kvh = blockIdx.y;
  const int chunk0 = blockIdx.z * p.chunk_pages;
  const int r_begin = p.row0 + blockIdx.x * p.block_rows;
  const int r_end = min(r_begin + p.block_rows, p.row0 + p.rows);
  const int G = p.group, C = p.cols;

  int row = r_begin;
  while (row < r_end) {
    // the rows of this block that belong to one request
    const RowPlace at = find_row<kScoreThreads>(p.seq_lens, p.qsl, p.batch, row, p.max_len);
    if (at.b < 0) break;                      // behind the last request
    const int stop = p.qsl != nullptr ? min(r_end, max(row + 1, p.qsl[at.b + 1])) : row + 1;
    const int first_row = row, m = stop - row;
    row = stop;
    if (at.bad) continue;                     // (reported by the selection kernel)
    // pages the block's last row can choose by score
    const int n = at.pos + m - 1 < 0 ? 0 : ((at.pos + m - 1) >> p.ps_log2) + 1;
    if (n <= p.top || chunk0 >= n - p.last) continue;
    const int end = min(chunk0 + p.chunk_pages, n - p.last);

    // [q- | q+] of every column (token, head); heads beyond the group repeat head
    // 0, which changes no maximum
    const int tiles = (m * C + 7) / 8;
    __syncthreads();
    for (int i = tid; i < tiles * 8 * (D / 8); i += kScoreThreads) {
      const int col = i / (D / 8), d = (i % (D / 8)) * 8;
      const int tok = col / C, j = col - tok * C;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (tok < m)
        w = *reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(first_row + tok) * p.q_stride_tok +
                                            static_cast<int64_t>(kvh * G + (j < G ? j : 0)) * p.q_stride_head + d);
      uint32_t x[4] = {w.x, w.y, w.z, w.w}, lo[4], hi[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // by sign bit; a NaN of either sign spoils its own half, which is enough
        const uint32_t neg = ((x[e] >> 15) & 0x00010001u) * 0xffffu;
        lo[e] = x[e] & neg;
        hi[e] = x[e] & ~neg;
      }
      uint8_t* dst = qs + col * QROW + d * 2;
      *reinterpret_cast<uint4*>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(dst + D * 2) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
    __syncthreads();

    const int32_t* bt = p.block_table + at.b * p.bt_stride;
    const int64_t out_row0 = (static_cast<int64_t>(first_row - p.row0) * p.num_kv_heads + kvh) * p.row_pages;
    const int64_t tok_stride = static_cast<int64_t>(p.num_kv_heads) * p.row_pages;
    float a_max = 0.f;
    for (int p0 = chunk0 + warp * 16; p0 < end; p0 += kScoreWarps * 16) {
      uint4 a[2][NP];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pg = p0 + g + 8 * h;
        int id = pg < end ? bt[pg] : -1;
        if (pg < end && static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
          if (c == 0) atomicOr(p.err, kErrPageId);
          id = -1;
        }
        const uint16_t* src = p.bounds + id * p.bounds_stride_page + kvh * p.bounds_stride_head + 8 * c;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          a[h][i] = id >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + 32 * i)) : make_uint4(0u, 0u, 0u, 0u);
      }
      // the largest finite bound (a page with another one has no finite score)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v = 0u;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          v = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(v, a[h][i].x), a[h][i].y), a[h][i].z),
                            a[h][i].w);
        v = absmax_bf16x2(v, v >> 16);
        v = absmax_bf16x2(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = absmax_bf16x2(v, __shfl_xor_sync(0xffffffffu, v, 2));
        const float f = __uint_as_float((v & 0x7fffu) << 16);
        if (f <= FLT_MAX) a_max = fmaxf(a_max, f);
      }
      float best[4];
      int tile_in_token = 0;
      for (int t = 0; t < tiles; ++t) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t* src = qs + (t * 8 + g) * QROW + 16 * c;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const uint4 b = *reinterpret_cast<const uint4*>(src + 64 * i);
          const uint32_t f0[4] = {a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y};
          const uint32_t f1[4] = {a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w};
          mma_bf16(d, f0, b.x, b.y);
          mma_bf16(d, f1, b.z, b.w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = finite_or_inf(d[e]);
        // columns 2c, 2c + 1 of pages g (d0, d1) and g + 8 (d2, d3)
        if (C == 1) {                          // every column is a token
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int pg = p0 + g + 8 * (e >> 1), tok = t * 8 + 2 * c + (e & 1);
            if (pg < end && tok < m) p.scores[out_row0 + tok * tok_stride + pg] = d[e];
          }
          continue;
        }
        float x = fmaxf(d[0], d[1]), y = fmaxf(d[2], d[3]);
        if (C >= 4) {
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
        }
        if (C >= 8) {
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
        }
        if (C > 8) {                           // a token of several tiles
          best[0] = tile_in_token == 0 ? x : fmaxf(best[0], x);
          best[1] = tile_in_token == 0 ? y : fmaxf(best[1], y);
          x = best[0];
          y = best[1];
          tile_in_token = tile_in_token + 1 == C / 8 ? 0 : tile_in_token + 1;
          if (tile_in_token != 0) continue;
        }
        const int tok = (t * 8 + 2 * c) / C;
        if (tok < m && (2 * c) % C == 0) {
          float* dst = p.scores + out_row0 + tok * tok_stride + p0 + g;
          if (p0 + g < end) dst[0] = x;
          if (p0 + g + 8 < end) dst[8] = y;
        }
      }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) a_max = fmaxf(a_max, __shfl_xor_sync(0xffffffffu, a_max, k));
    if (lane == 0) s_a[warp] = a_max;
    __syncthreads();
    if (tid < m) {
      float v = 0.f;
      for (int w = 0; w < kScoreWarps; ++w) v = fmaxf(v, s_a[w]);
      p.amax[(static_cast<int64_t>(first_row + tid - p.row0) * p.num_kv_heads + kvh) * p.n_chunks + blockIdx.z] = v;
    }
  }
}

// ---- selection ----------------------------------------------------------------

// Order-preserving map of a float (no NaN; -0 counts as 0) to unsigned.
__device__ __forceinline__ uint32_t key32(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_key32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key64(double f) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f + 0.0));
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

struct SelShared {
  uint32_t hist[256];
  uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
  uint32_t digit, left;
  int n_list;
  double value[kListCap];
  int index[kListCap];
};

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* tmp) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, k));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) v = max(v, tmp[w]);
  return v;
}
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* tmp) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) v += tmp[w];
  return v;
}

// The k-th largest (k >= 1) of the keys that get(i, &key) yields for i in [0, n),
// by 8 bits at a time from the top of the range they span.
template <class Get>
__device__ uint32_t kth_largest(SelShared& s, int n, uint32_t k, Get get) {
  const int tid = threadIdx.x;
  uint32_t top = 0, low_inv = 0;
  for (int i = tid; i < n; i += kSelThreads) {
    uint32_t key;
    if (!get(i, &key)) continue;
    top = max(top, key);
    low_inv = max(low_inv, ~key);
  }
  top = block_max(top, s.warp_a);
  const uint32_t low = ~block_max(low_inv, s.warp_b);
  const uint32_t span = top - low;
  int shift = span == 0 ? 0 : 32 - __clz(span);     // bits the range takes
  uint32_t prefix = 0;                              // of key - low, above `shift`
  while (shift > 0) {
    const int bits = min(8, shift);
    const int below = shift - bits;
    s.hist[tid] = 0;                                // (256 threads, 256 bins)
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      uint32_t key;
      if (!get(i, &key)) continue;
      const uint32_t x = key - low;
      if ((shift < 32 ? x >> shift : 0u) == prefix) atomicAdd(&s.hist[(x >> below) & ((1u << bits) - 1u)], 1u);
    }
    __syncthreads();
    // count of the bins above each: thread t takes bin 255 - t
    uint32_t mine = s.hist[255 - tid], sum = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, m);
      if ((tid & 31) >= m) sum += v;
    }
    if ((tid & 31) == 31) s.warp_a[tid >> 5] = sum;
    __syncthreads();
    for (int w = 0; w < (tid >> 5); ++w) sum += s.warp_a[w];
    if (sum >= k && sum - mine < k) {               // exactly one bin
      s.digit = 255 - tid;
      s.left = k - (sum - mine);
    }
    __syncthreads();
    prefix = (prefix << bits) | s.digit;
    k = s.left;
    shift = below;
    __syncthreads();
  }
  return low + prefix;
}

// Exact score of a page for the group, in 64 bits, by one warp.
template <int D>
__device__ double exact_score(const SelectParams& p, const int32_t* bt, int row, int kvh, int page) {
  constexpr int V = D / 32;                          // dims per lane
  const int lane = threadIdx.x & 31;
  const int id = bt[page];
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) return 0.0;
  const uint16_t* lo = p.bounds + id * p.bounds_stride_page + kvh * p.bounds_stride_head + lane * V;
  float l[V], h[V];
  bool odd = false;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    l[e] = bf16_to_f32(lo[e]);
    h[e] = bf16_to_f32(lo[D + e]);
    odd |= !(fabsf(l[e]) <= FLT_MAX) || !(fabsf(h[e]) <= FLT_MAX);
  }
  if (__any_sync(0xffffffffu, odd)) return INFINITY;
  double best = -INFINITY;
  for (int j = 0; j < p.group; ++j) {
    const uint16_t* q = p.q + static_cast<int64_t>(row) * p.q_stride_tok +
                        static_cast<int64_t>(kvh * p.group + j) * p.q_stride_head + lane * V;
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float x = bf16_to_f32(q[e]);
      sum += static_cast<double>(x) * static_cast<double>(x < 0.f ? l[e] : h[e]);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (!(fabs(sum) <= DBL_MAX)) sum = INFINITY;
    best = fmax(best, sum);
  }
  return best;
}

// One CTA = one (query row, kv head).  Which pages are chosen, and which are
// still undecided, is kept as bit maps in shared memory; the chosen ones are
// written out in ascending order at the end.
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t bits[];                 // chosen, then undecided
  __shared__ SelShared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = p.row0 + blockIdx.x;
  const int kvh = blockIdx.y;
  const RowPlace at = find_row<kSelThreads>(p.seq_lens, p.qsl, p.batch, row, p.max_len);
  if (at.b < 0) return;
  if (at.bad) {
    if (tid == 0) atomicOr(p.err, kErrCapacity);
    return;
  }
  const int n = at.pos < 0 ? 0 : (at.pos >> p.ps_log2) + 1;
  int32_t* out = p.pages + (static_cast<int64_t>(row) * p.num_kv_heads + kvh) * p.top;
  if (n <= p.top) {                                  // every page
    for (int i = tid; i < p.top; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int words = (n + 31) / 32;
  uint32_t* chosen = bits;
  uint32_t* open = bits + words;
  const int32_t* bt = p.block_table + at.b * p.bt_stride;
  const int64_t cell = static_cast<int64_t>(row - p.row0) * p.num_kv_heads + kvh;
  float* score = p.scores + cell * p.row_pages;
  const int lo = p.first, hi = n - p.last;           // pages chosen by score: [lo, hi)
  const uint32_t want = p.top - p.first - p.last;    // (n > top, so hi - lo > want)

  float above = INFINITY, below = INFINITY;          // scores beyond decide; [below, above] is open
  bool all_open = false, ties = true;                // ties: what is open is exactly equal
  if (want > 0) {
    // eps of this row
    float q1 = 0.f;
    for (int j = warp; j < p.group; j += kSelWarps) {
      const uint16_t* q = p.q + static_cast<int64_t>(row) * p.q_stride_tok +
                          static_cast<int64_t>(kvh * p.group + j) * p.q_stride_head;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) sum += fabsf(bf16_to_f32(q[lane + 32 * e]));
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      q1 = sum > q1 || sum != sum ? sum : q1;
    }
    // (non-negative floats order as integers, a NaN above them all)
    q1 = __uint_as_float(block_max(__float_as_uint(q1) & 0x7fffffffu, s.warp_a));
    float am = 0.f;
    const int chunks = (hi + p.chunk_pages - 1) / p.chunk_pages;
    for (int i = tid; i < chunks; i += kSelThreads) am = fmaxf(am, p.amax[cell * p.n_chunks + i]);
    am = __uint_as_float(block_max(__float_as_uint(am), s.warp_b));
    // |q|_1 itself is summed in 32 bits: a hundredth more covers it; sums below
    // the normal range may be flushed: 2 D times the smallest normal covers them.
    // A q that is not finite gives every page +infinity, a zero one zero: exact.
    const float size = q1 * am;
    const float eps = !(q1 <= FLT_MAX) || q1 == 0.f || am == 0.f ? 0.f
                      : size <= FLT_MAX ? 1.01f * (D * 0x1p-21f) * size + 2 * D * FLT_MIN : INFINITY;

    const uint32_t kth = kth_largest(s, hi - lo, want, [&](int i, uint32_t* key) {
      *key = key32(score[lo + i]);
      return true;
    });
    const float t = from_key32(kth);
    all_open = !(eps <= FLT_MAX);
    ties = !all_open && (eps == 0.f || t == INFINITY);
    above = __fadd_ru(t, 2.f * eps);
    below = __fadd_rd(t, -2.f * eps);
  }

  // decide what 32 bits can
  if (tid == 0) s.n_list = 0;
  __syncthreads();
  uint32_t decided = 0, n_open = 0;
  for (int w = warp; w < words; w += kSelWarps) {
    const int i = w * 32 + lane;
    bool in = i < n && (i < lo || i >= hi), maybe = false;
    bool scored = false;
    if (want > 0 && i >= lo && i < hi) {
      const float x = score[i];
      scored = !all_open && x > above;
      maybe = all_open || (!scored && x >= below);
      in |= scored;
    }
    const uint32_t in_w = __ballot_sync(0xffffffffu, in), open_w = __ballot_sync(0xffffffffu, maybe);
    const uint32_t scored_w = __ballot_sync(0xffffffffu, scored);
    if (lane == 0) {
      chosen[w] = in_w;
      open[w] = open_w;
      decided += __popc(scored_w);
      n_open += __popc(open_w);
    }
  }
  decided = block_sum(decided, s.warp_a);
  n_open = block_sum(n_open, s.warp_b);
  uint32_t need = want - decided;                    // to take from the open ones

  if (need > 0 && need < n_open && !ties) {
    if (n_open <= kListCap) {
      // rank them by their exact scores
      for (int w = tid; w < words; w += kSelThreads)
        for (uint32_t m = open[w]; m != 0; m &= m - 1) s.index[atomicAdd(&s.n_list, 1)] = w * 32 + __ffs(m) - 1;
      __syncthreads();
      for (int i = warp; i < static_cast<int>(n_open); i += kSelWarps) {
        const double v = exact_score<D>(p, bt, row, kvh, s.index[i]);
        if (lane == 0) s.value[i] = v;
      }
      __syncthreads();
      for (int i = tid; i < static_cast<int>(n_open); i += kSelThreads) {
        const double v = s.value[i];
        const int page = s.index[i];
        uint32_t better = 0;
        for (int j = 0; j < static_cast<int>(n_open); ++j)
          better += s.value[j] > v || (s.value[j] == v && s.index[j] < page);
        if (better < need) atomicOr(&chosen[page >> 5], 1u << (page & 31));
      }
      need = 0;
    } else {
      // too many to rank: the need-th largest exact score by its upper, then its
      // lower 32 bits, kept in place of the 32-bit scores
      for (int half = 0; half < 2 && need > 0; ++half) {
        for (int w = warp; w < words; w += kSelWarps)
          for (uint32_t m = open[w]; m != 0; m &= m - 1) {
            const int i = w * 32 + __ffs(m) - 1;
            const uint64_t k = key64(exact_score<D>(p, bt, row, kvh, i));
            if (lane == 0) score[i] = __uint_as_float(static_cast<uint32_t>(half == 0 ? k >> 32 : k));
          }
        __syncthreads();
        const uint32_t kth = kth_largest(s, n, need, [&](int i, uint32_t* key) {
          *key = __float_as_uint(score[i]);
          return (open[i >> 5] >> (i & 31) & 1u) != 0;
        });
        uint32_t taken = 0;
        __syncthreads();
        for (int w = tid; w < words; w += kSelThreads) {
          uint32_t win = 0, stay = 0;
          for (uint32_t m = open[w]; m != 0; m &= m - 1) {
            const int b = __ffs(m) - 1;
            const uint32_t key = __float_as_uint(score[w * 32 + b]);
            win |= (key > kth ? 1u : 0u) << b;
            stay |= (key == kth ? 1u : 0u) << b;
          }
          chosen[w] |= win;
          open[w] = stay;
          taken += __popc(win);
        }
        need -= block_sum(taken, s.warp_a);
      }
    }
  }
  __syncthreads();

  // the lowest `need` of what is still open are equal to the border: take them;
  // then write the chosen pages in order.  Thread t holds words [t per, (t+1) per).
  const int per = (words + kSelThreads - 1) / kSelThreads;
  auto scan = [&](uint32_t v) {                      // sum over the threads before this one
    uint32_t sum = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, m);
      if (lane >= m) sum += x;
    }
    __syncthreads();
    if (lane == 31) s.warp_a[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += s.warp_a[w];
    return sum - v;
  };
  if (need > 0) {
    uint32_t mine = 0;
    for (int w = tid * per; w < min((tid + 1) * per, words); ++w) mine += __popc(open[w]);
    uint32_t before = scan(mine);
    for (int w = tid * per; w < min((tid + 1) * per, words); ++w)
      for (uint32_t m = open[w]; m != 0 && before < need; m &= m - 1, ++before) chosen[w] |= m & (0u - m);
  }
  uint32_t mine = 0;
  for (int w = tid * per; w < min((tid + 1) * per, words); ++w) mine += __popc(chosen[w]);
  uint32_t at_out = scan(mine);
  for (int w = tid * per; w < min((tid + 1) * per, words); ++w)
    for (uint32_t m = chosen[w]; m != 0 && at_out < static_cast<uint32_t>(p.top); m &= m - 1)
      out[at_out++] = w * 32 + __ffs(m) - 1;
}

template <int D>
cudaError_t launch(const SelectParams& p, int chunks, cudaStream_t st) {
  const int tiles = (p.block_rows * p.cols + 7) / 8;
  const int smem = tiles * 8 * (4 * D + 64);
  cudaError_t e = cudaFuncSetAttribute(score_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (chunks > 0) {
    const dim3 grid((p.rows + p.block_rows - 1) / p.block_rows, p.num_kv_heads, chunks);
    score_kernel<D><<<grid, kScoreThreads, smem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const dim3 grid(p.rows, p.num_kv_heads);
  select_kernel<D><<<grid, kSelThreads, p.row_pages / 32 * 8, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_select_pages(const pa_sparse_plan_t* plan, const void* q, int64_t q_stride_tok,
                                     int64_t q_stride_head, const void* bounds, int64_t bounds_stride_page,
                                     int64_t bounds_stride_head, int32_t num_pages, const int32_t* block_table,
                                     int64_t bt_stride, const int32_t* seq_lens, const int32_t* query_start_loc,
                                     int32_t batch, int32_t total_q, int32_t* pages, void* scratch,
                                     int64_t scratch_bytes, void* stream) {
  const pa_status st = check_sparse_call(plan, block_table, bt_stride, seq_lens, query_start_loc, batch, total_q,
                                         scratch, scratch_bytes);
  if (st != PA_OK) return st;
  if (batch == 0 || total_q == 0) return PA_OK;
  const pa_sparse_shape& s = plan->shape;
  if (!q || !bounds || !pages || num_pages <= 0) return PA_ERR_INVALID_ARG;
  if (q_stride_tok <= 0 || q_stride_head <= 0 || bounds_stride_page <= 0 || bounds_stride_head <= 0)
    return PA_ERR_INVALID_ARG;
  auto at = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0; };
  if (!at(q, 16) || q_stride_tok % 8 || q_stride_head % 8 || !at(bounds, 16) || bounds_stride_page % 8 ||
      bounds_stride_head % 8 || !at(pages, 4))
    return PA_ERR_UNSUPPORTED;
  SelectParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.bounds = static_cast<const uint16_t*>(bounds);
  p.bounds_stride_page = bounds_stride_page;
  p.bounds_stride_head = bounds_stride_head;
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.batch = batch;
  p.num_kv_heads = s.num_kv_heads;
  p.group = s.num_q_heads / s.num_kv_heads;
  // columns per token: the group rounded up to a divisor or a multiple of 8
  p.cols = p.group > 8 ? (p.group + 7) / 8 * 8 : p.group > 4 ? 8 : p.group > 2 ? 4 : p.group;
  p.ps_log2 = __builtin_ctz(static_cast<unsigned>(s.page_size));
  p.max_len = static_cast<int64_t>(s.max_pages_per_seq) * s.page_size;
  p.top = s.top_pages;
  p.first = s.first_pages;
  p.last = s.last_pages;
  p.row_pages = static_cast<int>(score_pages(s));
  p.n_chunks = static_cast<int>(score_chunks(s));
  p.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + kScratchHeaderBytes);
  p.err = static_cast<uint32_t*>(scratch);
  // rows per score CTA: one for decode; for chunks as many as a request brings on
  // average, up to 64 columns
  int block = 1;
  if (query_start_loc != nullptr) {
    const int each = (total_q + batch - 1) / batch;
    while (block < each && block * 2 * p.cols <= 64) block *= 2;
  }
  p.block_rows = block;
  // pages per score CTA: as many as leave about eight CTAs per SM
  const int64_t blocks = static_cast<int64_t>((std::min(total_q, plan->score_rows) + block - 1) / block);
  const int64_t pages_all = blocks * s.num_kv_heads * p.row_pages;
  int64_t chunk = kScorePagesMin;
  while (chunk * 2 <= 1024 && pages_all / (chunk * 2) >= static_cast<int64_t>(s.num_sms) * 8) chunk *= 2;
  p.chunk_pages = static_cast<int>(chunk);
  // a capacity of no more than top_pages pages needs no scores
  const int chunks = s.max_pages_per_seq <= s.top_pages || s.top_pages == s.first_pages + s.last_pages
                         ? 0
                         : static_cast<int>((p.row_pages + chunk - 1) / chunk);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  for (int r = 0; r < total_q; r += plan->score_rows) {
    p.row0 = r;
    p.rows = std::min(plan->score_rows, total_q - r);
    p.amax = p.scores + sparse_score_bytes(s, p.rows) / 4 -
             (static_cast<int64_t>(p.rows) * s.num_kv_heads * score_chunks(s) * 4 + 255) / 256 * 64;
    p.pages = pages;
    cudaError_t e;
    switch (s.head_dim) {
      case 64: e = launch<64>(p, chunks, str); break;
      case 128: e = launch<128>(p, chunks, str); break;
      default: e = launch<256>(p, chunks, str); break;
    }
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}
