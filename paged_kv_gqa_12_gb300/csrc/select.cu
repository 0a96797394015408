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
// bits: products of bf16 are exact there, one of a dim's two products is zero,
// and each of the other D, with the 2 D / 16 running sums they are added to, is
// taken to be off by at most 2^-23 of the largest partial sum; that is at most |q|_1 A,
// A the largest bound in magnitude.  That a term aligned to the largest of its sum
// keeps these 24 bits is an assumption on the hardware, nowhere documented; measured
// on random sums, one large dim beside small ones, sums that cancel and all magnitudes
// mixed (D 64 to 256, 3 million scores), |s - u| was at most 1.8 x 2^-23 |q|_1 A, 0.6 %
// of the band that follows from it: |s - u| <= eps = D 2^-22 |q|_1 A.  Against
// the K-th largest s, t, pages above t + 2 eps are in, pages below t - 2 eps are
// out, and only those between are summed again, to more than 64-bit precision.
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

// |q|_1 is summed times this: 256 bf16 of any size stay below the largest float.
constexpr float kQScale = 0x1p-8f;

// Selection by T threads a row: scores kept per thread, steps of the score
// histogram, undecided pages ranked in shared memory.
template <int T>
struct Sel {
  static constexpr int kBins = T == 32 ? 256 : T <= 256 ? 1024 : 2048;
  static constexpr int kListCap = 2 * T < 512 ? 2 * T : 512;
};

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
  int batch, num_kv_heads, group, hpt, ps_log2;   // hpt: heads of a token in a score tile (1, 2, 4, 8)
  int64_t max_len;
  int top, first, last;
  int row0, rows;             // query rows of this pass
  int num_sms;
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
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// A sum that is not finite becomes NaN, which max_nan carries to the end.
__device__ __forceinline__ float nan_if_infinite(float s) { return fmaf(s, 0.f, s); }
__device__ __forceinline__ float inf_if_nan(float s) { return s == s ? s : INFINITY; }

// Two bf16 split by sign bit into the factors of the lower and of the upper
// bounds; a NaN of either sign spoils its own half, which is enough.
__device__ __forceinline__ uint32_t sign_mask(uint32_t x) {   // 0xffff where a bf16 is negative
  uint32_t m;
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(m) : "r"(x));
  return m;
}
__device__ __forceinline__ uint32_t negatives(uint32_t x) { return x & sign_mask(x); }
__device__ __forceinline__ uint32_t positives(uint32_t x) { return x & ~sign_mask(x); }
__device__ __forceinline__ uint4 negatives(uint4 x) {
  return make_uint4(negatives(x.x), negatives(x.y), negatives(x.z), negatives(x.w));
}
__device__ __forceinline__ uint4 positives(uint4 x) {
  return make_uint4(positives(x.x), positives(x.y), positives(x.z), positives(x.w));
}

// ---- scores -------------------------------------------------------------------
// A warp takes 16 pages as the M rows of its MMAs and up to 8 query columns as N.
// Thread (g, c) of an A fragment holds any four k-pairs of pages g and g + 8 as
// long as B agrees, so it takes 16 contiguous bytes of bounds for two k-steps, and
// the query factors are read the same way.

// The largest magnitude of a page's bounds over the four lanes of its row (0 where
// one is not finite: such a page has no finite score).
__device__ __forceinline__ float row_amax(uint32_t v) {
  v = absmax_bf16x2(v, v >> 16);
  v = absmax_bf16x2(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = absmax_bf16x2(v, __shfl_xor_sync(0xffffffffu, v, 2));
  const float f = __uint_as_float((v & 0x7fffu) << 16);
  return f <= FLT_MAX ? f : 0.f;
}
__device__ __forceinline__ uint32_t fold_abs(uint32_t v, const uint4& x) {
  return absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(v, x.x), x.y), x.z), x.w);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// One query row of at most 8 heads (decode): one CTA = (row, kv head, page chunk).
// The kernel is the stream of the bounds: a page's 4 D bytes of a kv head are one
// bulk copy, 16 of them a stage, each warp with a ring of its own, so that an SM
// has some 200 KB on the way and no warp waits for another.  Query column g (head
// g, or head 0 again: the same maximum) stays in registers.
template <int D>
struct One {
  static constexpr int NS = D == 64 ? 2 : 1;          // stages a warp
  static constexpr int ROW = 4 * D + 64;              // bytes from page to page: free of bank conflicts
  static constexpr int STAGE = 16 * ROW;
  static constexpr int SMEM = kScoreWarps * NS * (STAGE + 8);
};
template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_one_kernel(const SelectParams p) {
  using O = One<D>;
  constexpr int NP = 2 * D / 32;              // 16-byte pieces per thread and row
  constexpr int kStep = kScoreWarps * 16;
  extern __shared__ __align__(16) uint8_t rings[];
  __shared__ float s_a[kScoreWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int r = blockIdx.x / p.num_kv_heads;
  const int kvh = blockIdx.x - r * p.num_kv_heads;
  const int chunk0 = blockIdx.y * p.chunk_pages;
  const int row = p.row0 + r;
  pdl_launch_dependents();   // the selection may start up; it waits for this grid's scores

  uint64_t* bar = reinterpret_cast<uint64_t*>(rings + kScoreWarps * O::NS * O::STAGE) + warp * O::NS;
  const uint32_t ring = smem_u32(rings + warp * O::NS * O::STAGE);
  if (lane == 0) {
    for (int s = 0; s < O::NS; ++s) mbar_init(&bar[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const RowPlace at = find_row<kScoreThreads>(p.seq_lens, p.qsl, p.batch, row, p.max_len);
  if (at.b < 0 || at.bad) return;             // (a bad one is reported by the selection kernel)
  const int n = at.pos < 0 ? 0 : (at.pos >> p.ps_log2) + 1;
  if (n <= p.top || chunk0 >= n - p.last) return;
  const int end = min(chunk0 + p.chunk_pages, n - p.last);

  // lane i < 16 copies page p0 + i; one behind the chunk's end repeats its last, one
  // outside the pool reads page 0 and scores 0
  const int32_t* bt = p.block_table + at.b * p.bt_stride;
  const uint8_t* base = reinterpret_cast<const uint8_t*>(p.bounds + kvh * p.bounds_stride_head);
  const int64_t page_bytes = p.bounds_stride_page * 2;
  uint32_t lost[O::NS];
  auto page_id = [&](int p0) { return bt[min(p0 + (lane & 15), end - 1)]; };
  auto issue = [&](int id, int s) {
    const bool out = static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages);
    lost[s] = __ballot_sync(0xffffffffu, out);
    if (lost[s] != 0 && lane == 0) atomicOr(p.err, kErrPageId);
    if (lane == 0) mbar_arrive_expect_tx(&bar[s], 16 * 4 * D);
    __syncwarp();
    if (lane < 16)
      bulk_load(ring + s * O::STAGE + lane * O::ROW, base + (out ? 0 : id) * page_bytes, 4 * D, &bar[s]);
  };
  int p_next = chunk0 + warp * 16;            // of the next stage to fill
  int id = page_id(p_next);
#pragma unroll
  for (int s = 0; s < O::NS; ++s) {
    if (p_next < end) issue(id, s);
    p_next += kStep;
    id = page_id(p_next);
  }

  uint4 q[NP / 2];
  const uint16_t* qh = p.q + static_cast<int64_t>(row) * p.q_stride_tok +
                       static_cast<int64_t>(kvh * p.group + (g < p.group ? g : 0)) * p.q_stride_head + 8 * c;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) q[i] = *reinterpret_cast<const uint4*>(qh + 32 * i);

  float* out_row = p.scores + (static_cast<int64_t>(r) * p.num_kv_heads + kvh) * p.row_pages;
  float a_max = 0.f;
  int it = 0;
  for (int p0 = chunk0 + warp * 16; p0 < end; p0 += kStep, ++it) {
    const int s = it % O::NS;
    if (!__all_sync(0xffffffffu, mbar_wait(&bar[s], (it / O::NS) & 1, p.err))) {
      // give up (the error word says so), but not before the other stage's copies had their time to land
      if (O::NS > 1 && p0 + kStep < end) mbar_wait(&bar[(it + 1) % O::NS], ((it + 1) / O::NS) & 1, p.err);
      break;
    }
    const uint8_t* src = rings + (warp * O::NS + s) * O::STAGE + g * O::ROW + 16 * c;
    // (two independent sums: one after the other they would wait on each MMA's latency)
    float d[2][4] = {};
    uint32_t v0 = 0u, v1 = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NP / 2; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + (h * (NP / 2) + i) * 64);
        const uint4 y = *reinterpret_cast<const uint4*>(src + 8 * O::ROW + (h * (NP / 2) + i) * 64);
        const uint4 b = h == 0 ? negatives(q[i]) : positives(q[i]);
        const uint32_t f0[4] = {x.x, y.x, x.y, y.y}, f1[4] = {x.z, y.z, x.w, y.w};
        mma_bf16(d[i & 1], f0, b.x, b.y);
        mma_bf16(d[i & 1], f1, b.z, b.w);
        v0 = fold_abs(v0, x);
        v1 = fold_abs(v1, y);
      }
    const uint32_t gone = lost[O::NS == 1 ? 0 : s];
    __syncwarp();
    if (p_next < end) {                       // the stage is read: refill it
      fence_proxy_async_smem();
      issue(id, s);
    }
    p_next += kStep;
    id = page_id(p_next);
    a_max = fmaxf(a_max, fmaxf(row_amax(v0), row_amax(v1)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // columns 2c and 2c + 1 of page g + 8 h
      float x = max_nan(nan_if_infinite(d[0][2 * h] + d[1][2 * h]), nan_if_infinite(d[0][2 * h + 1] + d[1][2 * h + 1]));
      x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 2));
      const int pg = p0 + g + 8 * h;
      if (c == 0 && pg < end) out_row[pg] = (gone >> (g + 8 * h) & 1u) ? 0.f : inf_if_nan(x);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) a_max = fmaxf(a_max, __shfl_xor_sync(0xffffffffu, a_max, k));
  if (lane == 0) s_a[warp] = a_max;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kScoreWarps; ++w) a_max = fmaxf(a_max, s_a[w]);
    p.amax[(static_cast<int64_t>(r) * p.num_kv_heads + kvh) * p.n_chunks + blockIdx.y] = a_max;
  }
}

// Blocks of query rows, or rows of more heads: one CTA = (row block, kv head, page
// chunk).  The bounds are read through L2 by every block, so they go straight
// from global memory into A fragments; the factors of the block's rows lie in
// shared memory: a tile of 8 columns holds `hpt` heads of 8 / hpt tokens, the
// group's heads run over the tiles of a token group, and their maximum is taken
// in registers (and over the hpt columns by shuffles, none from 8 tokens on).
template <int D>
__global__ void __launch_bounds__(kScoreThreads, D == 256 ? 2 : 4) score_block_kernel(const SelectParams p) {
  constexpr int K2 = 2 * D;
  constexpr int NP = K2 / 32;                 // 16-byte pieces per thread and row
  constexpr int QROW = K2 * 2 + 64;           // bytes of a query column: rows 64 bytes apart in the banks
  extern __shared__ __align__(16) uint8_t qs[];
  __shared__ float s_a[kScoreWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int block = blockIdx.x / p.num_kv_heads;
  const int kvh = blockIdx.x - block * p.num_kv_heads;
  const int chunk0 = blockIdx.y * p.chunk_pages;
  const int r_begin = p.row0 + block * p.block_rows;
  const int r_end = min(r_begin + p.block_rows, p.row0 + p.rows);
  const int G = p.group;
  pdl_launch_dependents();

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
    const int32_t* bt = p.block_table + at.b * p.bt_stride;
    const uint16_t* q0 = p.q + static_cast<int64_t>(first_row) * p.q_stride_tok +
                         static_cast<int64_t>(kvh * G) * p.q_stride_head;

    // pool pages of fragment rows g and g + 8; pages behind the chunk's end repeat
    // its last one, a page outside the pool reads page 0 and scores 0
    int id[2];
    bool lost[2];
    auto page_ids = [&](int p0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) id[h] = bt[min(p0 + g + 8 * h, end - 1)];
    };
    page_ids(chunk0 + warp * 16);

    const int tpt = 8 / p.hpt;
    const int groups = (m + tpt - 1) / tpt, head_tiles = (G + p.hpt - 1) / p.hpt;
    __syncthreads();
    for (int i = tid; i < groups * head_tiles * 8 * (D / 8); i += kScoreThreads) {
      const int col = i / (D / 8), d = (i % (D / 8)) * 8;
      const int tile = col >> 3, tg = tile / head_tiles;
      const int tok = tg * tpt + (col & 7) / p.hpt;
      const int head = (tile - tg * head_tiles) * p.hpt + (col & (p.hpt - 1));
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (tok < m)                            // heads beyond the group repeat head 0: the same maximum
        x = *reinterpret_cast<const uint4*>(q0 + tok * p.q_stride_tok +
                                            static_cast<int64_t>(head < G ? head : 0) * p.q_stride_head + d);
      *reinterpret_cast<uint4*>(qs + col * QROW + d * 2) = negatives(x);
      *reinterpret_cast<uint4*>(qs + col * QROW + (D + d) * 2) = positives(x);
    }
    __syncthreads();

    const int64_t out_row0 = (static_cast<int64_t>(first_row - p.row0) * p.num_kv_heads + kvh) * p.row_pages;
    const int64_t tok_stride = static_cast<int64_t>(p.num_kv_heads) * p.row_pages;
    float a_max = 0.f;
    for (int p0 = chunk0 + warp * 16; p0 < end; p0 += kScoreWarps * 16) {
      uint4 a[2][NP];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lost[h] = static_cast<unsigned>(id[h]) >= static_cast<unsigned>(p.num_pages);
        const uint16_t* src = p.bounds + (lost[h] ? 0 : id[h]) * p.bounds_stride_page +
                              kvh * p.bounds_stride_head + 8 * c;
#pragma unroll
        for (int i = 0; i < NP; ++i) a[h][i] = __ldg(reinterpret_cast<const uint4*>(src + 32 * i));
      }
      if (lost[0] || lost[1]) atomicOr(p.err, kErrPageId);
      page_ids(p0 + kScoreWarps * 16);        // (of the next pages)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v = 0u;
#pragma unroll
        for (int i = 0; i < NP; ++i) v = fold_abs(v, a[h][i]);
        a_max = fmaxf(a_max, row_amax(v));
      }
      for (int tg = 0; tg < groups; ++tg) {
        // columns 2c, 2c + 1 of pages g (0, 1) and g + 8 (2, 3); several tiles side by
        // side: one after the other their sums would wait on each MMA's latency
        float best[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        constexpr int U = 4;
        const uint8_t* src0 = qs + (tg * head_tiles * 8 + g) * QROW + 16 * c;
        for (int ht = 0; ht < head_tiles; ht += U) {
          float d[U][4] = {};
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const uint32_t f0[4] = {a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y};
            const uint32_t f1[4] = {a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w};
#pragma unroll
            for (int u = 0; u < U; ++u) {     // (tiles beyond the last repeat it)
              const uint4 b = *reinterpret_cast<const uint4*>(src0 + min(ht + u, head_tiles - 1) * 8 * QROW + 64 * i);
              mma_bf16(d[u], f0, b.x, b.y);
              mma_bf16(d[u], f1, b.z, b.w);
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) best[e] = max_nan(best[e], nan_if_infinite(d[u][e]));
        }
        auto store = [&](int tok, int h, float s) {
          const int pg = p0 + g + 8 * h;
          if (tok < m && pg < end) p.scores[out_row0 + tok * tok_stride + pg] = lost[h] ? 0.f : inf_if_nan(s);
        };
        if (p.hpt == 1) {                     // a column is a token
#pragma unroll
          for (int e = 0; e < 4; ++e) store(tg * 8 + 2 * c + (e & 1), e >> 1, best[e]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = max_nan(best[2 * h], best[2 * h + 1]);
            if (p.hpt >= 4) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 1));
            if (p.hpt >= 8) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 2));
            if ((2 * c & (p.hpt - 1)) == 0) store(tg * tpt + 2 * c / p.hpt, h, x);
          }
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
      p.amax[(static_cast<int64_t>(first_row + tid - p.row0) * p.num_kv_heads + kvh) * p.n_chunks + blockIdx.y] = v;
    }
  }
}

// ---- selection ----------------------------------------------------------------

__device__ __forceinline__ uint64_t key64(double f) {   // order-preserving; -0 counts as 0
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f + 0.0));
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// The power of two that brings a positive finite x into [1, 2), within the normal
// range (a zero or infinite x: any).
__device__ __forceinline__ float inverse_power(float x) {
  const int e = static_cast<int>(__float_as_uint(x) >> 23);          // biased exponent
  return __uint_as_float(static_cast<uint32_t>(min(max(254 - e, 1), 254)) << 23);
}

template <int T>
struct SelShared {
  static constexpr int kBins = Sel<T>::kBins, kListCap = Sel<T>::kListCap;
  uint32_t hist[kBins];
  float red[4][32];
  uint32_t warp_sum[32];
  uint32_t infs, decided, n_open, digit, left;
  double value[kListCap];
  int index[kListCap];
};

// Over the CTA: the maximum of each of N values (T threads; every thread gets it).
template <int T, int N>
__device__ __forceinline__ void block_max(float (&v)[N], SelShared<T>& s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) v[i] = fmaxf(v[i], __shfl_xor_sync(0xffffffffu, v[i], k));
  if constexpr (T == 32) {
    __syncthreads();
  } else {
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s.red[i][threadIdx.x >> 5] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = s.red[i][lane & (T / 32 - 1)];
#pragma unroll
      for (int k = T / 64; k > 0; k >>= 1) v[i] = fmaxf(v[i], __shfl_xor_sync(0xffffffffu, v[i], k));
    }
  }
}

// Sum of v over the threads before this one.
template <int T>
__device__ __forceinline__ uint32_t sum_before(uint32_t v, SelShared<T>& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t sum = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, sum, m);
    if (lane >= m) sum += x;
  }
  if constexpr (T == 32) return sum - v;
  __syncthreads();
  if (lane == 31) s.warp_sum[warp] = sum;
  __syncthreads();
  for (int w = 0; w < warp; ++w) sum += s.warp_sum[w];
  return sum - v;
}

// The bin of s.hist[0 .. n_bins) (n_bins a multiple of T or half of it) that
// holds the k-th largest, into s.digit, and its rank within the bin, into s.left.
template <int T>
__device__ __forceinline__ void find_bin(SelShared<T>& s, int n_bins, uint32_t k) {
  const int per = n_bins > T ? n_bins / T : 1;
  const int first = n_bins - 1 - static_cast<int>(threadIdx.x) * per;   // this thread's highest bin
  uint32_t mine = 0;
  if (first >= 0)
    for (int i = 0; i < per; ++i) mine += s.hist[first - i];
  uint32_t before = sum_before<T>(mine, s);
  if (before < k && before + mine >= k)   // (one thread)
    for (int i = 0; i < per; ++i) {
      const uint32_t h = s.hist[first - i];
      if (before + h >= k) {
        s.digit = first - i;
        s.left = k - before;
        break;
      }
      before += h;
    }
  __syncthreads();
}

// The k-th largest of the 32-bit keys in `keys` of the pages marked in `open`.
template <int T>
__device__ __noinline__ uint32_t kth_largest(SelShared<T>& s, const uint32_t* keys, const uint32_t* open, int n, uint32_t k) {
  uint32_t prefix = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += T) s.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += T)
      if ((open[i >> 5] >> (i & 31) & 1u) != 0 && (shift == 24 || keys[i] >> (shift + 8) == prefix))
        atomicAdd(&s.hist[keys[i] >> shift & 255u], 1u);
    __syncthreads();
    find_bin<T>(s, 256, k);
    prefix = prefix << 8 | s.digit;
    k = s.left;
    __syncthreads();
  }
  return prefix;
}

// a + b = s + e exactly (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float& a, float b, float& e) {
  const float s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  a = s;
}

// Exact score of a page for the group by one warp, scaled by the powers of two
// sq sa (which bring |q|_1 to [256, 512) and the bounds to about 1, so that products
// stay in range).  A product of two bf16 is exact in 32 bits and the sums are kept in
// three floats each, s + t + u: what is lost is below 2^-53 of the largest, and
// the slow 64-bit pipe only joins the three.  Eight lanes take a head.
template <int D>
__device__ double exact_score(const SelectParams& p, const int32_t* bt, int row, int kvh, int page, float sq,
                              float sa) {
  const int lane = threadIdx.x & 31, slot = lane >> 3, sub = lane & 7;
  const int id = bt[page];
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) return 0.0;
  const uint16_t* src = p.bounds + id * p.bounds_stride_page + kvh * p.bounds_stride_head + 8 * sub;
  uint4 lo[D / 64], hi[D / 64];
  uint32_t big = 0u;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    lo[i] = *reinterpret_cast<const uint4*>(src + 64 * i);
    hi[i] = *reinterpret_cast<const uint4*>(src + D + 64 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      big = absmax_bf16x2(absmax_bf16x2(big, (&lo[i].x)[e]), (&hi[i].x)[e]);
  }
  big = absmax_bf16x2(big, big >> 16) & 0x7fffu;
  if (__any_sync(0xffffffffu, big > 0x7f7fu)) return INFINITY;   // an infinity or NaN
  double best = -INFINITY;
  for (int j = slot; j - slot < p.group; j += 4) {
    const uint16_t* q = p.q + static_cast<int64_t>(row) * p.q_stride_tok +   // (heads beyond the group repeat its last)
                        static_cast<int64_t>(kvh * p.group + min(j, p.group - 1)) * p.q_stride_head + 8 * sub;
    float s = 0.f, t = 0.f, u = 0.f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 qv = *reinterpret_cast<const uint4*>(q + 64 * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int shift = (e & 1) * 16;
        const float x = bf16_to_f32(static_cast<uint16_t>((&qv.x)[e >> 1] >> shift));
        const uint32_t w = x < 0.f ? (&lo[i].x)[e >> 1] : (&hi[i].x)[e >> 1];
        float err;
        two_sum(s, __fmul_rn(x * sq, bf16_to_f32(static_cast<uint16_t>(w >> shift)) * sa), err);
        two_sum(t, err, err);
        u += err;
      }
    }
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) {
      const float s2 = __shfl_xor_sync(0xffffffffu, s, k), t2 = __shfl_xor_sync(0xffffffffu, t, k);
      const float u2 = __shfl_xor_sync(0xffffffffu, u, k);
      float e1, e2;
      two_sum(s, s2, e1);
      two_sum(t, t2, e2);
      u += u2 + e2;
      two_sum(t, e1, e1);
      u += e1;
    }
    best = fmax(best, static_cast<double>(s) + (static_cast<double>(t) + static_cast<double>(u)));
  }
  best = fmax(best, __shfl_xor_sync(0xffffffffu, best, 8));
  return fmax(best, __shfl_xor_sync(0xffffffffu, best, 16));
}

// One CTA = one (query row, kv head); a thread keeps kPer of the row's scores in
// registers (rows of more than kPer T pages read them again).  The K-th largest
// is located by one histogram over kBins equal steps between the smallest and
// the largest score, and ranked among the few of its step; of a crowded step the
// two edges take the place of t: in above the upper edge + 2 eps, out below the
// lower edge - 2 eps.  What is chosen and what is open is kept as bit maps in
// shared memory, and the chosen pages are written in ascending order at the end.
template <int D, int T, int kPer>
__global__ void __launch_bounds__(T) select_kernel(const SelectParams p) {
  constexpr int W = T / 32;
  constexpr int kBins = Sel<T>::kBins, kListCap = Sel<T>::kListCap;
  extern __shared__ uint32_t bits[];                 // chosen, then open
  __shared__ SelShared<T> s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = p.row0 + blockIdx.x;
  const int kvh = blockIdx.y;
  const RowPlace at = find_row<T>(p.seq_lens, p.qsl, p.batch, row, p.max_len);
  const int n = at.pos < 0 ? 0 : (at.pos >> p.ps_log2) + 1;
  int32_t* out = p.pages + (static_cast<int64_t>(row) * p.num_kv_heads + kvh) * p.top;
  if (at.b < 0 || at.bad || n <= p.top) {
    if (at.b >= 0 && at.bad && tid == 0) atomicOr(p.err, kErrCapacity);
    if (at.b >= 0 && !at.bad)
      for (int i = tid; i < p.top; i += T) out[i] = i < n ? i : -1;   // every page
    pdl_wait_primary();                              // (this grid ends no earlier than the scores')
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

  // the largest |q|_1 of the group's heads (before the scores are waited for), times
  // kQScale: the scaled elements are exact (a subnormal bf16's too) and up to 256 of
  // them have a finite sum, so the sum is infinite only where q is not finite.  D / 8
  // lanes a head.
  float q1 = 0.f;
  for (int j0 = 0; j0 < p.group; j0 += W * (256 / D)) {
    const int j = min(j0 + tid / (D / 8), p.group - 1);
    const uint4 x = *reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(row) * p.q_stride_tok +
                                                    static_cast<int64_t>(kvh * p.group + j) * p.q_stride_head +
                                                    tid % (D / 8) * 8);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sum += kQScale * fabsf(__uint_as_float((&x.x)[e] << 16)) +
             kQScale * fabsf(__uint_as_float((&x.x)[e] & 0xffff0000u));
#pragma unroll
    for (int k = D / 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    q1 = sum <= FLT_MAX ? fmaxf(q1, sum) : INFINITY;
  }
  for (int i = tid; i < kBins; i += T) s.hist[i] = 0;
  if (tid == 0) s.infs = s.decided = s.n_open = 0;
  __syncthreads();
  pdl_wait_primary();

  // scores of pages that are not chosen by score read as -infinity, which none has
  float first_v[kPer];
  auto load = [&](int i) { return i >= lo && i < hi ? score[i] : -INFINITY; };
#pragma unroll
  for (int j = 0; j < kPer; ++j) first_v[j] = load(j * T + tid);
  auto each = [&](auto f) {                          // f(page, score): whole warps on 32 neighbours
    for (int base = 0; base < n; base += kPer * T) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = base + j * T + tid;
        if (i - lane < n) f(i, base == 0 ? first_v[j] : load(i));
      }
    }
  };

  float above = INFINITY, below = INFINITY;
  bool all_open = false, ties = true;                // ties: what is open is exactly equal
  float sq = 1.f, sa = 1.f;                          // 1 / (kQScale |q|_1) and 1 / A, as powers of two
  if (want > 0) {
    float v[4] = {-INFINITY, -INFINITY, 0.f, q1};    // largest and -smallest finite score, A, kQScale |q|_1
    uint32_t infs = 0;
    each([&](int, float x) {
      infs += x == INFINITY;
      if (fabsf(x) <= FLT_MAX) {
        v[0] = fmaxf(v[0], x);
        v[1] = fmaxf(v[1], -x);
      }
    });
    const int chunks = (hi + p.chunk_pages - 1) / p.chunk_pages;
    for (int i = tid; i < chunks; i += T) v[2] = fmaxf(v[2], p.amax[cell * p.n_chunks + i]);
    if (infs != 0) atomicAdd(&s.infs, infs);
    block_max<T>(v, s);                              // (its barrier publishes s.infs)
    infs = s.infs;
    const float top = v[0], low = -v[1], am = v[2];
    // |q|_1 itself is summed in 32 bits: a hundredth more covers it.  Factors and
    // sums below the normal range may be flushed: (|q|_1 + D A + 2 D) times the
    // smallest normal covers them.  Where a sum could overflow everything is open.
    // A q that is not finite gives every page +infinity, a zero one zero: exact.
    const float size = v[3] * am;                    // kQScale |q|_1 A
    sq = inverse_power(v[3]);
    sa = inverse_power(am);
    const float eps = !(v[3] <= FLT_MAX) || v[3] == 0.f || am == 0.f ? 0.f
                      : size <= 0.5f * kQScale * FLT_MAX
                          ? 1.01f * (D * 0x1p-22f / kQScale) * size +
                                (v[3] * (FLT_MIN / kQScale) + (D * am + 2 * D) * FLT_MIN)
                          : INFINITY;
    all_open = !(eps <= FLT_MAX);
    ties = !all_open;
    if (infs >= want && !all_open) {
      above = below = INFINITY;                      // infinities alone, all alike
    } else if (!all_open) {
      ties = eps == 0.f && top == low;
      float t_lo = low, t_hi = top;
      const float half = 0.5f * top - 0.5f * low;    // (does not overflow)
      const float step = kBins / half;
      if (half > 0.f && step <= FLT_MAX) {
        auto bin = [&](float x) { return min(kBins - 1, static_cast<int>((0.5f * x - 0.5f * low) * step)); };
        each([&](int, float x) {
          if (fabsf(x) <= FLT_MAX) atomicAdd(&s.hist[bin(x)], 1u);
        });
        __syncthreads();
        find_bin<T>(s, kBins, want - infs);
        const int digit = s.digit;
        const uint32_t in_bin = s.hist[digit], left = s.left;
        if (in_bin <= 32) {                          // the K-th itself: rank the step's few
          each([&](int i, float x) {
            if (fabsf(x) <= FLT_MAX && bin(x) == digit) s.index[atomicAdd(&s.infs, 1u) - infs] = __float_as_int(x);
          });
          __syncthreads();
          const float x = lane < static_cast<int>(in_bin) ? __int_as_float(s.index[lane]) : -INFINITY;
          uint32_t larger = 0;
          for (uint32_t j = 0; j < in_bin; ++j) {
            const float y = __shfl_sync(0xffffffffu, x, j);
            larger += y > x || (y == x && static_cast<int>(j) < lane);
          }
          t_lo = t_hi = __shfl_sync(0xffffffffu, x, __ffs(__ballot_sync(0xffffffffu, larger == left - 1)) - 1);
          __syncthreads();                           // (the list is used again)
        } else {                                     // the step's edges, with room for the roundings of bin() and of this
          const float width = 2.f * (half / kBins), slop = 0x1p-20f * (fabsf(top) + fabsf(low));
          t_lo = fmaxf(low, low + digit * width - slop);
          t_hi = fminf(top, low + (digit + 1) * width + slop);
        }
      }
      above = __fadd_ru(t_hi, 2.f * eps);
      below = __fadd_rd(t_lo, -2.f * eps);
    }
  }

  // decide what 32 bits can
  uint32_t n_in = 0;
  each([&](int i, float x) {
    const bool cand = want > 0 && x != -INFINITY;
    const bool sure = cand && !all_open && x > above;
    const bool maybe = cand && !sure && (all_open || x >= below);
    const uint32_t in_w = __ballot_sync(0xffffffffu, sure || (i < n && (i < lo || i >= hi)));
    const uint32_t open_w = __ballot_sync(0xffffffffu, maybe);
    n_in += __popc(in_w);
    if (lane == 0) {
      chosen[i >> 5] = in_w;
      open[i >> 5] = open_w;
    }
    if (open_w != 0) {                               // (the same for the warp)
      uint32_t at_list = 0;
      if (lane == 0) at_list = atomicAdd(&s.n_open, __popc(open_w));
      at_list = __shfl_sync(0xffffffffu, at_list, 0) + __popc(open_w & ((1u << lane) - 1u));
      if (maybe && at_list < kListCap) s.index[at_list] = i;
    }
  });
  if (lane == 0) atomicAdd(&s.decided, n_in);
  __syncthreads();
  const uint32_t n_open = s.n_open;
  uint32_t need = p.top - s.decided;                 // to take from the open ones

  if (need > 0 && need < n_open && !ties) {
    if (n_open <= kListCap) {
      // rank them by their exact scores
      for (uint32_t i = warp; i < n_open; i += W) {
        const double v = exact_score<D>(p, bt, row, kvh, s.index[i], sq, sa);
        if (lane == 0) s.value[i] = v;
      }
      __syncthreads();
      for (uint32_t i = tid; i < n_open; i += T) {
        const double v = s.value[i];
        const int page = s.index[i];
        uint32_t better = 0;
        for (uint32_t j = 0; j < n_open; ++j) better += s.value[j] > v || (s.value[j] == v && s.index[j] < page);
        if (better < need) atomicOr(&chosen[page >> 5], 1u << (page & 31));
      }
      need = 0;
    } else {
      // too many to rank: the need-th largest exact score by its upper, then its
      // lower 32 bits, kept in place of the 32-bit scores
      uint32_t* keys = reinterpret_cast<uint32_t*>(score);
      for (int half = 0; half < 2 && need > 0; ++half) {
        for (int w = warp; w < words; w += W)
          for (uint32_t m = open[w]; m != 0; m &= m - 1) {
            const int i = w * 32 + __ffs(m) - 1;
            const uint64_t k = key64(exact_score<D>(p, bt, row, kvh, i, sq, sa));
            if (lane == 0) keys[i] = static_cast<uint32_t>(half == 0 ? k >> 32 : k);
          }
        __syncthreads();
        const uint32_t kth = kth_largest<T>(s, keys, open, n, need);
        uint32_t taken = 0;
        if (tid == 0) s.decided = 0;
        __syncthreads();
        for (int w = tid; w < words; w += T) {
          uint32_t win = 0, stay = 0;
          for (uint32_t m = open[w]; m != 0; m &= m - 1) {
            const int b = __ffs(m) - 1;
            win |= (keys[w * 32 + b] > kth ? 1u : 0u) << b;
            stay |= (keys[w * 32 + b] == kth ? 1u : 0u) << b;
          }
          chosen[w] |= win;
          open[w] = stay;
          taken += __popc(win);
        }
        if (taken != 0) atomicAdd(&s.decided, taken);
        __syncthreads();
        need -= s.decided;
        __syncthreads();
      }
    }
  }
  __syncthreads();

  // the lowest `need` of what is still open equal the border: take them; then
  // write the chosen pages in order.  Thread t holds words [t per, (t + 1) per).
  const int per = (words + T - 1) / T;
  const int w0 = tid * per, w1 = min(w0 + per, words);
  if (need > 0) {
    uint32_t mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(open[w]);
    uint32_t before = sum_before<T>(mine, s);
    for (int w = w0; w < w1; ++w)
      for (uint32_t m = open[w]; m != 0 && before < need; m &= m - 1, ++before) chosen[w] |= m & (0u - m);
  }
  uint32_t mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(chosen[w]);
  uint32_t at_out = sum_before<T>(mine, s);
  for (int w = w0; w < w1; ++w)
    for (uint32_t m = chosen[w]; m != 0 && at_out < static_cast<uint32_t>(p.top); m &= m - 1)
      out[at_out++] = w * 32 + __ffs(m) - 1;
}

template <int D, int T, int kPer>
cudaError_t launch_select(const SelectParams& p, bool scored, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.rows, p.num_kv_heads);
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = p.row_pages / 32 * 8;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = scored ? 1 : 0;   // overlaps the score kernel's end, and waits for its scores
  return cudaLaunchKernelEx(&cfg, select_kernel<D, T, kPer>, p);
}

// Shared memory of a score CTA of `rows` rows.
int score_smem(const SelectParams& p, int D, int rows) {
  const int tpt = 8 / p.hpt;
  return (rows + tpt - 1) / tpt * ((p.group + p.hpt - 1) / p.hpt) * 8 * (4 * D + 64);
}

template <int D>
cudaError_t launch(const SelectParams& p, int chunks, cudaStream_t st) {
  if (chunks > 0) {
    const bool one = p.block_rows == 1 && p.group <= 8;
    const int smem = one ? One<D>::SMEM : score_smem(p, D, p.block_rows);
    auto kern = one ? score_one_kernel<D> : score_block_kernel<D>;
    // The limit is the kernel's, not this call's (128 heads of a row; a block of several
    // rows stays below 48 KB): of two host threads that set a size of their own, one
    // could launch under the other's.
    const int most = one ? One<D>::SMEM : 128 * (4 * D + 64);
    if (most > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
    }
    const dim3 grid((p.rows + p.block_rows - 1) / p.block_rows * p.num_kv_heads, chunks);
    kern<<<grid, kScoreThreads, smem, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // Threads per row: sixteen scores each where rows are many (the fixed work of a
  // row is per warp: 3200 rows of 512 pages 30.3 us against 34.8 with eight, 45.8
  // with four), eight where they are few and the time of one row counts (512 rows of
  // 2048 pages 64.7 us against 66.3 with sixteen, 73.6 with four); at most 512
  // or 1024 (longer rows read their scores again).  Those figures are of one code for
  // both counts; compiled apart the two calls take 29.7 and 62.2 us.
  if (static_cast<int64_t>(p.rows) * p.num_kv_heads >= 8 * p.num_sms) {
    if (p.row_pages <= 32 * 16) return launch_select<D, 32, 16>(p, chunks > 0, st);
    if (p.row_pages <= 64 * 16) return launch_select<D, 64, 16>(p, chunks > 0, st);
    if (p.row_pages <= 128 * 16) return launch_select<D, 128, 16>(p, chunks > 0, st);
    if (p.row_pages <= 256 * 16) return launch_select<D, 256, 16>(p, chunks > 0, st);
    return launch_select<D, 512, 16>(p, chunks > 0, st);
  }
  if (p.row_pages <= 64 * 8) return launch_select<D, 64, 8>(p, chunks > 0, st);
  if (p.row_pages <= 256 * 8) return launch_select<D, 256, 8>(p, chunks > 0, st);
  return launch_select<D, 1024, 8>(p, chunks > 0, st);
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
  p.ps_log2 = __builtin_ctz(static_cast<unsigned>(s.page_size));
  p.max_len = static_cast<int64_t>(s.max_pages_per_seq) * s.page_size;
  p.num_sms = s.num_sms;
  p.top = s.top_pages;
  p.first = s.first_pages;
  p.last = s.last_pages;
  p.row_pages = static_cast<int>(score_pages(s));
  p.n_chunks = static_cast<int>(score_chunks(s));
  p.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + kScratchHeaderBytes);
  p.err = static_cast<uint32_t*>(scratch);
  // rows per score CTA: one for decode; for chunks as many as a request brings on
  // average, as far as their factors take 48 KB of shared memory (400 rows of 4
  // requests 30.3 us; with 24 KB 32.9, with 96 KB 41.3)
  auto heads_per_tile = [&](int rows) {
    int h = 8;
    while (h > 1 && (h / 2 >= p.group || 8 / h < rows)) h /= 2;
    return h;
  };
  p.block_rows = 1;
  p.hpt = heads_per_tile(1);
  if (query_start_loc != nullptr) {
    const int each = (total_q + batch - 1) / batch;
    while (p.block_rows < each) {
      SelectParams next = p;
      next.block_rows *= 2;
      next.hpt = heads_per_tile(next.block_rows);
      if (next.block_rows > kScoreThreads || score_smem(next, s.head_dim, next.block_rows) > 48 * 1024) break;
      p = next;
    }
  }
  // Pages per score CTA: few enough that one wave of CTAs takes them all, at most
  // 256 (contexts differ in length: shorter chunks balance; 64 requests of 4 to 32 K
  // tokens take 64.3 us with 128, 64.6 with 256, 64.2 with 512).  Blocks of several
  // rows also stage queries: two waves, at most 512 (400 rows of 4 requests with 64 /
  // 128 / 256 pages: 42.1 / 37.7 / 41.6 us).
  const int64_t blocks = (std::min(total_q, plan->score_rows) + p.block_rows - 1) / p.block_rows;
  const int64_t pages_all = blocks * s.num_kv_heads * p.row_pages;
  const int64_t slots = static_cast<int64_t>(s.num_sms) * (p.block_rows == 1 ? 4 : 8);
  const int64_t even = (pages_all / slots + kScorePagesMin - 1) / kScorePagesMin * kScorePagesMin;
  const int64_t chunk = std::min<int64_t>(std::max<int64_t>(even, kScorePagesMin), p.block_rows == 1 ? 256 : 512);
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
