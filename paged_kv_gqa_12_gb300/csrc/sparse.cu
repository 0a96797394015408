// Attention over chosen pages (sm_103a), and the plan it shares with page
// selection.
//
// For query row r, kv head g: J = { j <= pos : j / ps in pages[r][g] },
//   out = sum_J exp(s_j) V_j / Z,  Z = sum_J exp(s_j) (+ exp(sink)),  lse = ln Z,
// the sums of the decode kernel over another key set, with an online softmax
// in the log2 domain and 32-bit accumulators.
//
// Like decode the kernel streams K and V once and is bound by bytes in flight
// (one query token: 4 D flops per 4 D bytes of bf16 K and V, times the group).
//   * One CTA = one (row, split of its pages, kv head [, 16 heads of a large
//     group]), 4 warps, each with a private ring of stages that its lane 0
//     refills by TMA from the pages; no barrier between warps in the loop.
//   * A split takes an equal share of the list's entries, whatever they hold, so
//     that its first loads (list, then block table) wait for nothing else.  Its
//     pages are laid side by side: key x is slot x % ps of entry x / ps.  Each
//     entry's pool page and the number of its keys at or before pos (`lim`) are
//     staged in shared memory once, so the loop is that of a dense sequence and
//     only tiles with lim < their keys are masked.
//   * S^T = K Q^T and O^T += V^T P^T on warp-level bf16 MMAs, the group's heads
//     as N = 8: with 8 query rows a 128-row tcgen05 tile would be 1/16 used.
//   * Splits are merged by the CTA that finishes last (arrival counters in the
//     scratch header), so a call is one launch and no CTA waits.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "ptx.cuh"
#include "sparse.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSmem = 232448;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kBelow = 1.f - 0x1p-12f;

struct SparseParams {
  const uint16_t* q;
  int64_t q_stride_tok, q_stride_head;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  const int32_t* qsl;
  int batch, num_q_heads, num_kv_heads, group, ps_log2, num_pages;
  int64_t max_len;
  int max_pages;
  const int32_t* pages;       // [rows, Hkv, top]
  int top;
  float scale_log2, cap_log2, scale_over_cap;
  const float* sinks;
  float k_scale, v_scale;
  const float* k_scales;
  const float* v_scales;
  uint16_t* out;
  int64_t out_stride_tok, out_stride_head;
  float* lse;
  float* o_part;              // [rows, Hq, splits, D]
  float* lse_part;            // [rows, Hq, splits]
  int splits, head_groups, list_cap;
  uint32_t* counters;         // [rows, Hkv * head_groups]
  uint32_t* err;
};

template <int D, bool FP8, int NH8>
struct Cfg;
// Keys per stage and stages per warp.  The rings are small, so that many CTAs
// share an SM and a call of a few hundred rows is one wave of them; a warp that
// waits for its one stage is covered by the others.  Measured, 64 rows of 2048
// keys over 8 kv heads (us; TS x NS):
//   bf16  D 64: 16x2 62.3, 32x1 62.8, 16x1 66.9, 64x1 75.7, 16x4 86.3
//   bf16 D 128: 16x1 86.6, 32x1 102, 16x2 108; 16 heads a kv head: 16x2 53.1, 32x1 54.6, 16x1 64.8
//   bf16 D 256: 16x1 170, 32x1 181, 16x2 188
//   e4m3  D 64: 64x1 51.8, 32x1 53.0, 16x2 53.1, 16x1 64.2
//   e4m3 D 128: 16x2 75.9, 16x3 75.8, 16x1 80.4, 32x2 98.9; D 256: 32x1 137, 16x2 148, 16x1 157
// CTAS are the CTAs that share an SM by their registers, which the launch bounds
// hold the compiler to (the figures above are without them): the plan counts on
// them.  e4m3 D 64 has five where the compiler by itself makes room for four: 400
// rows of 2048 keys 181 -> 173.5 us, the 64 rows 51.2 -> 51.5.  e4m3 D 128 held to its
// own four takes 75.3 -> 71.4, with five 80.4; the others do not change.  (All of this
// with one bf16 of small weights; see the P V step.)
template <int NH8> struct Cfg<64, false, NH8> { static constexpr int TS = 16, NS = 2, CTAS = NH8 == 1 ? 5 : 4; };
template <int NH8> struct Cfg<128, false, NH8> { static constexpr int TS = 16, NS = NH8 == 1 ? 1 : 2, CTAS = NH8 == 1 ? 5 : 3; };
template <int NH8> struct Cfg<256, false, NH8> { static constexpr int TS = 16, NS = 1, CTAS = NH8 == 1 ? 3 : 2; };
template <int NH8> struct Cfg<64, true, NH8> { static constexpr int TS = 64, NS = 1, CTAS = NH8 == 1 ? 5 : 3; };
template <int NH8> struct Cfg<128, true, NH8> { static constexpr int TS = 16, NS = 2, CTAS = NH8 == 1 ? 4 : 3; };
template <int NH8> struct Cfg<256, true, NH8> { static constexpr int TS = 32, NS = 1, CTAS = 2; };

template <int D, bool FP8, int NH8>
struct Tile {
  static constexpr int TS = Cfg<D, FP8, NH8>::TS;
  static constexpr int NS = Cfg<D, FP8, NH8>::NS;
  static constexpr int E = FP8 ? 1 : 2;
  static constexpr int ROW = D * E;                     // bytes of a key of one head
  static constexpr int RB = ROW < 128 ? ROW : 128;      // bytes per TMA box row
  static constexpr int NCC = ROW / RB;                  // column chunks
  static constexpr int BYTES = TS * ROW;                // K (or V) of a stage
  static constexpr int STAGE = 2 * BYTES;
  // a warp's ring; at the end it holds the warp's state, [8 NH8][D] and two [8 NH8] floats
  static constexpr int STATE = (8 * NH8 * (D + 2) * 4 + 1023) / 1024 * 1024;
  static constexpr int WARP = NS * STAGE > STATE ? NS * STAGE : STATE;
  static constexpr int MT = TS / 16;
  static constexpr int KS = D / 16;

  // Byte (row, byte of the row) of a stage as TMA writes it: column chunks,
  // rows of RB bytes, 16-byte units swizzled by the row.
  __device__ static __forceinline__ uint32_t at(int row, int byte) {
    const int cc = byte / RB, x = byte % RB;
    const uint32_t sw = RB == 128 ? (row & 7) : ((row >> 1) & 3);
    return static_cast<uint32_t>(cc * TS * RB + row * RB) + ((((x >> 4) ^ sw) << 4) | (x & 15));
  }
};

__device__ __forceinline__ uint32_t pack_bf16x2_down(float lo, float hi) {   // rounded towards zero
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float lanes8_max(float v) {   // over the 8 lanes of equal lane % 4
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float lanes8_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// Output of (row, head) where nothing is attended: 0, and the sink or -inf.
__device__ __forceinline__ void write_empty(const SparseParams& p, int D, int row, int head0, int heads) {
  for (int i = threadIdx.x; i < heads * D; i += kThreads) {
    const int h = head0 + i / D, d = i % D;
    p.out[row * p.out_stride_tok + h * p.out_stride_head + d] = 0;
    if (d == 0 && p.lse != nullptr)
      p.lse[static_cast<int64_t>(row) * p.num_q_heads + h] = p.sinks != nullptr ? p.sinks[h] : -INFINITY;
  }
}

// Merge of a row's splits for `heads` heads by their log-sum-exps: a thread
// takes four dims of one head and folds the splits, eight loads in flight,
// into a running maximum, sum and weighted output.
template <int D>
__device__ __forceinline__ void merge(const SparseParams& p, int n, int row, int head0, int heads) {
  constexpr int C = D / 4;
  constexpr int U = 8;
  for (int e = threadIdx.x; e < heads * C; e += kThreads) {
    const int h = head0 + e / C;
    const int d = (e % C) * 4;
    const int64_t at = (static_cast<int64_t>(row) * p.num_q_heads + h) * p.splits;
    const float* lp = p.lse_part + at;
    const float* op = p.o_part + at * D + d;
    float M = p.sinks != nullptr ? p.sinks[h] * kLog2e : -INFINITY;
    float Z = M == -INFINITY ? 0.f : 1.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < n; s0 += U) {
      float l[U];
      float4 o[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = s0 + u < n;
        l[u] = ok ? __ldcg(lp + s0 + u) * kLog2e : -INFINITY;
        o[u] = ok ? __ldcg(reinterpret_cast<const float4*>(op + static_cast<int64_t>(s0 + u) * D))
                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = l[0];
#pragma unroll
      for (int u = 1; u < U; ++u) top = fmaxf(top, l[u]);
      if (top > M) {
        const float f = ex2(M - top);
        Z *= f;
        acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
        M = top;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (l[u] == -INFINITY) continue;   // padding, or a split without a key
        const float w = ex2(l[u] - M);
        Z += w;
        acc.x += w * o[u].x; acc.y += w * o[u].y; acc.z += w * o[u].z; acc.w += w * o[u].w;
      }
    }
    const float inv = Z > 0.f ? 1.f / Z : (Z != Z ? Z : 0.f);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * p.out_stride_tok + h * p.out_stride_head + d);
    dst[0] = pack_bf16x2(acc.x * inv, acc.y * inv);
    dst[1] = pack_bf16x2(acc.z * inv, acc.w * inv);
    if (d == 0 && p.lse != nullptr)
      p.lse[static_cast<int64_t>(row) * p.num_q_heads + h] = Z == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + lg2(Z)) * kLn2;
  }
}

template <int D, bool FP8, int NH8, bool CAP>
__global__ void __launch_bounds__(kThreads, Cfg<D, FP8, NH8>::CTAS)
sparse_attn_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const SparseParams p) {
  using T = Tile<D, FP8, NH8>;
  constexpr int TS = T::TS, NS = T::NS;
  const int row = blockIdx.x / p.splits;
  const int split = blockIdx.x - row * p.splits;
  const int kvh = blockIdx.y / p.head_groups;
  const int part = (blockIdx.y - kvh * p.head_groups) * 16;       // first head of the group here
  const int heads = min(16, p.group - part);
  const int head0 = kvh * p.group + part;
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int ps = 1 << p.ps_log2;

  // entries [e0, e1) of the row's list are this split's; the first of each thread
  // leaves before the row's place is known
  const int e0 = split * p.list_cap;
  const int entries = min(p.top - e0, p.list_cap);
  const int32_t* list = p.pages + (static_cast<int64_t>(row) * p.num_kv_heads + kvh) * p.top + e0;
  int entry = tid < entries ? list[tid] : -1;

  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_used;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * T::WARP);
  int32_t* ids = reinterpret_cast<int32_t*>(bars + kWarps * NS);
  int32_t* lims = ids + p.list_cap;
  if (tid == 0) {
    s_used = 0;
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    for (int i = 0; i < kWarps * NS; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  const RowPlace at = find_row<kThreads>(p.seq_lens, p.qsl, p.batch, row, p.max_len);
  if (at.b < 0) return;                                    // behind the last request
  if (at.bad) {
    if (tid == 0) atomicOr(p.err, kErrCapacity);
    return;
  }
  if (at.pos < 0) {                                        // a request without keys
    if (split == 0) write_empty(p, D, row, head0, heads);
    return;
  }
  const int32_t* bt = p.block_table + at.b * p.bt_stride;
  __syncthreads();                                         // s_used
  int used = 0;
  for (int i = tid; i < entries; i += kThreads) {
    if (i != tid) entry = list[i];
    int id = p.num_pages, lim = 0;                         // an out-of-range box: zeros
    if (entry >= 0 && entry < p.max_pages) {
      id = bt[entry];
      const int left = at.pos + 1 - (entry << p.ps_log2);  // keys of the page at or before pos
      lim = min(max(left, 0), ps);
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
        if (lim > 0) atomicOr(p.err, kErrPageId);
        id = p.num_pages;
      }
    }
    ids[i] = id;
    lims[i] = lim;
    if (lim > 0) used = i + 1;
  }
  used = __reduce_max_sync(0xffffffffu, used);
  if (lane == 0 && used > 0) atomicMax(&s_used, used);
  __syncthreads();
  // keys of the listed pages, side by side: x is slot x % ps of entry x / ps
  const int key_end = s_used << p.ps_log2;
  const int tiles = (key_end + TS - 1) / TS;

  uint8_t* ring = smem + warp * T::WARP;
  uint64_t* bar = bars + warp * NS;
  const int br = min(ps, TS);                              // rows per TMA box

  // Lane 0: fetch local tile k into `stage`; boxes without an attended key are
  // left out (their rows are masked).
  auto fetch = [&](int k, int stage) {
    const int x0 = k * TS;
    uint8_t* ks = ring + stage * T::STAGE;
    uint8_t* vs = ks + T::BYTES;
    uint32_t want = 0;
    for (int j = 0; j < TS / br; ++j) {
      const int x = x0 + j * br;
      if (x < key_end && (x & (ps - 1)) < lims[x >> p.ps_log2]) want |= 1u << j;
    }
    mbar_arrive_expect_tx(&bar[stage], static_cast<uint32_t>(__popc(want) * br * T::ROW * 2));
    for (int j = 0; j < TS / br; ++j) {
      if (!(want >> j & 1u)) continue;
      const int x = x0 + j * br;
      const int id = ids[x >> p.ps_log2];
#pragma unroll
      for (int cc = 0; cc < T::NCC; ++cc) {
        const int dst = cc * TS * T::RB + j * br * T::RB;
        tma_load_4d(ks + dst, &tmk, cc * (T::RB / T::E), kvh, x & (ps - 1), id, &bar[stage]);
        tma_load_4d(vs + dst, &tmv, cc * (T::RB / T::E), kvh, x & (ps - 1), id, &bar[stage]);
      }
    }
  };
  if (lane == 0)
    for (int s = 0; s < NS; ++s)
      if (warp + s * kWarps < tiles) fetch(warp + s * kWarps, s);
  __syncwarp();

  // Q^T fragments (B operand: k = dim, n = head)
  uint32_t qf[T::KS][NH8][2];
#pragma unroll
  for (int j = 0; j < NH8; ++j) {
    const int h = j * 8 + g;
    const bool ok = h < heads;
    const uint16_t* src = p.q + row * p.q_stride_tok + (head0 + (ok ? h : 0)) * p.q_stride_head;
#pragma unroll
    for (int ks = 0; ks < T::KS; ++ks) {
      // e4m3: thread c owns dims [c D/4, (c+1) D/4) so that its bytes are contiguous
      const int d0 = FP8 ? c * (D / 4) + ks * 4 : ks * 16 + 2 * c;
      const int d1 = FP8 ? d0 + 2 : d0 + 8;
      qf[ks][j][0] = ok ? *reinterpret_cast<const uint32_t*>(src + d0) : 0u;
      qf[ks][j][1] = ok ? *reinterpret_cast<const uint32_t*>(src + d1) : 0u;
    }
  }

  float o[T::KS][NH8][4];
  float m_run[NH8][2], l_run[NH8][2];
#pragma unroll
  for (int j = 0; j < NH8; ++j) {
#pragma unroll
    for (int i = 0; i < T::KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    m_run[j][0] = m_run[j][1] = -INFINITY;
    l_run[j][0] = l_run[j][1] = 0.f;
  }
  const uint64_t k_sc = dequant_scale2(p.k_scales != nullptr ? p.k_scales[at.b] : p.k_scale);
  const uint64_t v_sc = dequant_scale2(p.v_scales != nullptr ? p.v_scales[at.b] : p.v_scale);

  int it = 0;
  for (int k = warp; k < tiles; k += kWarps, ++it) {
    const int stage = it % NS;
    if (!__all_sync(0xffffffffu, mbar_wait(&bar[stage], (it / NS) & 1, p.err))) {
      // give up (the error word says so), but not before the later stages' copies had their time to land
      for (int i = 1; i < NS; ++i)
        if (k + i * kWarps < tiles) mbar_wait(&bar[(it + i) % NS], ((it + i) / NS) & 1, p.err);
      break;
    }
    const uint8_t* kst = ring + stage * T::STAGE;
    const uint8_t* vst = kst + T::BYTES;
    const uint32_t ku = smem_u32(kst), vu = smem_u32(vst);
    const int x0 = k * TS;
    // attended keys of each 16-key group: those before `left` (a group lies in one page)
    int left[T::MT];
    bool partial = false;
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt) {
      const int x = x0 + mt * 16;
      left[mt] = x < key_end ? lims[x >> p.ps_log2] - (x & (ps - 1)) : 0;
      partial |= left[mt] < 16;
    }

    // ---- S^T = K Q^T ----------------------------------------------------------
    float s[T::MT][NH8][4];
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt) {
#pragma unroll
      for (int j = 0; j < NH8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
      if constexpr (!FP8) {
        const int mi = lane >> 3;
        const int r = mt * 16 + (lane & 7) + ((mi & 1) << 3);
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks) {
          uint32_t a[4];
          ldsm_x4(a, ku + T::at(r, (ks * 16 + ((mi >> 1) << 3)) * 2));
#pragma unroll
          for (int j = 0; j < NH8; ++j) mma_bf16(s[mt][j], a, qf[ks][j][0], qf[ks][j][1]);
        }
      } else {
        constexpr int NV = D / 64;
        uint4 r0[NV], r1[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          r0[u] = *reinterpret_cast<const uint4*>(kst + T::at(mt * 16 + g, c * (D / 4) + 16 * u));
          r1[u] = *reinterpret_cast<const uint4*>(kst + T::at(mt * 16 + g + 8, c * (D / 4) + 16 * u));
        }
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(r0);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(r1);
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks) {
          uint32_t a[4];
          a[0] = dequant_e4m3x2<0>(w0[ks], k_sc);
          a[1] = dequant_e4m3x2<0>(w1[ks], k_sc);
          a[2] = dequant_e4m3x2<1>(w0[ks], k_sc);
          a[3] = dequant_e4m3x2<1>(w1[ks], k_sc);
#pragma unroll
          for (int j = 0; j < NH8; ++j) mma_bf16(s[mt][j], a, qf[ks][j][0], qf[ks][j][1]);
        }
      }
    }

    // ---- scale, soft-cap, mask -------------------------------------------------
    float mx[NH8][2];
#pragma unroll
    for (int j = 0; j < NH8; ++j) mx[j][0] = mx[j][1] = -INFINITY;
    auto scores = [&](auto masked) {
#pragma unroll
      for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
        for (int j = 0; j < NH8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = s[mt][j][e];
            if constexpr (CAP) {
              v = p.cap_log2 * tanhf(v * p.scale_over_cap);
            } else {
              v *= p.scale_log2;
            }
            if constexpr (decltype(masked)::value)
              if (g + ((e >> 1) << 3) >= left[mt]) v = -INFINITY;
            s[mt][j][e] = v;
            mx[j][e & 1] = fmaxf(mx[j][e & 1], v);
          }
    };
    if (partial) {
      scores(std::true_type{});
    } else {
      scores(std::false_type{});
    }

    // ---- online softmax --------------------------------------------------------
    float alpha[NH8][2], mu[NH8][2];
    bool grew = false;
#pragma unroll
    for (int j = 0; j < NH8; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[j][h] = lanes8_max(mx[j][h]);
        const float m = fmaxf(m_run[j][h], mx[j][h]);
        mu[j][h] = m == -INFINITY ? 0.f : m;
        grew |= m > m_run[j][h];
        alpha[j][h] = ex2(m_run[j][h] - mu[j][h]);
        m_run[j][h] = m;
      }
    const bool rescale = __any_sync(0xffffffffu, grew);   // else every alpha is 1
#pragma unroll
    for (int j = 0; j < NH8; ++j) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < T::MT; ++mt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][j][e] = ex2(s[mt][j][e] - mu[j][e & 1]);
        s0 += s[mt][j][0] + s[mt][j][2];
        s1 += s[mt][j][1] + s[mt][j][3];
      }
      l_run[j][0] = l_run[j][0] * alpha[j][0] + s0;
      l_run[j][1] = l_run[j][1] * alpha[j][1] + s1;
      if (rescale) {
#pragma unroll
        for (int i = 0; i < T::KS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][j][e] *= alpha[j][e & 1];
      }
    }
    // ---- O^T += V^T P^T --------------------------------------------------------
    // P goes into the MMAs as P_hi + P_lo, two bf16: off by 2^-15 of a weight.  One
    // bf16 would be off by up to 2^-8, in the same direction for equal weights, which
    // no number of keys averages out.  Choosing by tile whether the second part is
    // needed costs as much as always taking it (us, by tile / always: 64 rows of 2048
    // keys, bf16 D 128 86.4 / 86.2, e4m3 D 128 71.5 / 71.8, D 256 148 / 150; 400 e4m3
    // rows of D 64 172.9 / 166.1).  P_hi lies below P, by at least 2^-12 of it, so that
    // both parts are positive (or zero with P; P_lo of a weight below 2^-120 is too) and
    // an infinite V stays that infinity in either product (the chunk 168.4 us, the others
    // as they were).
    auto pv = [&](auto mask_tag) {
      constexpr bool MASK = decltype(mask_tag)::value;
#pragma unroll
      for (int mt = 0; mt < T::MT; ++mt) {
        uint32_t pb[NH8][2], pl[NH8][2];
#pragma unroll
        for (int j = 0; j < NH8; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = s[mt][j][2 * h], y = s[mt][j][2 * h + 1];
            const uint32_t w = pack_bf16x2_down(x * kBelow, y * kBelow);
            pb[j][h] = movmatrix_t(w);
            pl[j][h] =
                movmatrix_t(pack_bf16x2(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xffff0000u)));
          }
        // masked keys have P = 0, but their V may be stale or NaN: zero it
        uint32_t lo_mask = 0xffffffffu, hi_mask = 0xffffffffu;
        if constexpr (MASK) {
          const int x = 2 * c;
          lo_mask = (x < left[mt] ? 0x0000ffffu : 0u) | (x + 1 < left[mt] ? 0xffff0000u : 0u);
          hi_mask = (x + 8 < left[mt] ? 0x0000ffffu : 0u) | (x + 9 < left[mt] ? 0xffff0000u : 0u);
        }
        auto step = [&](int i, uint32_t (&a)[4]) {
          if constexpr (MASK) {
            a[0] &= lo_mask;
            a[1] &= lo_mask;
            a[2] &= hi_mask;
            a[3] &= hi_mask;
          }
#pragma unroll
          for (int j = 0; j < NH8; ++j) {
            mma_bf16(o[i][j], a, pb[j][0], pb[j][1]);
            mma_bf16(o[i][j], a, pl[j][0], pl[j][1]);
          }
        };
        if constexpr (!FP8) {
          const int mi = lane >> 3;
          const int r = mt * 16 + (lane & 7) + ((mi >> 1) << 3);
#pragma unroll
          for (int i = 0; i < T::KS; ++i) {
            uint32_t a[4];
            ldsm_x4_t(a, vu + T::at(r, (i * 16 + ((mi & 1) << 3)) * 2));
            step(i, a);
          }
        } else {
          // thread g owns dims [g D/8, (g+1) D/8): fragment i, row g is dim
          // g D/8 + 2i, row g + 8 the next
          constexpr int NW = D / 32;
          uint32_t v4[4][NW];
          const int r = mt * 16 + 2 * c;
#pragma unroll
          for (int u = 0; u < NW; u += 2)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint2 x = *reinterpret_cast<const uint2*>(
                  vst + T::at(r + (w & 1) + ((w >> 1) << 3), g * (D / 8) + 4 * u));
              v4[w][u] = x.x;
              v4[w][u + 1] = x.y;
            }
#pragma unroll
          for (int i = 0; i < T::KS; ++i) {
            const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(v4[0][i >> 1], v4[1][i >> 1], sel);
            const uint32_t y = __byte_perm(v4[2][i >> 1], v4[3][i >> 1], sel);
            uint32_t a[4] = {dequant_e4m3x2<0>(x, v_sc), dequant_e4m3x2<1>(x, v_sc), dequant_e4m3x2<0>(y, v_sc),
                             dequant_e4m3x2<1>(y, v_sc)};
            step(i, a);
          }
        }
      }
    };
    if (partial) {
      pv(std::true_type{});
    } else {
      pv(std::false_type{});
    }

    __syncwarp();
    if (lane == 0 && k + NS * kWarps < tiles) {
      fence_proxy_async_smem();
      fetch(k + NS * kWarps, stage);
    }
  }

  // ---- the four warps' states, merged in shared memory --------------------------
  // (each warp waited for all it fetched, so its ring is free)
  constexpr int HW = NH8 * 8;
  float* wo = reinterpret_cast<float*>(ring);   // [HW][D], then maxima [HW], then sums [HW]
#pragma unroll
  for (int j = 0; j < NH8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float l = lanes8_sum(l_run[j][h]);
      if (g == 0) {
        wo[HW * D + j * 8 + 2 * c + h] = m_run[j][h];
        wo[HW * D + HW + j * 8 + 2 * c + h] = l;
      }
    }
#pragma unroll
  for (int i = 0; i < T::KS; ++i)
#pragma unroll
    for (int j = 0; j < NH8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = FP8 ? g * (D / 8) + 2 * i + (e >> 1) : 16 * i + g + ((e >> 1) << 3);
        wo[(j * 8 + 2 * c + (e & 1)) * D + d] = o[i][j][e];
      }
  __syncthreads();

  for (int e = tid; e < heads * D; e += kThreads) {
    const int h = e / D, d = e - h * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, reinterpret_cast<const float*>(smem + w * T::WARP)[HW * D + h]);
    const float M0 = M == -INFINITY ? 0.f : M;
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* ws = reinterpret_cast<const float*>(smem + w * T::WARP);
      const float f = ex2(ws[HW * D + h] - M0);
      num += ws[h * D + d] * f;
      den += ws[HW * D + HW + h] * f;
    }
    const int hq = head0 + h;
    if (p.splits == 1) {
      float Z = den, f = 1.f, top = M0;
      if (p.sinks != nullptr) {
        const float sk = p.sinks[hq] * kLog2e;
        top = fmaxf(M, sk);
        if (top == -INFINITY) top = 0.f;
        f = ex2(M - top);
        Z = den * f + ex2(sk - top);
      }
      const float y = Z == 0.f ? 0.f : num * f / Z;
      p.out[row * p.out_stride_tok + hq * p.out_stride_head + d] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      if (d == 0 && p.lse != nullptr)
        p.lse[static_cast<int64_t>(row) * p.num_q_heads + hq] = (top + lg2(Z)) * kLn2;
    } else {
      const int64_t r = (static_cast<int64_t>(row) * p.num_q_heads + hq) * p.splits + split;
      p.o_part[r * D + d] = den == 0.f ? 0.f : num / den;
      if (d == 0) p.lse_part[r] = (M0 + lg2(den)) * kLn2;
    }
  }
  if (p.splits == 1) return;

  // ---- the split that finishes last merges ---------------------------------------
  // Partials, a fence, then the arrival; whoever completes the count acquires
  // them all and leaves the counter at zero.  No CTA waits for another.
  __syncthreads();
  int* last = reinterpret_cast<int*>(smem);
  if (tid == 0) {
    uint32_t* cnt = p.counters + static_cast<int64_t>(row) * gridDim.y + blockIdx.y;
    __threadfence();
    const bool done = atomicAdd(cnt, 1u) + 1 == static_cast<uint32_t>(p.splits);
    if (done) {
      atomicExch(cnt, 0u);
      __threadfence();
    }
    *last = done;
  }
  __syncthreads();
  if (*last) merge<D>(p, p.splits, row, head0, heads);
}

struct Variant {
  int tile_tokens, stages, smem0;   // smem0: without the page list
  int ctas;                         // that share an SM (by registers and shared memory)
};

template <int D, bool FP8, int NH8>
Variant variant_of() {
  using T = Tile<D, FP8, NH8>;
  const int smem = 1024 + kWarps * T::WARP + kWarps * T::NS * 8;
  return Variant{T::TS, T::NS, smem, std::min(Cfg<D, FP8, NH8>::CTAS, kMaxSmem / (smem + 2048))};
}

Variant variant(const pa_sparse_shape& s) {
  const bool fp8 = s.kv_dtype == PA_KV_FP8_E4M3, wide = std::min(s.num_q_heads / s.num_kv_heads, 16) > 8;
  switch (s.head_dim) {
    case 64:
      return fp8 ? (wide ? variant_of<64, true, 2>() : variant_of<64, true, 1>())
                 : (wide ? variant_of<64, false, 2>() : variant_of<64, false, 1>());
    case 128:
      return fp8 ? (wide ? variant_of<128, true, 2>() : variant_of<128, true, 1>())
                 : (wide ? variant_of<128, false, 2>() : variant_of<128, false, 1>());
    default:
      return fp8 ? (wide ? variant_of<256, true, 2>() : variant_of<256, true, 1>())
                 : (wide ? variant_of<256, false, 2>() : variant_of<256, false, 1>());
  }
}

template <int D, bool FP8>
cudaError_t launch(const CUtensorMap& tmk, const CUtensorMap& tmv, const SparseParams& p, dim3 grid, int smem,
                   cudaStream_t st) {
  const bool wide = std::min(p.group, 16) > 8, cap = p.cap_log2 > 0.f;
  auto kern = wide ? (cap ? sparse_attn_kernel<D, FP8, 2, true> : sparse_attn_kernel<D, FP8, 2, false>)
                   : (cap ? sparse_attn_kernel<D, FP8, 1, true> : sparse_attn_kernel<D, FP8, 1, false>);
  // The limit is the kernel's, not this call's (the longest list): of two host threads
  // that set a size of their own, one could launch under the other's.
  const int most = (wide ? variant_of<D, FP8, 2>() : variant_of<D, FP8, 1>()).smem0 + kMaxTopPages * 8;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, smem, st>>>(tmk, tmv, p);
  return cudaGetLastError();
}

int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// List entries of a split.
int list_entries(const pa_sparse_shape& s, int splits) { return (s.top_pages + splits - 1) / splits; }

}  // namespace

pa_status validate_sparse(const pa_sparse_shape& s) {
  if (s.num_q_heads <= 0 || s.num_kv_heads <= 0 || s.num_q_heads % s.num_kv_heads != 0) return PA_ERR_INVALID_ARG;
  if (s.max_batch < 0 || s.max_pages_per_seq < 0 || s.max_total_q < 0 || s.num_splits < 0 || s.num_sms < 0)
    return PA_ERR_INVALID_ARG;
  if (s.kv_dtype != PA_KV_BF16 && s.kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (s.has_sinks != 0 && s.has_sinks != 1) return PA_ERR_INVALID_ARG;
  if (!(s.soft_cap >= 0.f) || !std::isfinite(s.soft_cap)) return PA_ERR_INVALID_ARG;
  if (s.top_pages < 1 || s.first_pages < 0 || s.last_pages < 1 || s.first_pages > s.top_pages ||
      s.last_pages > s.top_pages - s.first_pages)
    return PA_ERR_INVALID_ARG;
  if (s.head_dim != 64 && s.head_dim != 128 && s.head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (s.page_size != 16 && s.page_size != 32 && s.page_size != 64) return PA_ERR_UNSUPPORTED;
  if (s.num_q_heads / s.num_kv_heads > 128 || s.num_kv_heads > 4096) return PA_ERR_UNSUPPORTED;
  if (s.max_pages_per_seq > kMaxSparsePages || s.top_pages > kMaxTopPages) return PA_ERR_UNSUPPORTED;
  if (s.max_total_q > (1 << 24) || s.max_batch > (1 << 24)) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Splits of each row: as many as keep the call one wave of the CTAs that the SMs
// hold, with at least 32 keys each, and 256 beyond sixteen (whose merging costs
// more than it gains).  Up to a quarter above one wave three splits fill the second
// one; stages of 64 keys do not divide so finely, and stay whole.
// Measured, rows of 2048 keys, 8 kv heads, head_dim 128 bf16 (us by splits): 1 row
// 1: 35.2, 8: 10.6, 16: 8.8, 32: 10.0, 64: 12.7; 16 rows 1: 50.9, 5: 30.7, 8: 35.3;
// 64 rows (512 pairs on 760 slots) 1: 86.6, 2: 96.5.  Pairs a slot, 1 / 2 / 3 splits:
//   bf16 D 128   1.0 126/133/137, 1.02 159/146/142, 1.15 165/152/150, 1.25 170/159/162, 1.4 175/176/184
//   e4m3 D 128   1.0 73/83/91, 1.03 102/97/98, 1.15 114/108/106, 1.25 113/110/111, 1.4 117/119/128
//   bf16 D 256   1.0 150/159/163, 1.02 187/170/167, 1.16 194/181/179, 1.25 198/189/193, 1.4 208/213/218
//   bf16 D 64    1.0 86/93/99, 1.02 108/102/102, 1.15 114/109/106, 1.25 114/113/115, 1.4 117/127/133
//   e4m3 D 64 (stages of 64)   1.0 69/79/87, 1.02 81/82/88, 1.15 94/94/96, 1.25 100/101/105
// The arrival counters of the scratch header bound the rows that may be split at all
// (a call beyond them has work enough).
int sparse_splits(const pa_sparse_shape& s, int64_t rows) {
  const int64_t pairs = rows * s.num_kv_heads * sparse_head_groups(s);
  if (pairs <= 0 || pairs > kMergeCounters) return 1;
  const int64_t keys = static_cast<int64_t>(s.top_pages) * s.page_size;
  if (s.num_splits > 0) return std::min(s.num_splits, s.top_pages);
  const Variant v = variant(s);
  const int64_t slots = static_cast<int64_t>(s.num_sms) * v.ctas;
  int64_t n = std::min({slots / pairs, keys / 32, std::max<int64_t>(16, keys / 256)});
  if (pairs > slots && 4 * pairs <= 5 * slots && v.tile_tokens < 64) n = std::min<int64_t>(3, keys / 256);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(n, s.top_pages)));
}

int64_t sparse_partial_bytes(const pa_sparse_shape& s, int64_t partial_rows) {
  const int64_t n = partial_rows * s.num_q_heads;
  return align_up(n * s.head_dim * 4, 256) + align_up(n * 4, 256);
}

int64_t sparse_score_bytes(const pa_sparse_shape& s, int64_t score_rows) {
  const int64_t n = score_rows * s.num_kv_heads;
  return align_up(n * score_pages(s) * 4, 256) + align_up(n * score_chunks(s) * 4, 256);
}

pa_status check_sparse_call(const pa_sparse_plan_t* plan, const int32_t* block_table, int64_t bt_stride,
                            const int32_t* seq_lens, const int32_t* qsl, int32_t batch, int32_t total_q,
                            const void* scratch, int64_t scratch_bytes) {
  if (!plan) return PA_ERR_INVALID_ARG;
  const pa_sparse_shape& s = plan->shape;
  if (validate_sparse(s) != PA_OK || s.num_sms <= 0) return PA_ERR_INVALID_ARG;
  if (batch < 0 || batch > s.max_batch || total_q < 0 || total_q > s.max_total_q) return PA_ERR_INVALID_ARG;
  if (!qsl && total_q != batch) return PA_ERR_INVALID_ARG;
  if (!scratch) return PA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(scratch) % 256) return PA_ERR_UNSUPPORTED;
  // a plan edited by hand must not index past the scratch it states
  if (plan->partial_rows < 0 || plan->score_rows < 1) return PA_ERR_INVALID_ARG;
  const int64_t need = kScratchHeaderBytes + std::max(sparse_partial_bytes(s, plan->partial_rows),
                                                      sparse_score_bytes(s, plan->score_rows));
  if (plan->scratch_bytes < need) return PA_ERR_INVALID_ARG;
  if (scratch_bytes < plan->scratch_bytes) return PA_ERR_SCRATCH_TOO_SMALL;
  if (batch == 0 || total_q == 0) return PA_OK;
  if (!block_table || !seq_lens || bt_stride < s.max_pages_per_seq) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_sparse_plan(const pa_sparse_shape* shape, pa_sparse_plan_t* plan) {
  if (!shape || !plan) return PA_ERR_INVALID_ARG;
  const pa_status st = validate_sparse(*shape);
  if (st != PA_OK) return st;
  pa_sparse_plan_t p;
  std::memset(&p, 0, sizeof p);
  p.shape = *shape;
  if (p.shape.num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&p.shape.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  const pa_sparse_shape& s = p.shape;
  const Variant v = variant(s);
  int64_t partial = 0;
  int fewest = 0;   // splits of the call that splits least: the longest page list of a CTA
  const int64_t split_rows =
      std::min<int64_t>(s.max_total_q, kMergeCounters / (static_cast<int64_t>(s.num_kv_heads) * sparse_head_groups(s)));
  for (int64_t r = 1; r <= split_rows; ++r) {
    const int n = sparse_splits(s, r);
    if (n > 1) partial = std::max(partial, r * n);
    fewest = r == 1 ? n : std::min(fewest, n);
  }
  if (split_rows < s.max_total_q || fewest < 1) fewest = 1;
  p.tile_tokens = v.tile_tokens;
  p.stages = v.stages;
  p.warps = kWarps;
  p.smem_bytes = v.smem0 + list_entries(s, fewest) * 8;
  if (p.smem_bytes > kMaxSmem) return PA_ERR_UNSUPPORTED;
  p.partial_rows = static_cast<int32_t>(partial);
  const int64_t row_bytes = std::max<int64_t>(1, s.num_kv_heads * score_pages(s) * 4);
  p.score_rows = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(s.max_total_q, kScoreBytes / row_bytes)));
  p.scratch_bytes =
      kScratchHeaderBytes + std::max(sparse_partial_bytes(s, p.partial_rows), sparse_score_bytes(s, p.score_rows));
  *plan = p;
  return PA_OK;
}

extern "C" pa_status pa_sparse_attend(const pa_sparse_plan_t* plan, const void* q, int64_t q_stride_tok,
                                      int64_t q_stride_head, const void* k_cache, const void* v_cache,
                                      int64_t kv_stride_page, int64_t kv_stride_tok, int64_t kv_stride_head,
                                      int32_t num_pages, const int32_t* block_table, int64_t bt_stride,
                                      const int32_t* seq_lens, const int32_t* query_start_loc, int32_t batch,
                                      int32_t total_q, const int32_t* pages, float scale, const float* sinks,
                                      float k_scale, float v_scale, const float* k_scales, const float* v_scales,
                                      void* out, int64_t out_stride_tok, int64_t out_stride_head, float* lse,
                                      void* scratch, int64_t scratch_bytes, void* stream) {
  pa_status st = check_sparse_call(plan, block_table, bt_stride, seq_lens, query_start_loc, batch, total_q, scratch,
                                   scratch_bytes);
  if (st != PA_OK) return st;
  const pa_sparse_shape& s = plan->shape;
  if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale)) return PA_ERR_INVALID_ARG;
  if ((sinks != nullptr) != (s.has_sinks != 0)) return PA_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0) return PA_OK;
  if (!q || !out || !pages || !k_cache || !v_cache || num_pages <= 0) return PA_ERR_INVALID_ARG;
  if (q_stride_tok <= 0 || q_stride_head <= 0 || out_stride_tok <= 0 || out_stride_head <= 0 || kv_stride_page <= 0 ||
      kv_stride_tok <= 0 || kv_stride_head <= 0)
    return PA_ERR_INVALID_ARG;
  auto at = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0; };
  const bool fp8 = s.kv_dtype == PA_KV_FP8_E4M3;
  const int e = fp8 ? 1 : 2;
  // q and out are accessed as bf16 pairs; the caches feed TMA
  if (!at(q, 4) || q_stride_tok % 2 || q_stride_head % 2 || !at(out, 4) || out_stride_tok % 2 ||
      out_stride_head % 2 || !at(lse, 4) || !at(pages, 4))
    return PA_ERR_UNSUPPORTED;
  if (!at(k_cache, 16) || !at(v_cache, 16) || (kv_stride_page * e) % 16 || (kv_stride_tok * e) % 16 ||
      (kv_stride_head * e) % 16)
    return PA_ERR_UNSUPPORTED;
  const int splits = sparse_splits(s, total_q);
  if (splits > 1 && static_cast<int64_t>(total_q) * splits > plan->partial_rows) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(total_q) * splits > INT32_MAX) return PA_ERR_UNSUPPORTED;
  const Variant v = variant(s);
  const int cap = list_entries(s, splits);
  const int smem = v.smem0 + cap * 8;
  if (plan->tile_tokens != v.tile_tokens || smem > kMaxSmem) return PA_ERR_INVALID_ARG;
  const int box_rows = std::min(s.page_size, v.tile_tokens);
  CUtensorMap tmk, tmv;
  if ((st = make_kv_map(&tmk, k_cache, fp8, s.head_dim, s.num_kv_heads, s.page_size, num_pages, kv_stride_page,
                        kv_stride_tok, kv_stride_head, box_rows)) != PA_OK)
    return st;
  if ((st = make_kv_map(&tmv, v_cache, fp8, s.head_dim, s.num_kv_heads, s.page_size, num_pages, kv_stride_page,
                        kv_stride_tok, kv_stride_head, box_rows)) != PA_OK)
    return st;
  SparseParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.batch = batch;
  p.num_q_heads = s.num_q_heads;
  p.num_kv_heads = s.num_kv_heads;
  p.group = s.num_q_heads / s.num_kv_heads;
  p.ps_log2 = __builtin_ctz(static_cast<unsigned>(s.page_size));
  p.num_pages = num_pages;
  p.max_len = static_cast<int64_t>(s.max_pages_per_seq) * s.page_size;
  p.max_pages = s.max_pages_per_seq;
  p.pages = pages;
  p.top = s.top_pages;
  p.scale_log2 = scale * kLog2e;
  p.cap_log2 = s.soft_cap > 0.f ? s.soft_cap * kLog2e : 0.f;
  p.scale_over_cap = s.soft_cap > 0.f ? scale / s.soft_cap : 0.f;
  p.sinks = sinks;
  p.k_scale = fp8 ? k_scale : 1.f;
  p.v_scale = fp8 ? v_scale : 1.f;
  p.k_scales = fp8 ? k_scales : nullptr;
  p.v_scales = fp8 ? v_scales : nullptr;
  p.out = static_cast<uint16_t*>(out);
  p.out_stride_tok = out_stride_tok;
  p.out_stride_head = out_stride_head;
  p.lse = lse;
  uint8_t* sc = static_cast<uint8_t*>(scratch);
  p.o_part = reinterpret_cast<float*>(sc + kScratchHeaderBytes);
  p.lse_part = p.o_part + align_up(static_cast<int64_t>(plan->partial_rows) * s.num_q_heads * s.head_dim * 4, 256) / 4;
  p.splits = splits;
  p.head_groups = sparse_head_groups(s);
  p.list_cap = cap;
  p.counters = reinterpret_cast<uint32_t*>(sc + kMergeCounterOffset);
  p.err = reinterpret_cast<uint32_t*>(sc);
  const dim3 grid(static_cast<unsigned>(total_q) * splits, s.num_kv_heads * p.head_groups);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  cudaError_t r;
  switch (s.head_dim) {
    case 64: r = fp8 ? launch<64, true>(tmk, tmv, p, grid, smem, str) : launch<64, false>(tmk, tmv, p, grid, smem, str); break;
    case 128: r = fp8 ? launch<128, true>(tmk, tmv, p, grid, smem, str) : launch<128, false>(tmk, tmv, p, grid, smem, str); break;
    default: r = fp8 ? launch<256, true>(tmk, tmv, p, grid, smem, str) : launch<256, false>(tmk, tmv, p, grid, smem, str); break;
  }
  return r == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
