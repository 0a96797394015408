// Attention over a paged cache of 8-bit codes (e4m3 or int8) with a scale for
// each page and kv head: K_j = code * k_scale[page][g], V_j likewise.
//
// Few rows a request (decode, drafted tokens): one split-KV kernel.
//   s_j = scale * ks * (q . code_j);  out = sum_j softmax(s)_j vs code_j
// The scales are constant over a page, so they never touch the elements: codes
// go into f16 matrix products as they are (both kinds are exact in f16), ks
// multiplies the score, and vs is carried by the weight.  With
//   x_j = s_j log2 e + log2 vs_j,  m = max x_j,  p_j = 2^(x_j - m + 14)
// the output is sum p_j code_j / sum p_j / vs_j: the weight that meets the codes
// is p itself, the addition of log2 vs rides in the score's multiply-add, and the
// denominator's 1 / vs in its own.  m bounds every term of the output, so p <= 2^14
// whatever the pages' scales are, and a weight in f16 is off by half a step,
// 2^-12, down to 2^-28 of the row's largest.  q enters in f16 as well, scaled by a
// power of two a row (largest value in [2^14, 2^15): exact to 2^-32 of it).
//
// The codes are read once from HBM, which bounds the kernel; per code it spends
// about a quarter of the instructions that dequantising to bf16 takes.  A CTA is a
// (split, kv head and group of up to 16 rows, request); its four warps take tiles
// of TS keys in turn, each with a private ring of stages filled by TMA from the
// pages.  S^T = K Q^T and O^T += V^T P^T keep the rows in the products' 8-wide
// dimension.  ldmatrix brings four codes of a key (K), or two codes of two
// neighbouring keys (V, transposed), into a register; which dims those are is a
// fixed permutation that the q fragments and the output follow.  Splits are merged
// by the CTA that finishes last, as in decode.
//
// Many rows a request (chunks): see "chunks" below.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "blocks.cuh"
#include "extend.h"
#include "pa.h"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxSmem = 232448;
constexpr float kWeightBias = 14.f;           // weights are at most 2^14 (f16 holds 65504)
constexpr float kLeastScale = 0x1p-100f;      // V scales below count as this one: its log2 and inverse are finite

struct BlockParams {
  const uint16_t* q;
  int64_t q_stride_tok, q_stride_head;
  const float* k_scales;
  const float* v_scales;
  int64_t scale_stride;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  const int32_t* qsl;         // null: one row a request
  int batch, total_q, max_new, max_kv;
  int num_q_heads, num_kv_heads, group, page_size, num_pages;
  float scale_log2, cap_log2, scale_over_cap;
  int window;
  const float* sinks;
  uint16_t* out;
  int64_t out_stride_tok, out_stride_head;
  float* lse;
  float* o_part;              // [total_q, Hq, max_splits, D] normalised split outputs
  float* lse_part;            // [total_q, Hq, max_splits]
  int max_splits, split_tiles, fixed_splits, bt_cache, row_groups;
  uint32_t* merge_cnt;        // [batch, Hkv * row_groups] arrival counters
  uint32_t* err;
};

// log2 of a V scale and its inverse, of the K scale: what a page's keys need.
struct PageScale {
  float k, v_log2, v_inv, pad;
};

template <int D, int NH8, int TS, int NS>
struct Traits {
  static constexpr int RB = D < 128 ? D : 128;      // bytes per TMA box row
  static constexpr int NCC = D / RB;                // column chunks per key row
  static constexpr int TILE = TS * D;               // K (or V) bytes per stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int WARP_BYTES = NS * STAGE;
  static constexpr int MT = TS / 16;
  static constexpr int KS = D / 16;                 // 16-code units per row
  static constexpr int HW = NH8 * 8;
  static_assert(RB == 128 || RB == 64, "row bytes must use the 128B or 64B swizzle");
  static_assert(WARP_BYTES >= HW * (D + 2) * 4, "a warp's final state fits in its ring");

  // Byte offset of 16-byte unit `u` of key row `row` as TMA writes it.
  __device__ static __forceinline__ uint32_t unit(int row, int u) {
    constexpr int UPB = RB / 16;
    const int cc = u / UPB;
    const uint32_t sw = (RB == 128) ? (row & 7) : ((row >> 1) & 3);
    return static_cast<uint32_t>(cc * (TS * RB) + row * RB) + (((u % UPB) ^ sw) << 4);
  }
};

struct Split {
  int lo, hi;            // attended keys of the request [lo, hi)
  int tile0, n_tiles, per, n;
};

__device__ __forceinline__ Split split_of(const BlockParams& p, int L, int n_new, int ts) {
  Split r;
  r.hi = L;
  r.lo = p.window > 0 ? max(0, L - n_new - p.window + 1) : 0;
  r.tile0 = r.lo / ts;
  r.n_tiles = (r.hi + ts - 1) / ts - r.tile0;
  r.per = p.fixed_splits > 0 ? (r.n_tiles + p.fixed_splits - 1) / p.fixed_splits : p.split_tiles;
  r.n = (r.n_tiles + r.per - 1) / r.per;
  r.per = (r.n_tiles + r.n - 1) / r.n;      // equal splits
  r.n = (r.n_tiles + r.per - 1) / r.per;
  return r;
}

// Splits of the R rows of one group, merged by their LSEs: thread t takes 4
// consecutive dims of one row, eight splits' loads in flight together.
template <int D>
__device__ __forceinline__ void merge_rows(const BlockParams& p, int n_splits, int R, int row0, int kvh, int64_t qs) {
  constexpr int C = D / 4;
  constexpr int U = 8;
  for (int e = threadIdx.x; e < R * C; e += kWarps * 32) {
    const int rr = e / C;
    const int d = (e - rr * C) * 4;
    const int tq = (row0 + rr) / p.group;
    const int hq = kvh * p.group + (row0 + rr - tq * p.group);
    const int64_t orow = qs + tq;
    const int64_t at = (orow * p.num_q_heads + hq) * p.max_splits;
    const bool has_sink = p.sinks != nullptr;
    float M = has_sink ? p.sinks[hq] * kLog2e : -INFINITY;
    float Z = has_sink ? 1.f : 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < n_splits; s0 += U) {
      float l[U];
      float4 o[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = s0 + u < n_splits;
        l[u] = ok ? __ldcg(p.lse_part + at + s0 + u) * kLog2e : -INFINITY;
        o[u] = ok ? __ldcg(reinterpret_cast<const float4*>(p.o_part + (at + s0 + u) * D + d))
                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mx = l[0];
#pragma unroll
      for (int u = 1; u < U; ++u) mx = fmaxf(mx, l[u]);
      if (mx > M) {
        const float f = ex2(M - mx);
        Z *= f;
        acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
        M = mx;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (l[u] == -INFINITY) continue;      // padding, or a split with no key for this row
        const float w = ex2(l[u] - M);
        Z += w;
        acc.x += w * o[u].x; acc.y += w * o[u].y; acc.z += w * o[u].z; acc.w += w * o[u].w;
      }
    }
    const float inv = Z > 0.f ? 1.f / Z : 0.f;
    uint16_t* outp = p.out + orow * p.out_stride_tok + static_cast<int64_t>(hq) * p.out_stride_head + d;
    reinterpret_cast<uint32_t*>(outp)[0] = pack_bf16x2(acc.x * inv, acc.y * inv);
    reinterpret_cast<uint32_t*>(outp)[1] = pack_bf16x2(acc.z * inv, acc.w * inv);
    if (d == 0 && p.lse != nullptr)
      p.lse[orow * p.num_q_heads + hq] = M == -INFINITY ? -INFINITY : (M + lg2(Z)) * kLn2;
  }
}

template <int D, bool I8, int NH8, int TS, int NS, bool CAP>
__global__ void __launch_bounds__(kWarps * 32)
block_split_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const BlockParams p) {
  using T = Traits<D, NH8, TS, NS>;
  const int split = blockIdx.x;
  const int kvh = blockIdx.y / p.row_groups;
  const int rg = blockIdx.y - kvh * p.row_groups;
  const int b = blockIdx.z;
  const int L = p.seq_lens[b];
  const int qs = p.qsl != nullptr ? p.qsl[b] : b;
  const int n_new = p.qsl != nullptr ? p.qsl[b + 1] - qs : 1;
  const int G = p.group;
  const int tid = threadIdx.x;
  const bool leads = tid == 0 && split == 0 && blockIdx.y == 0;
  if (n_new == 0) return;
  if (n_new < 0 || n_new > p.max_new || qs < 0 || static_cast<int64_t>(qs) + n_new > p.total_q || L < 0 ||
      L > p.max_kv || (p.qsl != nullptr && L < n_new)) {
    if (leads) atomicOr(p.err, kErrCapacity);
    return;
  }
  const int row0 = rg * (NH8 * 8);                       // first (token, head) row of this CTA
  const int R = min(n_new * G - row0, NH8 * 8);
  if (R <= 0) return;
  if (L == 0) {        // (decode of an empty request) no key: O = 0, LSE the sink's or -inf
    if (split == 0)
      for (int i = tid; i < R * D; i += kWarps * 32) {
        const int rr = i / D, d = i - rr * D;
        const int hq = kvh * G + row0 + rr;
        p.out[static_cast<int64_t>(qs) * p.out_stride_tok + static_cast<int64_t>(hq) * p.out_stride_head + d] = 0;
        if (d == 0 && p.lse != nullptr)
          p.lse[static_cast<int64_t>(qs) * p.num_q_heads + hq] = p.sinks != nullptr ? p.sinks[hq] : -INFINITY;
      }
    return;
  }
  const Split r = split_of(p, L, n_new, TS);
  if (split >= r.n) return;
  if (r.n > p.max_splits) {                              // a length beyond the planned capacity
    if (leads) atomicOr(p.err, kErrCapacity);
    return;
  }
  const int tile_begin = r.tile0 + split * r.per;
  const int tile_end = min(tile_begin + r.per, r.tile0 + r.n_tiles);
  const int tok_lo = max(r.lo, tile_begin * TS);
  const int tok_hi = min(r.hi, tile_end * TS);
  const int ps = p.page_size;
  const int ps_log2 = __ffs(ps) - 1;
  const int pg0 = (tile_begin * TS) >> ps_log2;
  const int pg1 = (tok_hi + ps - 1) >> ps_log2;          // <= ceil(L / ps)
  // tiles where every row sees every key need no mask per element
  const int pos_first = L - n_new;
  const int lo_last = p.window > 0 ? L - p.window : 0;
  const int full_lo = max(tok_lo, lo_last);
  const int full_hi = min(tok_hi, pos_first + 1);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * T::WARP_BYTES);
  PageScale* sc_s = reinterpret_cast<PageScale*>(bars + ((kWarps * NS + 1) & ~1));
  int32_t* bt_s = reinterpret_cast<int32_t*>(sc_s + p.bt_cache);

  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int g = lane >> 2;
  const int c = lane & 3;

  // (a split longer than its slice of the table would be a planner's mistake; it
  // still reports to the merge)
  const bool bt_fits = pg1 - pg0 <= p.bt_cache;
  if (!bt_fits && tid == 0) atomicOr(p.err, kErrSchedOverflow);
  const int n_tiles = bt_fits ? tile_end - tile_begin : 0;
  const int n_pages = bt_fits ? pg1 - pg0 : 0;
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(b) * p.bt_stride + pg0;
  // a page id outside the pool becomes the coordinate num_pages, whose box reads as zeros
  for (int i = tid; i < n_pages; i += kWarps * 32) {
    int id = bt_row[i];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
      if (((pg0 + i + 1) << ps_log2) > tok_lo) atomicOr(p.err, kErrPageId);
      id = p.num_pages;
    }
    bt_s[i] = id;
  }
  if (tid == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    for (int i = 0; i < kWarps * NS; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  __syncthreads();

  uint8_t* wbase = smem + warp * T::WARP_BYTES;
  uint64_t* wbar = bars + warp * NS;

  // Lane 0: fetch local tile k into `stage`.  Boxes wholly past the end of the
  // sequence are not fetched; their rows are masked.
  auto issue = [&](int k, int stage) {
    const int t0 = (tile_begin + k) * TS;
    const int br = ps < TS ? ps : TS;
    int nb = 0;
    for (int j = 0; j < TS / br; ++j) nb += (t0 + j * br < L) ? 1 : 0;
    uint8_t* kst = wbase + stage * T::STAGE;
    uint8_t* vst = kst + T::TILE;
    mbar_arrive_expect_tx(&wbar[stage], static_cast<uint32_t>(nb * br * D * 2));
    for (int j = 0; j < nb; ++j) {
      const int t = t0 + j * br;
      const int page = bt_s[(t >> ps_log2) - pg0];
      const int slot = t & (ps - 1);
#pragma unroll
      for (int cc = 0; cc < T::NCC; ++cc) {
        const int dst = cc * TS * T::RB + j * br * T::RB;
        tma_load_4d(kst + dst, &tmk, cc * T::RB, kvh, slot, page, &wbar[stage]);
        tma_load_4d(vst + dst, &tmv, cc * T::RB, kvh, slot, page, &wbar[stage]);
      }
    }
  };
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) {
      const int k = warp + s * kWarps;
      if (k < n_tiles) issue(k, s);
    }
  }
  __syncwarp();

  // scales of this head's pages (under the first tiles' loads); a page wholly before the
  // window adds nothing, whatever its scales hold by now
  for (int i = tid; i < n_pages; i += kWarps * 32) {
    const int id = bt_s[i];
    const bool in = id < p.num_pages && ((pg0 + i + 1) << ps_log2) > tok_lo;
    const int64_t at = static_cast<int64_t>(in ? id : 0) * p.scale_stride + kvh;
    const float ks = in ? p.k_scales[at] : 0.f;
    const float vs = in ? fmaxf(p.v_scales[at], kLeastScale) : kLeastScale;
    sc_s[i] = PageScale{ks, lg2(vs), 1.f / vs, 0.f};
  }

  // Q^T fragments (B operand): unit ks of a row holds dims 16 ks ..; thread c has
  // codes 4c .. 4c + 3 of it.  Each row times 2^e with its largest value in [2^14, 2^15).
  uint32_t qf[T::KS][NH8][2];
  float rsl[NH8][2];         // the score factor of this thread's two accumulator rows
#pragma unroll
  for (int j = 0; j < NH8; ++j) {
    const int rr = j * 8 + g;
    const bool ok = rr < R;
    const int tq = ok ? (row0 + rr) / G : 0;
    const int hq = ok ? row0 + rr - tq * G : 0;
    const uint16_t* qh = p.q + static_cast<int64_t>(qs + tq) * p.q_stride_tok +
                         static_cast<int64_t>(kvh * G + hq) * p.q_stride_head + 4 * c;
    uint32_t most = 0;
#pragma unroll
    for (int ks = 0; ks < T::KS; ++ks) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = ok ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + 2 * h) : 0u;
        qf[ks][j][h] = w;
        most = max(most, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
      }
    }
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const uint32_t e = max(most >> 7, 15u);              // biased exponent of the row's largest value
    const float up = __uint_as_float((268u - e) << 23);  // 2^(14 - (e - 127))
#pragma unroll
    for (int ks = 0; ks < T::KS; ++ks)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = qf[ks][j][h];
        qf[ks][j][h] = pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t er = __shfl_sync(0xffffffffu, e, (2 * c + h) * 4);
      rsl[j][h] = (CAP ? p.scale_over_cap : p.scale_log2) * __uint_as_float((er - 14u) << 23);
    }
  }

  float o[T::KS][NH8][4];
#pragma unroll
  for (int i = 0; i < T::KS; ++i)
#pragma unroll
    for (int j = 0; j < NH8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
  float m_run[NH8][2], l_run[NH8][2];
  int rpos[NH8][2], rlo[NH8][2];      // this thread's two rows: last and first attended key
#pragma unroll
  for (int j = 0; j < NH8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m_run[j][h] = -INFINITY;
      l_run[j][h] = 0.f;
      rpos[j][h] = pos_first + (row0 + min(j * 8 + 2 * c + h, R - 1)) / G;
      rlo[j][h] = p.window > 0 ? rpos[j][h] - p.window + 1 : 0;
    }
  __syncthreads();                    // sc_s

  const int mi = lane >> 3, mr = lane & 7;
  int it = 0;
  for (int k = warp; k < n_tiles; k += kWarps, ++it) {
    const int stage = it % NS;
    const uint32_t parity = static_cast<uint32_t>((it / NS) & 1);
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&wbar[stage], parity, p.err));
    if (!ok) break;
    const uint32_t kst_u = smem_u32(wbase + stage * T::STAGE);
    const uint32_t vst_u = kst_u + T::TILE;
    const int t0 = (tile_begin + k) * TS;
    const bool partial = (t0 < full_lo) || (t0 + TS > full_hi);

    // ---- S^T = K Q^T over the codes ----------------------------------------
    float s[T::MT][NH8][4];
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt) {
#pragma unroll
      for (int j = 0; j < NH8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
      const int row = mt * 16 + mr + ((mi & 1) << 3);
#pragma unroll
      for (int u = 0; u < T::KS; u += 2) {
        uint32_t w[4];               // keys 0-7 and 8-15 of unit u, then of unit u + 1
        ldsm_x4(w, kst_u + T::unit(row, u + (mi >> 1)));
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint32_t a[4];
          if constexpr (I8) {
            const uint32_t x0 = w[2 * v] ^ 0x80808080u, x1 = w[2 * v + 1] ^ 0x80808080u;
            a[0] = int8x2_to_f16x2<0x4140>(x0);
            a[1] = int8x2_to_f16x2<0x4140>(x1);
            a[2] = int8x2_to_f16x2<0x4342>(x0);
            a[3] = int8x2_to_f16x2<0x4342>(x1);
          } else {
            a[0] = e4m3x2_to_f16x2<0>(w[2 * v]);
            a[1] = e4m3x2_to_f16x2<0>(w[2 * v + 1]);
            a[2] = e4m3x2_to_f16x2<1>(w[2 * v]);
            a[3] = e4m3x2_to_f16x2<1>(w[2 * v + 1]);
          }
#pragma unroll
          for (int j = 0; j < NH8; ++j) mma_f16(s[mt][j], a, qf[u + v][j][0], qf[u + v][j][1]);
        }
      }
    }

    // ---- scales, soft-cap, mask; online softmax (log2 domain) --------------
    // (the 16 keys of an m-tile lie in one page)
    float mx[NH8][2];
    float v_inv[T::MT];
#pragma unroll
    for (int j = 0; j < NH8; ++j) mx[j][0] = mx[j][1] = -INFINITY;
    auto scores = [&](auto masked_tag) {
      constexpr bool MASKED = decltype(masked_tag)::value;
#pragma unroll
      for (int mt = 0; mt < T::MT; ++mt) {
        // (a tile's last m-tiles may lie behind the request's last page)
        const int pg = min(((t0 + mt * 16) >> ps_log2), pg1 - 1) - pg0;
        const float4 ps4 = *reinterpret_cast<const float4*>(&sc_s[pg]);
        v_inv[mt] = ps4.z;
#pragma unroll
        for (int j = 0; j < NH8; ++j) {
          const float f[2] = {ps4.x * rsl[j][0], ps4.x * rsl[j][1]};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v;
            if constexpr (CAP) {
              v = fmaf(p.cap_log2, tanhf(s[mt][j][e] * f[e & 1]), ps4.y);
            } else {
              v = fmaf(s[mt][j][e], f[e & 1], ps4.y);
            }
            if constexpr (MASKED) {
              const int tok = t0 + mt * 16 + g + ((e >> 1) << 3);
              if (tok < tok_lo || tok >= tok_hi || tok > rpos[j][e & 1] || tok < rlo[j][e & 1]) v = -INFINITY;
            }
            s[mt][j][e] = v;
            mx[j][e & 1] = fmaxf(mx[j][e & 1], v);
          }
        }
      }
    };
    if (partial) {
      scores(std::true_type{});
    } else {
      scores(std::false_type{});
    }
    float alpha[NH8][2], mu[NH8][2];
    bool grew = false;
#pragma unroll
    for (int j = 0; j < NH8; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float m = mx[j][h];
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        const float m_new = fmaxf(m_run[j][h], m);
        const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
        grew |= m_new > m_run[j][h];
        alpha[j][h] = ex2(m_run[j][h] - m_use);
        m_run[j][h] = m_new;
        mu[j][h] = m_use - kWeightBias;
      }
    const bool rescale = __any_sync(0xffffffffu, grew);
#pragma unroll
    for (int j = 0; j < NH8; ++j) {
      float ls0 = 0.f, ls1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < T::MT; ++mt) {
        s[mt][j][0] = ex2(s[mt][j][0] - mu[j][0]);
        s[mt][j][1] = ex2(s[mt][j][1] - mu[j][1]);
        s[mt][j][2] = ex2(s[mt][j][2] - mu[j][0]);
        s[mt][j][3] = ex2(s[mt][j][3] - mu[j][1]);
        ls0 = fmaf(s[mt][j][0] + s[mt][j][2], v_inv[mt], ls0);
        ls1 = fmaf(s[mt][j][1] + s[mt][j][3], v_inv[mt], ls1);
      }
      l_run[j][0] = fmaf(l_run[j][0], alpha[j][0], ls0);
      l_run[j][1] = fmaf(l_run[j][1], alpha[j][1], ls1);
      if (rescale) {
#pragma unroll
        for (int i = 0; i < T::KS; ++i) {
          o[i][j][0] *= alpha[j][0];
          o[i][j][1] *= alpha[j][1];
          o[i][j][2] *= alpha[j][0];
          o[i][j][3] *= alpha[j][1];
        }
      }
    }

    // ---- O^T += V^T P^T over the codes ---------------------------------------
    auto pv = [&](auto mask_tag) {
      constexpr bool MASK = decltype(mask_tag)::value;
#pragma unroll
      for (int mt = 0; mt < T::MT; ++mt) {
        uint32_t pb[NH8][2];
#pragma unroll
        for (int j = 0; j < NH8; ++j) {
          pb[j][0] = movmatrix_t(pack_f16x2(s[mt][j][0], s[mt][j][1]));
          pb[j][1] = movmatrix_t(pack_f16x2(s[mt][j][2], s[mt][j][3]));
        }
        // masked keys have P = 0, but their codes may be stale (NaN in e4m3): zeroed
        uint32_t vm_lo = 0xffffffffu, vm_hi = 0xffffffffu;
        if constexpr (MASK) {
          const int tk = t0 + mt * 16 + 2 * c;
          auto valid = [&](int t) { return t >= tok_lo && t < tok_hi; };
          vm_lo = (valid(tk) ? 0x0000ffffu : 0u) | (valid(tk + 1) ? 0xffff0000u : 0u);
          vm_hi = (valid(tk + 8) ? 0x0000ffffu : 0u) | (valid(tk + 9) ? 0xffff0000u : 0u);
        }
        const int row = mt * 16 + mr + ((mi & 1) << 3);
#pragma unroll
        for (int u = 0; u < T::KS; u += 2) {
          uint32_t w[4];             // of unit u: keys 0-7, 8-15; then of unit u + 1
          ldsm_x4_t(w, vst_u + T::unit(row, u + (mi >> 1)));
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            // bytes of w: dims 2g, 2g + 1 of key 2c, then of key 2c + 1.  Row g of the
            // product is dim 2g of the unit, row g + 8 dim 2g + 1
            uint32_t a[4];
            if constexpr (I8) {
              const uint32_t x0 = w[2 * v] ^ 0x80808080u, x1 = w[2 * v + 1] ^ 0x80808080u;
              a[0] = int8x2_to_f16x2<0x4240>(x0);
              a[1] = int8x2_to_f16x2<0x4341>(x0);
              a[2] = int8x2_to_f16x2<0x4240>(x1);
              a[3] = int8x2_to_f16x2<0x4341>(x1);
            } else {
              const uint32_t x0 = __byte_perm(w[2 * v], 0, 0x3120), x1 = __byte_perm(w[2 * v + 1], 0, 0x3120);
              a[0] = e4m3x2_to_f16x2<0>(x0);
              a[1] = e4m3x2_to_f16x2<1>(x0);
              a[2] = e4m3x2_to_f16x2<0>(x1);
              a[3] = e4m3x2_to_f16x2<1>(x1);
            }
            if constexpr (MASK) {
              a[0] &= vm_lo;
              a[1] &= vm_lo;
              a[2] &= vm_hi;
              a[3] &= vm_hi;
            }
#pragma unroll
            for (int j = 0; j < NH8; ++j) mma_f16(o[u + v][j], a, pb[j][0], pb[j][1]);
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
    const int kn = k + NS * kWarps;
    if (lane == 0 && kn < n_tiles) {
      fence_proxy_async_smem();
      issue(kn, stage);
    }
  }

  // ---- merge the four warps' states in shared memory -----------------------
  // (every copy a warp issued was waited for in its loop, or an expired wait ended
  // the loop: then its copies may still land in this region, and the call's
  // results are void)
  float* wo = reinterpret_cast<float*>(wbase);   // [HW][D]
  float* wm = wo + T::HW * D;
  float* wl = wm + T::HW;
#pragma unroll
  for (int j = 0; j < NH8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_run[j][h];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) {
        wm[j * 8 + 2 * c + h] = m_run[j][h];
        wl[j * 8 + 2 * c + h] = l;
      }
    }
#pragma unroll
  for (int i = 0; i < T::KS; ++i)
#pragma unroll
    for (int j = 0; j < NH8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float2*>(wo + (j * 8 + 2 * c + e) * D + 16 * i + 2 * g) =
            make_float2(o[i][j][e], o[i][j][e + 2]);
  __syncthreads();

  const bool direct = (r.n == 1);
  for (int e = tid; e < R * D; e += kWarps * 32) {
    const int h = e / D;
    const int d = e - h * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      M = fmaxf(M, (reinterpret_cast<const float*>(smem + w * T::WARP_BYTES) + T::HW * D)[h]);
    if (M == -INFINITY) M = 0.f;
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* wob = reinterpret_cast<const float*>(smem + w * T::WARP_BYTES);
      const float f = ex2(wob[T::HW * D + h] - M);
      num += wob[h * D + d] * f;
      den += wob[T::HW * D + T::HW + h] * f;
    }
    const int tq = (row0 + h) / G;
    const int hq = kvh * G + (row0 + h - tq * G);
    const int64_t orow = qs + tq;
    // den = sum 2^(x - M + 14) / vs: the row's LSE is M - 14 + log2 den
    const float lse2 = den == 0.f ? -INFINITY : M - kWeightBias + lg2(den);
    const float ov = den == 0.f ? 0.f : num / den;
    if (direct) {
      float f = 1.f, total = lse2;
      if (p.sinks != nullptr) {
        const float sk = p.sinks[hq] * kLog2e;
        const float top = fmaxf(lse2, sk);
        const float z = ex2(lse2 - top) + ex2(sk - top);
        f = ex2(lse2 - top) / z;
        total = top + lg2(z);
      }
      p.out[orow * p.out_stride_tok + static_cast<int64_t>(hq) * p.out_stride_head + d] =
          __bfloat16_as_ushort(__float2bfloat16_rn(ov * f));
      if (d == 0 && p.lse != nullptr) p.lse[orow * p.num_q_heads + hq] = total * kLn2;
    } else {
      const int64_t row = (orow * p.num_q_heads + hq) * p.max_splits + split;
      p.o_part[row * D + d] = ov;
      if (d == 0) p.lse_part[row] = lse2 * kLn2;
    }
  }
  if (direct) return;

  // ---- the last split of these rows to finish merges --------------------------
  __syncthreads();
  int* s_last = reinterpret_cast<int*>(smem);
  if (tid == 0) {
    uint32_t* cnt = p.merge_cnt + static_cast<int64_t>(b) * gridDim.y + blockIdx.y;
    __threadfence();
    const uint32_t prev = atomicAdd(cnt, 1u);
    const int last = prev + 1 == static_cast<uint32_t>(r.n);
    if (last) {
      atomicExch(cnt, 0u);
      __threadfence();
    }
    *s_last = last;
  }
  __syncthreads();
  if (*s_last == 0) return;
  merge_rows<D>(p, r.n, R, row0, kvh, qs);
}

// Keys per stage and stages per warp.
template <int D> struct Choice;
template <> struct Choice<64> { static constexpr int TS = 32, NS = 3; };
template <> struct Choice<128> { static constexpr int TS = 32, NS = 2; };
template <> struct Choice<256> { static constexpr int TS = 16, NS = 3; };

int tile_of(int D) { return D == 64 ? Choice<64>::TS : D == 128 ? Choice<128>::TS : Choice<256>::TS; }

template <int D>
int smem_of(int bt_cache) {
  using C = Choice<D>;
  return 1024 + kWarps * C::NS * 2 * C::TS * D + ((kWarps * C::NS + 1) & ~1) * 8 +
         bt_cache * static_cast<int>(sizeof(PageScale) + 4);
}

int smem_bytes(int D, int bt_cache) {
  return D == 64 ? smem_of<64>(bt_cache) : D == 128 ? smem_of<128>(bt_cache) : smem_of<256>(bt_cache);
}

template <int D, bool I8, int NH8>
cudaError_t launch_split(const CUtensorMap& tmk, const CUtensorMap& tmv, const BlockParams& p, dim3 grid, int smem,
                         cudaStream_t stream) {
  using C = Choice<D>;
  auto kern = p.cap_log2 > 0.f ? block_split_kernel<D, I8, NH8, C::TS, C::NS, true>
                               : block_split_kernel<D, I8, NH8, C::TS, C::NS, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kWarps * 32, smem, stream>>>(tmk, tmv, p);
  return cudaGetLastError();
}

// ---- chunks ------------------------------------------------------------------
// Many rows a request are bound by the products, so they run on the tcgen05
// kernel of pa_extend, whose operands are 16 bits wide: every attended page is
// first copied, once, into the scratch workspace (page i of request b at copy page
// b * maxp + i), which every query tile reads: the codes of K as bf16 and those of V as
// f16, both exact, and the page's scales, which that kernel's softmax folds in.
// Requests whose copies exceed kMaxCopyBytes together are taken in groups, one
// after the other through the same copy.
constexpr int64_t kMaxCopyBytes = int64_t{2} << 30;

struct CopyParams {
  const uint8_t* k;
  const uint8_t* v;
  int64_t stride_page, stride_tok, stride_head;   // bytes
  const float* k_scales;
  const float* v_scales;
  int64_t scale_stride;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  const int32_t* qsl;
  int num_pages, page_size, num_kv_heads, window, maxp, max_kv, total_q;
  uint16_t* kc;
  uint16_t* vc;
  float2* page_scales;        // [copy page][Hkv]: K scale, log2 of the V scale
  int32_t* bt_copy;
  uint32_t* err;
};

// Sixteen codes as 16-bit numbers, exactly: f16, or bf16 by way of fp32.
template <bool I8, bool BF16>
__device__ __forceinline__ void widen_unit(const uint4& w, uint4* dst) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (I8) {
      const uint32_t x = in[k] ^ 0x80808080u;
      out[2 * k] = int8x2_to_f16x2<0x4140>(x);
      out[2 * k + 1] = int8x2_to_f16x2<0x4342>(x);
    } else {
      out[2 * k] = e4m3x2_to_f16x2<0>(in[k]);
      out[2 * k + 1] = e4m3x2_to_f16x2<1>(in[k]);
    }
  }
  if constexpr (BF16) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&out[k]));
      out[k] = pack_bf16x2(f.x, f.y);
    }
  }
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// One CTA a (page of a request, request).
template <int D, bool I8>
__global__ void __launch_bounds__(256) block_copy_kernel(const CopyParams p) {
  const int i = blockIdx.x;
  const int b = blockIdx.y;
  const int64_t dst_page = static_cast<int64_t>(b) * p.maxp + i;
  if (threadIdx.x == 0) p.bt_copy[dst_page] = static_cast<int32_t>(dst_page);
  const int L = p.seq_lens[b];
  const int qs = p.qsl[b];
  const int n = p.qsl[b + 1] - qs;
  const int ctx = L - n;
  if (n <= 0 || ctx < 0 || L > p.max_kv || qs < 0 || static_cast<int64_t>(qs) + n > p.total_q) return;
  const int ps = p.page_size;
  const int first = p.window > 0 ? max(0, ctx - p.window + 1) : 0;
  if ((i + 1) * ps <= first || i * ps >= L) return;
  const int src = p.block_table[static_cast<int64_t>(b) * p.bt_stride + i];
  constexpr int UPH = D / 16;
  const int units = ps * p.num_kv_heads * UPH;
  const int64_t page_elems = static_cast<int64_t>(ps) * p.num_kv_heads * D;
  uint4* kd = reinterpret_cast<uint4*>(p.kc + dst_page * page_elems);
  uint4* vd = reinterpret_cast<uint4*>(p.vc + dst_page * page_elems);
  if (src < 0 || src >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrPageId);
    for (int u = threadIdx.x; u < 2 * units; u += blockDim.x) {
      kd[u] = make_uint4(0, 0, 0, 0);
      vd[u] = make_uint4(0, 0, 0, 0);
    }
    for (int h = threadIdx.x; h < p.num_kv_heads; h += blockDim.x)
      p.page_scales[dst_page * p.num_kv_heads + h] = make_float2(0.f, lg2(kLeastScale));
    return;
  }
  for (int h = threadIdx.x; h < p.num_kv_heads; h += blockDim.x) {
    const int64_t at = static_cast<int64_t>(src) * p.scale_stride + h;
    p.page_scales[dst_page * p.num_kv_heads + h] = make_float2(p.k_scales[at], lg2(fmaxf(p.v_scales[at], kLeastScale)));
  }
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    const int tok = u / (p.num_kv_heads * UPH);
    const int rem = u - tok * (p.num_kv_heads * UPH);
    const int head = rem / UPH;
    const int64_t off = static_cast<int64_t>(src) * p.stride_page + static_cast<int64_t>(tok) * p.stride_tok +
                        static_cast<int64_t>(head) * p.stride_head + (rem - head * UPH) * 16;
    widen_unit<I8, true>(*reinterpret_cast<const uint4*>(p.k + off), kd + 2 * u);
    widen_unit<I8, false>(*reinterpret_cast<const uint4*>(p.v + off), vd + 2 * u);
  }
}

int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

pa_shape as_shape(const pa_block_shape& s, int mode) {
  pa_shape e{};
  e.mode = mode;
  e.num_q_heads = s.num_q_heads;
  e.num_kv_heads = s.num_kv_heads;
  e.head_dim = s.head_dim;
  e.page_size = s.page_size;
  e.kv_dtype = PA_KV_BF16;
  e.max_batch = s.max_batch;
  e.max_pages_per_seq = s.max_pages_per_seq;
  e.max_total_q = s.max_total_q;
  e.window = s.window;
  e.has_sinks = s.has_sinks;
  e.soft_cap = s.soft_cap;
  e.num_splits = s.num_splits;
  e.num_sms = s.num_sms;
  return e;
}

int64_t copy_bytes_a_request(const pa_block_shape& s) {      // K (or V), 16 bits
  return static_cast<int64_t>(s.max_pages_per_seq) * s.page_size * s.num_kv_heads * s.head_dim * 2;
}

struct ChunkScratch {
  int64_t work, table, scales, k, v, end;     // offsets
};

ChunkScratch chunk_scratch(const pa_block_shape& s, int64_t group) {
  ChunkScratch c;
  c.work = kScratchHeaderBytes;
  c.table = c.work + align_up(extend_work_capacity(as_shape(s, PA_MODE_EXTEND)) * 32, 256);
  c.scales = c.table + align_up(group * s.max_pages_per_seq * 4, 256);
  c.k = c.scales + align_up(group * s.max_pages_per_seq * s.num_kv_heads * 8, 256);
  c.v = c.k + align_up(group * copy_bytes_a_request(s), 256);
  c.end = c.v + align_up(group * copy_bytes_a_request(s), 256);
  return c;
}

int rows_of(const pa_block_shape& s) { return std::max(s.max_new, 1) * (s.num_q_heads / s.num_kv_heads); }
int nh8_of(const pa_block_shape& s) { return rows_of(s) <= 8 ? 1 : 2; }

int64_t partial_rows(const pa_block_shape& s, int64_t max_splits) {
  return static_cast<int64_t>(s.max_total_q) * s.num_q_heads * max_splits;
}

int64_t split_scratch(const pa_block_shape& s, int64_t max_splits) {
  const int64_t rows = max_splits > 1 ? partial_rows(s, max_splits) : 0;
  return kScratchHeaderBytes + align_up(rows * s.head_dim * 4, 256) + align_up(rows * 4, 256);
}

// Above this many rows a kv head (of one request) the chunked form is taken.
constexpr int kSplitRows = 64;

pa_status validate(const pa_block_shape& s) {
  if (s.code != PA_CODE_E4M3 && s.code != PA_CODE_INT8) return PA_ERR_INVALID_ARG;
  if (s.max_new < 1) return PA_ERR_INVALID_ARG;
  const pa_status st = validate_shape(as_shape(s, PA_MODE_EXTEND));
  if (st != PA_OK) return st;
  if (s.max_batch > 65535) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

pa_status plan_split(const pa_block_shape& s, const int32_t* lens, int32_t batch, int num_sms, pa_block_plan_t* out) {
  const int TS = tile_of(s.head_dim);
  const int NH = nh8_of(s) * 8;
  const int groups = static_cast<int>(cdiv(rows_of(s), NH));
  const int64_t ctas_y = static_cast<int64_t>(s.num_kv_heads) * groups;
  if (ctas_y > 65535) return PA_ERR_UNSUPPORTED;
  auto keys = [&](int64_t L) {
    return s.window > 0 ? std::min<int64_t>(L, static_cast<int64_t>(s.window) + s.max_new - 1) : L;
  };
  const int64_t max_n = keys(static_cast<int64_t>(s.max_pages_per_seq) * s.page_size);
  const int64_t max_tiles = max_n > 0 ? cdiv(max_n, TS) + (s.window > 0 ? 1 : 0) : 1;
  int64_t split_tiles = 0, per_max, max_splits;
  if (s.num_splits > 0) {
    max_splits = std::min<int64_t>(s.num_splits, max_tiles);
    per_max = cdiv(max_tiles, max_splits);
  } else {
    int64_t units = 0;
    if (lens) {
      for (int b = 0; b < batch; ++b) units += cdiv(keys(lens[b]), TS);
      units *= ctas_y;
    } else {
      units = static_cast<int64_t>(s.max_batch) * ctas_y * max_tiles;
    }
    const int64_t slots = static_cast<int64_t>(num_sms) * 3;
    split_tiles = std::max<int64_t>(8, cdiv(units, slots * 4));
    split_tiles = std::min<int64_t>(split_tiles, max_tiles);
    max_splits = cdiv(max_tiles, split_tiles);
    per_max = split_tiles;
  }
  // the last split of a (request, kv head, row group) merges, counted in the header: more of them than
  // counters go unsplit
  if (max_splits > 1 && s.max_batch * ctas_y > kMergeCounters) {
    if (s.num_splits > 0) return PA_ERR_UNSUPPORTED;
    max_splits = 1;
    split_tiles = per_max = max_tiles;
  }
  const int64_t bt_cache = cdiv(per_max * TS, s.page_size) + 2;
  if (bt_cache > 8192 || smem_bytes(s.head_dim, static_cast<int>(bt_cache)) > kMaxSmem) return PA_ERR_UNSUPPORTED;
  out->chunked = 0;
  out->tile_tokens = TS;
  out->split_tiles = static_cast<int32_t>(split_tiles);
  out->max_splits = static_cast<int32_t>(max_splits);
  out->row_groups = groups;
  out->bt_cache = static_cast<int32_t>(bt_cache);
  out->smem_bytes = smem_bytes(s.head_dim, out->bt_cache);
  out->scratch_bytes = split_scratch(s, max_splits);
  return PA_OK;
}

pa_status plan_chunks(const pa_block_shape& s, pa_block_plan_t* out) {
  const pa_shape e = as_shape(s, PA_MODE_EXTEND);
  if (extend_work_capacity(e) * s.num_kv_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;
  const int64_t one = std::max<int64_t>(2 * copy_bytes_a_request(s), 1);
  const int64_t group = std::max<int64_t>(1, std::min<int64_t>(std::max(s.max_batch, 1), kMaxCopyBytes / one));
  if (group * s.max_pages_per_seq > INT32_MAX) return PA_ERR_UNSUPPORTED;
  out->chunked = 1;
  out->group_requests = static_cast<int32_t>(group);
  out->max_splits = 1;
  out->tile_tokens = 64;
  out->scratch_bytes = chunk_scratch(s, group).end;
  return PA_OK;
}

template <int D>
cudaError_t launch_rows(bool i8, int nh8, const CUtensorMap& tmk, const CUtensorMap& tmv, const BlockParams& p,
                        dim3 grid, int smem, cudaStream_t st) {
  if (i8)
    return nh8 == 1 ? launch_split<D, true, 1>(tmk, tmv, p, grid, smem, st)
                    : launch_split<D, true, 2>(tmk, tmv, p, grid, smem, st);
  return nh8 == 1 ? launch_split<D, false, 1>(tmk, tmv, p, grid, smem, st)
                  : launch_split<D, false, 2>(tmk, tmv, p, grid, smem, st);
}

template <int D>
void launch_copy(bool i8, const CopyParams& p, dim3 grid, cudaStream_t st) {
  if (i8) {
    block_copy_kernel<D, true><<<grid, 256, 0, st>>>(p);
  } else {
    block_copy_kernel<D, false><<<grid, 256, 0, st>>>(p);
  }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_block_plan(const pa_block_shape* shape, const int32_t* host_seq_lens, int32_t batch,
                                   pa_block_plan_t* plan) {
  if (!shape || !plan) return PA_ERR_INVALID_ARG;
  pa_status st = validate(*shape);
  if (st != PA_OK) return st;
  if (host_seq_lens) {
    if (batch < 0 || batch > shape->max_batch) return PA_ERR_INVALID_ARG;
    const int64_t cap = static_cast<int64_t>(shape->max_pages_per_seq) * shape->page_size;
    for (int b = 0; b < batch; ++b)
      if (host_seq_lens[b] < 0 || host_seq_lens[b] > cap) return PA_ERR_INVALID_ARG;
  }
  int num_sms = shape->num_sms;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || num_sms <= 0)
      return PA_ERR_CUDA;
  }
  pa_block_plan_t p;
  std::memset(&p, 0, sizeof p);
  p.shape = *shape;
  p.shape.num_sms = num_sms;
  st = rows_of(*shape) <= kSplitRows ? plan_split(*shape, host_seq_lens, batch, num_sms, &p)
                                     : plan_chunks(*shape, &p);
  if (st != PA_OK) return st;
  *plan = p;
  return PA_OK;
}

extern "C" pa_status pa_block_attend(
    const pa_block_plan_t* plan, const void* q, int64_t q_stride_tok, int64_t q_stride_head, const void* k_cache,
    const void* v_cache, int64_t kv_stride_page, int64_t kv_stride_tok, int64_t kv_stride_head, int32_t num_pages,
    const float* k_scales, const float* v_scales, int64_t scale_stride, const int32_t* block_table, int64_t bt_stride,
    const int32_t* seq_lens, const int32_t* query_start_loc, int32_t batch, int32_t total_q, float scale,
    const float* sinks, void* out, int64_t out_stride_tok, int64_t out_stride_head, float* lse, void* scratch,
    int64_t scratch_bytes, void* stream) {
  if (!plan || validate(plan->shape) != PA_OK) return PA_ERR_INVALID_ARG;
  const pa_block_shape& s = plan->shape;
  if (batch < 0 || batch > s.max_batch || total_q < 0 || total_q > s.max_total_q) return PA_ERR_INVALID_ARG;
  if (!query_start_loc && total_q != batch) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  if ((sinks != nullptr) != (s.has_sinks != 0)) return PA_ERR_INVALID_ARG;
  if (!scratch) return PA_ERR_INVALID_ARG;
  if (scratch_bytes < plan->scratch_bytes || scratch_bytes < kScratchHeaderBytes) return PA_ERR_SCRATCH_TOO_SMALL;
  if (!aligned(scratch, 256)) return PA_ERR_UNSUPPORTED;
  // a plan edited by hand must match what its shape lays out
  const bool chunked = plan->chunked != 0;
  if (chunked != (rows_of(s) > kSplitRows)) return PA_ERR_INVALID_ARG;
  const int NH = nh8_of(s) * 8;
  const int groups = static_cast<int>(cdiv(rows_of(s), NH));
  if (chunked) {
    if (plan->group_requests < 1 ||
        static_cast<int64_t>(plan->group_requests) * s.max_pages_per_seq > INT32_MAX ||
        plan->scratch_bytes < chunk_scratch(s, plan->group_requests).end)
      return PA_ERR_INVALID_ARG;
    if (!query_start_loc && batch > 0) return PA_ERR_INVALID_ARG;      // (one row a request: a plan of max_new 1)
  } else {
    if (plan->max_splits < 1 || plan->split_tiles < 0 || (plan->split_tiles == 0 && s.num_splits == 0) ||
        plan->bt_cache < 1 || plan->bt_cache > 8192 || plan->row_groups != groups ||
        plan->tile_tokens != tile_of(s.head_dim) || plan->smem_bytes != smem_bytes(s.head_dim, plan->bt_cache) ||
        plan->smem_bytes > kMaxSmem || plan->scratch_bytes < split_scratch(s, plan->max_splits) ||
        (plan->max_splits > 1 &&
         static_cast<int64_t>(s.max_batch) * s.num_kv_heads * groups > kMergeCounters))
      return PA_ERR_INVALID_ARG;
  }
  if (batch == 0 || total_q == 0) return PA_OK;
  if (!q || !out || !k_scales || !v_scales || !block_table || !seq_lens || bt_stride < 0 || scale_stride < 0)
    return PA_ERR_INVALID_ARG;
  if (scale_stride < s.num_kv_heads && num_pages > 1) return PA_ERR_INVALID_ARG;
  if (q_stride_tok <= 0 || q_stride_head <= 0 || out_stride_tok <= 0 || out_stride_head <= 0)
    return PA_ERR_INVALID_ARG;
  // few rows: bf16 pairs; chunks: q feeds a TMA tensor map, out is written 16 bytes at a time
  const uintptr_t row_bytes = chunked ? 16 : 4;
  const int64_t row_elems = static_cast<int64_t>(row_bytes) / 2;
  if (!aligned(q, row_bytes) || !aligned(out, row_bytes) || q_stride_tok % row_elems || q_stride_head % row_elems ||
      out_stride_tok % row_elems || out_stride_head % row_elems)
    return PA_ERR_UNSUPPORTED;
  if ((lse && !aligned(lse, 4)) || !aligned(k_scales, 4) || !aligned(v_scales, 4) || (sinks && !aligned(sinks, 4)) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || (query_start_loc && !aligned(query_start_loc, 4)))
    return PA_ERR_UNSUPPORTED;
  pa_shape kv = as_shape(s, PA_MODE_EXTEND);
  kv.kv_dtype = PA_KV_FP8_E4M3;                       // (one byte an element)
  pa_status st = check_kv(kv, k_cache, v_cache, kv_stride_page, kv_stride_tok, kv_stride_head, num_pages);
  if (st != PA_OK) return st;
  const bool i8 = s.code == PA_CODE_INT8;
  uint8_t* sc = static_cast<uint8_t*>(scratch);
  cudaStream_t strm = static_cast<cudaStream_t>(stream);

  if (!chunked) {
    const int box_rows = std::min(s.page_size, plan->tile_tokens);
    CUtensorMap tmk, tmv;
    if ((st = make_kv_map(&tmk, k_cache, true, s.head_dim, s.num_kv_heads, s.page_size, num_pages, kv_stride_page,
                          kv_stride_tok, kv_stride_head, box_rows)) != PA_OK)
      return st;
    if ((st = make_kv_map(&tmv, v_cache, true, s.head_dim, s.num_kv_heads, s.page_size, num_pages, kv_stride_page,
                          kv_stride_tok, kv_stride_head, box_rows)) != PA_OK)
      return st;
    BlockParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride_tok = q_stride_tok;
    p.q_stride_head = q_stride_head;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.scale_stride = scale_stride;
    p.block_table = block_table;
    p.bt_stride = bt_stride;
    p.seq_lens = seq_lens;
    p.qsl = query_start_loc;
    p.batch = batch;
    p.total_q = total_q;
    p.max_new = s.max_new;
    p.max_kv = s.max_pages_per_seq * s.page_size;
    p.num_q_heads = s.num_q_heads;
    p.num_kv_heads = s.num_kv_heads;
    p.group = s.num_q_heads / s.num_kv_heads;
    p.page_size = s.page_size;
    p.num_pages = num_pages;
    p.scale_log2 = scale * kLog2e;
    p.cap_log2 = s.soft_cap > 0.f ? s.soft_cap * kLog2e : 0.f;
    p.scale_over_cap = s.soft_cap > 0.f ? scale / s.soft_cap : 0.f;
    p.window = s.window;
    p.sinks = sinks;
    p.out = static_cast<uint16_t*>(out);
    p.out_stride_tok = out_stride_tok;
    p.out_stride_head = out_stride_head;
    p.lse = lse;
    const int64_t rows = plan->max_splits > 1 ? partial_rows(s, plan->max_splits) : 0;
    p.o_part = reinterpret_cast<float*>(sc + kScratchHeaderBytes);
    p.lse_part = reinterpret_cast<float*>(sc + kScratchHeaderBytes + align_up(rows * s.head_dim * 4, 256));
    p.max_splits = plan->max_splits;
    p.split_tiles = plan->split_tiles;
    p.fixed_splits = s.num_splits > 0 ? plan->max_splits : 0;
    p.bt_cache = plan->bt_cache;
    p.row_groups = groups;
    p.merge_cnt = reinterpret_cast<uint32_t*>(sc + kMergeCounterOffset);
    p.err = reinterpret_cast<uint32_t*>(sc);
    const dim3 grid(plan->max_splits, s.num_kv_heads * groups, batch);
    cudaError_t e;
    switch (s.head_dim) {
      case 64: e = launch_rows<64>(i8, NH / 8, tmk, tmv, p, grid, plan->smem_bytes, strm); break;
      case 128: e = launch_rows<128>(i8, NH / 8, tmk, tmv, p, grid, plan->smem_bytes, strm); break;
      default: e = launch_rows<256>(i8, NH / 8, tmk, tmv, p, grid, plan->smem_bytes, strm); break;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }

  CUtensorMap tmq;
  if ((st = extend_q_map(&tmq, as_shape(s, PA_MODE_EXTEND), q, q_stride_tok, q_stride_head, total_q)) != PA_OK)
    return st;
  const ChunkScratch at = chunk_scratch(s, plan->group_requests);
  const int64_t maxp = s.max_pages_per_seq;
  CopyParams cp{};
  cp.k = static_cast<const uint8_t*>(k_cache);
  cp.v = static_cast<const uint8_t*>(v_cache);
  cp.stride_page = kv_stride_page;
  cp.stride_tok = kv_stride_tok;
  cp.stride_head = kv_stride_head;
  cp.k_scales = k_scales;
  cp.v_scales = v_scales;
  cp.scale_stride = scale_stride;
  cp.bt_stride = bt_stride;
  cp.num_pages = num_pages;
  cp.page_size = s.page_size;
  cp.num_kv_heads = s.num_kv_heads;
  cp.window = s.window;
  cp.maxp = static_cast<int>(maxp);
  cp.max_kv = s.max_pages_per_seq * s.page_size;
  cp.total_q = total_q;
  cp.kc = reinterpret_cast<uint16_t*>(sc + at.k);
  cp.vc = reinterpret_cast<uint16_t*>(sc + at.v);
  cp.page_scales = reinterpret_cast<float2*>(sc + at.scales);
  cp.bt_copy = reinterpret_cast<int32_t*>(sc + at.table);
  cp.err = reinterpret_cast<uint32_t*>(sc);
  for (int b0 = 0; b0 < batch; b0 += plan->group_requests) {
    const int n = std::min(plan->group_requests, batch - b0);
    cp.block_table = block_table + b0 * bt_stride;
    cp.seq_lens = seq_lens + b0;
    cp.qsl = query_start_loc + b0;
    const dim3 cgrid(static_cast<unsigned>(maxp), static_cast<unsigned>(n));
    if (maxp > 0) {
      switch (s.head_dim) {
        case 64: launch_copy<64>(i8, cp, cgrid, strm); break;
        case 128: launch_copy<128>(i8, cp, cgrid, strm); break;
        default: launch_copy<256>(i8, cp, cgrid, strm); break;
      }
      if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    }
    st = extend_over_copy(as_shape(s, PA_MODE_EXTEND), tmq, cp.kc, cp.vc, cp.page_scales, static_cast<int32_t>(n * maxp), cp.bt_copy, cp.seq_lens, cp.qsl, n, total_q, scale, sinks,
                          out, out_stride_tok, out_stride_head, lse, sc, sc + at.work, stream);
    if (st != PA_OK) return st;
  }
  return PA_OK;
}
