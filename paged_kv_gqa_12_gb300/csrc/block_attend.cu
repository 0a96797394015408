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
// denominator's 1 / vs in its own, in units that keep a long row of tiny scales
// finite.  m bounds every term of the output, so p <= 2^14
// whatever the pages' scales are, and a weight in f16 is off by half a step,
// 2^-11, down to 2^-28 of the row's largest.  q enters in f16 as well, scaled by a
// power of two a row (largest value in [2^14, 2^15): exact to 2^-32 of it).
//
// The codes are read once from HBM, which bounds the kernel; a code's way to
// f16 takes 0.75 (e4m3) or 1.25 (int8) instructions, where bf16(code * scale) takes 2.5.
// One wave of CTAs shares all tiles (of a request, a group of HG kv heads and of up to 8 or 16
// rows) evenly: a prefix sum over the requests gives each CTA its run of tiles, which
// may end one request and begin the next.  W compute warps are HG heads x KW groups
// of 16 keys of a tile; one more warp fetches a tile's codes, one TMA box for a page's
// slots of all HG heads, a ring of stages ahead and across requests.  Rows
// whose tiles lie in several shares are merged by a second kernel; what a share costs
// once (prefix sum, q, parts) is why there is one wave.  (Every warp with a
// ring and tiles of its own, equal splits of each request: 119 us for 64 requests of
// up to 8192 tokens, 59 for one of 131071.)
//
// S^T = K Q^T and O^T += V^T P^T keep the rows in the products' 8-wide dimension.
// ldmatrix brings four codes of a key (K), or two codes of two neighbouring keys (V,
// transposed), into a register; which dims those are is a fixed permutation that the
// q fragments and the output follow.  A page's scales wait in the lanes of the warp
// that needs them, 32 pages at a time.
//
// Measured (one GB300, CUDA-graph replay, 32 q and 8 kv heads of 128, pages of 16): 64
// requests of 512 to 8191 tokens int8 99.9 us, 5.7 TB/s; one of 131071 e4m3 54 us, eight
// of them 325 us, 6.6 TB/s (97 % of the copy bandwidth); of each call about 15 us are
// prefix sum and first loads (5 us), uneven shares (5) and the merge (5).  Up to four
// rows a request (16 a kv head) 114 us: 168 registers leave 8 compute warps an SM, whose
// dependent instructions are not hidden (two groups of 16 keys a warp at a time hide some).
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
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kWeightBias = 14.f;           // weights are at most 2^14 (f16 holds 65504)
constexpr float kLeastScale = 0x1p-100f;      // V scales below count as this one: its log2 and inverse are finite

// Rows whose parts lie in several shares: part 0 at place 2 share + 1, part i at place 2 (share + i).
struct MergeRecord {
  int n;                      // parts; 0: no record
  int share;
  int qs, kvh0, row0, rows, pad[2];
};
static_assert(sizeof(MergeRecord) == 32, "two 16-byte loads a record");

struct BlockParams {
  const uint16_t* q;
  int64_t q_stride_tok, q_stride_head;
  const float* k_scales;
  const float* v_scales;
  int64_t scale_stride;
  const uint8_t* v;           // the V codes and their strides (read here for NaN alone)
  int64_t v_stride_page, v_stride_tok, v_stride_head;
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
  float* o_part;              // [2 grid][HG][HW][D] normalised parts of rows
  float* lse_part;            // [2 grid][HG][HW] their LSEs, log2
  MergeRecord* records;       // [grid] the (request, heads, rows) that begins in a CTA's share and ends beyond, if any
  int min_tiles;              // fewest tiles a CTA is given
  int hg_log2;                // kv heads a CTA takes: 2^hg_log2
  uint32_t* err;
};

// Compute warps a CTA, stages of its ring, CTAs an SM, groups of 16 keys a warp and stage.  Measured with one group
// (64 requests of 512 to 8191 tokens, e4m3, us): heads of 64, up to 8 rows (8, 4, 2) 60.6, (4, 5, 3) 64.1, (8, 3, 3)
// 74.4, (4, 6, 4) 85.0; of 128 (4, 3, 3) 99.3, (8, 3, 1) 105.8, (8, 2, 2) 109.6, (4, 4, 3: two fit) 123.7; of 256 (4,
// 2, 2) 179.3, (8, 2, 1) 181.8, (4, 3, 1) 195.6; up to 16 rows, one to four tokens each: heads of 64 (4, 4, 3) 67.7,
// (8, 4, 2) 77.0; of 128 (4, 3, 2) 120.8, (4, 2, 2) 139.4 ((4, 2, 3) spills 400 bytes: 236); of 256 (4, 4, 1) 271, (8,
// 2, 1: 168 registers, spills) 435.
// Two groups: one maximum, rescaling and wait for 32 keys, and the second group's products beside the first's softmax.
// Up to 16 rows, heads of 64 67.4 -> 66.0 ((4, 3, 2): 156 registers), of 128 120.2 -> 114 ((4, 2, 2): 168, and up to 140
// bytes spilled); 16 requests of 2 to 8 K tokens 47.8 -> 48.6 (a tile is longer).  Up to 8 rows as they were (heads of
// 128 99.1, one long request 54.4 for 54.2): one group.
template <int D, int NH8> struct Choice;
template <> struct Choice<64, 1> { static constexpr int W = 8, NS = 4, CPS = 2, MT = 1; };
template <> struct Choice<64, 2> { static constexpr int W = 4, NS = 3, CPS = 2, MT = 2; };
template <> struct Choice<128, 1> { static constexpr int W = 4, NS = 3, CPS = 3, MT = 1; };
template <> struct Choice<128, 2> { static constexpr int W = 4, NS = 2, CPS = 2, MT = 2; };
template <> struct Choice<256, 1> { static constexpr int W = 4, NS = 2, CPS = 2, MT = 1; };
template <> struct Choice<256, 2> { static constexpr int W = 4, NS = 4, CPS = 1, MT = 1; };

// How much of a CTA's share a tile takes, and a (group of heads, group of rows) begun.  A tile of more than 8 rows costs
// 1.4 to 1.5 times one of up to 8 (two products instead of one under the same conversions), with two groups 1.25
// times (64 requests of 4 to 16 rows, us: 4 122, 5 114, 6 116); a beginning about a tile and a half (q, scales, parts).
constexpr int kTileWeight = 4, kStartWeight = 6;
constexpr int wide_weight(int groups) { return groups > 1 ? 5 : 6; }

template <int D, int NH8, int W, int NS, int MT>
struct Traits {
  static constexpr int RB = D < 128 ? D : 128;      // bytes per TMA box row
  static constexpr int NCC = D / RB;                // column chunks per key row
  static constexpr int TILE = W * MT * 16 * D;      // K (or V) bytes per stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int KS = D / 16;                 // 16-code units per row
  static constexpr int HW = NH8 * 8;
  static constexpr int WIDE = wide_weight(MT);      // units of a tile of more than 8 rows
  static constexpr int THREADS = (W + 1) * 32;
  static constexpr int STATES = W * (8 * D + 2 * HW) * 4;
  static constexpr int SMEM = 1024 + NS * STAGE + STATES + 2 * NS * 8;
  static_assert(RB == 128 || RB == 64, "row bytes must use the 128B or 64B swizzle");

  // Byte offset of 16-byte unit `u` of a warp's key row `row` (0 .. 15) as TMA writes it; column
  // chunks lie TILE / NCC apart.
  __device__ static __forceinline__ uint32_t unit(int row, int u) {
    constexpr int UPB = RB / 16;
    const uint32_t sw = (RB == 128) ? (row & 7) : ((row >> 1) & 3);
    return static_cast<uint32_t>((u / UPB) * (TILE / NCC) + row * RB) + (((u % UPB) ^ sw) << 4);
  }
};

// What a request brings: its rows, the tiles of TS keys they attend to, its (group of heads, group of rows) pairs y.
struct Request {
  int L, qs, n_new;
  int lo, tile0, n_tiles;
  int ys;                // groups of heads x groups of rows
  int weight;            // of a tile in a CTA's share
  __device__ __forceinline__ int units() const { return n_tiles > 0 ? n_tiles * weight + kStartWeight : 0; }   // a y
  // the first tile of a y that begins at or behind position `at` of its units: a tile belongs to the share that
  // holds its last unit, and what a y costs once comes with its first
  __device__ __forceinline__ int tile_at(int at) const { return max(0, at - kStartWeight) / weight; }
};

// (false: a length or packing beyond the plan)
template <class T>
__device__ __forceinline__ bool load_request(const BlockParams& p, int b, int ts, int hgroups, Request& r) {
  constexpr int hw = T::HW;
  r.L = p.seq_lens[b];
  r.qs = p.qsl != nullptr ? p.qsl[b] : b;
  r.n_new = p.qsl != nullptr ? packed_rows(r.qs, p.qsl[b + 1]) : 1;
  r.lo = r.tile0 = r.n_tiles = r.ys = 0;
  r.weight = hw > 8 && r.n_new * p.group > 8 ? T::WIDE : kTileWeight;
  if (r.n_new == 0) return true;
  if (r.n_new < 0 || r.n_new > p.max_new || r.qs < 0 || static_cast<int64_t>(r.qs) + r.n_new > p.total_q || r.L < 0 ||
      r.L > p.max_kv || (p.qsl != nullptr && r.L < r.n_new)) {
    r.n_new = 0;
    return false;
  }
  if (r.L == 0) return true;
  r.lo = p.window > 0 ? max(0, r.L - r.n_new - p.window + 1) : 0;
  r.tile0 = r.lo / ts;
  r.n_tiles = (r.L + ts - 1) / ts - r.tile0;
  r.ys = hgroups * ((r.n_new * p.group + hw - 1) / hw);
  return true;
}

__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(addr) : "memory");
  return w;
}
__device__ __forceinline__ void st_shared(uint32_t addr, const uint4& w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}

// All W compute warps of the CTA (the fetching warp does not take part).
template <int W>
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
}

// A finished row: where it goes, and the factor of its values (the sink, if any, joins the denominator);
// `lead` writes its LSE.
__device__ __forceinline__ uint16_t* finish_row(const BlockParams& p, int qs, int kvh, int row, float lse2, bool lead,
                                                float& factor) {
  const int tq = row / p.group;
  const int hq = kvh * p.group + (row - tq * p.group);
  const int64_t orow = qs + tq;
  factor = 1.f;
  if (p.sinks != nullptr) {
    const float sk = p.sinks[hq] * kLog2e;
    const float top = fmaxf(lse2, sk);
    const float own = ex2(lse2 - top), z = own + ex2(sk - top);
    factor = own / z;
    lse2 = top + lg2(z);
  }
  if (lead && p.lse != nullptr) p.lse[orow * p.num_q_heads + hq] = lse2 * kLn2;
  return p.out + orow * p.out_stride_tok + static_cast<int64_t>(hq) * p.out_stride_head;
}

template <int D, bool I8, int NH8, int W, int NS, int MT, bool CAP>
__global__ void __launch_bounds__((W + 1) * 32, (Choice<D, NH8>::CPS))
block_split_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const BlockParams p) {
  using T = Traits<D, NH8, W, NS, MT>;
  const int HG = 1 << p.hg_log2;
  const int KW = W >> p.hg_log2;                         // groups of 16 keys a stage
  const int TS = 16 * MT * KW;
  const int hgroups = p.num_kv_heads >> p.hg_log2;
  const int G = p.group;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int cta = blockIdx.x;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* states = reinterpret_cast<float*>(smem + NS * T::STAGE);   // [W][8][D], then [W][HW] maxima and sums
  float* wm = states + W * 8 * D;
  float* wl = wm + W * T::HW;
  uint64_t* full = reinterpret_cast<uint64_t*>(wl + W * T::HW);
  uint64_t* empty = full + NS;
  __shared__ int s_sum[W + 1];
  __shared__ int s_first, s_at;

  if (tid == W * 32) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], W);
    }
    fence_mbar_init();
  }

  if (tid == 0) p.records[cta].n = 0;
  // ---- this CTA's share of all requests' units --------------------------------
  const int per = (p.batch + T::THREADS - 1) / T::THREADS;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  int mine = 0;                                          // (the plan keeps all sums below 2^31)
  for (int b = b0; b < b1; ++b) {
    Request r;
    if (!load_request<T>(p, b, TS, hgroups, r) && cta == 0) atomicOr(p.err, kErrCapacity);
    mine += r.units() * r.ys;
  }
  // (decode of an empty request: no key, O = 0 and the LSE the sink's or -inf)
  if (p.qsl == nullptr)
    for (int b = cta; b < p.batch; b += gridDim.x) {
      if (p.seq_lens[b] != 0) continue;
      for (int i = tid; i < p.num_q_heads * (D / 2); i += T::THREADS) {
        const int hq = i / (D / 2), d = 2 * (i - hq * (D / 2));
        *reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(b) * p.out_stride_tok +
                                     static_cast<int64_t>(hq) * p.out_stride_head + d) = 0u;
        if (d == 0 && p.lse != nullptr)
          p.lse[static_cast<int64_t>(b) * p.num_q_heads + hq] = p.sinks != nullptr ? p.sinks[hq] : -INFINITY;
      }
    }
  int incl = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w <= W; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  // shares of at least min_tiles tiles (and a wide one: a share between two others of a y then holds a tile of
  // it): the first `more` of one unit more than the others
  const int least = max(p.min_tiles * kTileWeight, T::WIDE);
  const int C = min(static_cast<int>(gridDim.x), max(total > 0 ? 1 : 0, total / least));
  pdl_launch_dependents();             // (the merge kernel waits for this grid's end)
  if (cta >= C) return;
  const int share = total / C, more = total - share * C;
  const int begin = share * cta + min(cta, more);
  auto share_of = [&](int u) {
    const int m = more * (share + 1);
    return u < m ? u / (share + 1) : more + (u - m) / share;
  };
  const int end = begin + share + (cta < more ? 1 : 0);
  if (before <= begin && begin < before + mine) {
    int u = before;
    int b = b0;
    for (;; ++b) {
      Request r;
      load_request<T>(p, b, TS, hgroups, r);
      const int n = r.units() * r.ys;
      if (begin < u + n) break;
      u += n;
    }
    s_first = b;
    s_at = u;
  }
  __syncthreads();
  // place of the walk over the share: request and y, whose units begin at `pair0`; both the fetching warp and the
  // compute warps walk it, the former a ring ahead
  int b = s_first;
  Request r;
  load_request<T>(p, b, TS, hgroups, r);
  int y = (begin - s_at) / r.units();
  int pair0 = s_at + y * r.units();
  // its tiles that belong to this share
  auto tile_begin_of = [&]() { return r.tile_at(begin - pair0); };
  auto tile_end_of = [&]() { return min(r.n_tiles, r.tile_at(end - pair0)); };
  auto advance = [&]() {                 // to the next y; whether it begins in this share
    pair0 += r.units();
    if (pair0 >= end) return false;
    if (++y < r.ys) return true;
    y = 0;
    do {
      ++b;
      load_request<T>(p, b, TS, hgroups, r);
    } while (r.n_tiles == 0);            // (units are left, so a request with some follows)
    return true;
  };
  const int ps = p.page_size;
  const int ps_log2 = __ffs(ps) - 1;
  // the TMA coordinate of a page (-> `i`): an id outside the pool, or no attended page, becomes num_pages, whose
  // box reads as zeros
  auto page_coord = [&](int i, int tok_lo, int tok_hi, bool flag) {
    if ((i << ps_log2) >= tok_hi) return p.num_pages;
    const int id = p.block_table[static_cast<int64_t>(b) * p.bt_stride + i];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages)) return id;
    if (flag && ((i + 1) << ps_log2) > tok_lo) atomicOr(p.err, kErrPageId);
    return p.num_pages;
  };
  const int br = ps < TS ? ps : TS;      // slots a box

  if (warp == W) {
    // ---- the fetching warp: a stage's boxes lie one after the other, [head][slot] rows each ----
    const int box = br * T::RB << p.hg_log2;
    int it = 0;
    do {
      const int tile = tile_begin_of(), n = tile_end_of() - tile;
      if (n <= 0) continue;
      const int kvh0 = (y % hgroups) << p.hg_log2;
      const int tile_begin = r.tile0 + tile;
      const int tok_lo = max(r.lo, tile_begin * TS), tok_hi = min(r.L, (tile_begin + n) * TS);
      const int pg0 = (tile_begin * TS) >> ps_log2;
      int base = pg0;                    // lane i holds page base + i
      int coord = page_coord(base + lane, tok_lo, tok_hi, true);
      for (int k = 0; k < n; ++k, ++it) {
        const int stage = it % NS;
        if (it >= NS && !__all_sync(0xffffffffu, mbar_wait(&empty[stage], ((it / NS) - 1) & 1, p.err))) return;
        const int t0 = (tile_begin + k) * TS;
        int nb = 0;                      // boxes with a key of the sequence
        for (int j = 0; j < TS / br; ++j) nb += (t0 + j * br < r.L) ? 1 : 0;
        uint8_t* kst = smem + stage * T::STAGE;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(nb * (br << p.hg_log2) * D * 2));
        __syncwarp();
        for (int j = 0; j < nb; ++j) {
          const int t = t0 + j * br;
          const int i = t >> ps_log2;
          if (i - base >= 32) {
            base += 32;
            coord = page_coord(base + lane, tok_lo, tok_hi, true);
          }
          const int page = __shfl_sync(0xffffffffu, coord, i - base);
          if (lane == 0) {
#pragma unroll
            for (int cc = 0; cc < T::NCC; ++cc) {
              uint8_t* dst = kst + cc * (T::TILE / T::NCC) + j * box;
              tma_load_4d(dst, &tmk, cc * T::RB, t & (ps - 1), kvh0, page, &full[stage]);
              tma_load_4d(dst + T::TILE, &tmv, cc * T::RB, t & (ps - 1), kvh0, page, &full[stage]);
            }
          }
        }
      }
    } while (advance());
    return;
  }

  // ---- the compute warps -----------------------------------------------------------
  const int g = lane >> 2;
  const int c = lane & 3;
  const int hw = warp & (HG - 1);                        // head of the group
  const int kw = warp >> p.hg_log2;                      // MT 16-key groups of a stage
  const int mi = lane >> 3, mr = lane & 7;
  const int row = mr + ((mi & 1) << 3);
  // where this warp's groups of 16 rows lie in a stage
  const int key0 = kw * MT * 16;
  uint32_t place_u[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int key = key0 + 16 * mt;
    place_u[mt] = smem_u32(smem) + (static_cast<uint32_t>(key / br) * (br << p.hg_log2) + hw * br + key % br) * T::RB;
  }
  bool dead = false;                                     // a wait ran out: no more results
  int it = 0;
  do {
    const int tile = tile_begin_of(), n = tile_end_of() - tile;
    if (n <= 0) continue;
    const int kvh0 = (y % hgroups) << p.hg_log2;
    const int kvh = kvh0 + hw;
    const int row0 = (y / hgroups) * T::HW;              // first (token, head) row
    const int R = min(r.n_new * G - row0, T::HW);
    const int tile_begin = r.tile0 + tile;
    const int tok_lo = max(r.lo, tile_begin * TS), tok_hi = min(r.L, (tile_begin + n) * TS);
    // scales of this head's pages: lane i holds those of page base + i, and the next 32 pages' are on their way;
    // a page wholly before the window adds nothing, whatever its scales hold by now
    auto scales_of = [&](int i, float& ks, float& vs) {
      const int id = page_coord(i, tok_lo, tok_hi, false);
      const bool in = id < p.num_pages && ((i + 1) << ps_log2) > tok_lo;
      const int64_t sa = static_cast<int64_t>(in ? id : 0) * p.scale_stride + kvh;
      ks = in ? p.k_scales[sa] : 0.f;
      vs = in ? p.v_scales[sa] : 0.f;
    };
    int base = (tile_begin * TS) >> ps_log2;
    float page_k, page_v, next_k, next_v;
    scales_of(base + lane, page_k, page_v);
    scales_of(base + 32 + lane, next_k, next_v);
    page_v = lg2(fmaxf(page_v, kLeastScale));

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
      const uint16_t* qh = p.q + static_cast<int64_t>(r.qs + tq) * p.q_stride_tok +
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
    float m_run[NH8][2], l_run[NH8][2];
    float o[T::KS][NH8][4];
#pragma unroll
    for (int j = 0; j < NH8; ++j) m_run[j][0] = m_run[j][1] = -INFINITY, l_run[j][0] = l_run[j][1] = 0.f;
#pragma unroll
    for (int i = 0; i < T::KS; ++i)
#pragma unroll
      for (int j = 0; j < NH8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;

    // keys [full_lo, full_hi) are seen by every row: other 16-key groups mask each element
    const int full_lo = max(tok_lo, p.window > 0 ? r.L - p.window : 0);
    const int full_hi = min(tok_hi, r.L - r.n_new + 1);
    // (a request that brings at most 8 rows beside others of up to 16: NJ = 1 leaves the second 8 out)
    const int pos0 = r.L - r.n_new;                     // position of the first row's token
    uint32_t nan_codes = 0;              // e4m3: NaN met in V of keys that only some rows see
    // masked keys have P = 0, but their codes may be stale, NaN in e4m3 (of int8 every code is finite): V of the former
    // is zeroed, in this warp's own rows.  Of keys that some rows see and others do not, NaN codes alone become zeros;
    // the rows that see them get their NaN after the last tile.  (A second form of the products, with masks, is code that
    // requests of up to 8 and of up to 16 rows alternate between: 250 such requests 127 us for 126, int8 157 for 141.)
    auto clean = [&](int stage, int t0) {
      int ln = lane;                       // (kept from the compiler, as t0 below)
      asm volatile("" : "+r"(ln));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int tok = t0 + 16 * mt + (ln & 15);
        const uint32_t rows = place_u[mt] + stage * T::STAGE + T::TILE;
        if (tok < tok_lo || tok >= tok_hi) {
#pragma unroll
          for (int u = 0; u < T::KS; u += 2) st_shared(rows + T::unit(ln & 15, u + (ln >> 4)), make_uint4(0, 0, 0, 0));
        } else if (tok < full_lo || tok >= full_hi) {
#pragma unroll 1
          for (int u = 0; u < T::KS; u += 2) {
            const uint32_t at = rows + T::unit(ln & 15, u + (ln >> 4));
            const uint4 w = ld_shared(at);
            const uint4 nan = make_uint4(e4m3_nan4(w.x), e4m3_nan4(w.y), e4m3_nan4(w.z), e4m3_nan4(w.w));
            const uint32_t any = nan.x | nan.y | nan.z | nan.w;
            if (any != 0) {
              st_shared(at, make_uint4(w.x & ~nan.x, w.y & ~nan.y, w.z & ~nan.z, w.w & ~nan.w));
              nan_codes |= any;
            }
          }
        }
      }
      fence_proxy_async_smem();            // (the stage's next codes come by TMA)
      __syncwarp();
    };
    auto tiles = [&](auto nj_tag, int k0, int k1) {
    constexpr int NJ = decltype(nj_tag)::value;
    for (int k = k0; k < k1; ++k, ++it) {
      const int stage = it % NS;
      // (kept from the compiler, or it holds every offset from it in a register of its own: 200 bytes spilled)
      int t0 = (tile_begin + k) * TS + key0;
      asm volatile("" : "+r"(t0));         // this warp's first key
      // (a tile's pages lie in one run of 32; a page beyond the sequence's last holds only masked keys, any
      // scale will do)
      if ((t0 >> ps_log2) - base >= 32) {
        base += 32;
        page_k = next_k;
        page_v = lg2(fmaxf(next_v, kLeastScale));
        scales_of(base + 32 + lane, next_k, next_v);
      }
      float ks[MT], lv[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int from = ((t0 + 16 * mt) >> ps_log2) - base;
        ks[mt] = __shfl_sync(0xffffffffu, page_k, from);
        lv[mt] = __shfl_sync(0xffffffffu, page_v, from);
      }
      dead = dead || !__all_sync(0xffffffffu, mbar_wait(&full[stage], (it / NS) & 1, p.err));
      if (dead) continue;
      const bool partial = (t0 < full_lo) || (t0 + 16 * MT > full_hi);

      // ---- S^T = K Q^T over the codes ----------------------------------------
      float s[MT][NJ][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
        const uint32_t kst_u = place_u[mt] + stage * T::STAGE;
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
            for (int j = 0; j < NJ; ++j) mma_f16(s[mt][j], a, qf[u + v][j][0], qf[u + v][j][1]);
          }
        }
      }

      // ---- scales, soft-cap, mask; online softmax (log2 domain) --------------
      float mx[NJ][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float f[2] = {ks[mt] * rsl[j][0], ks[mt] * rsl[j][1]};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (CAP) {
              s[mt][j][e] = fmaf(p.cap_log2, tanhf(s[mt][j][e] * f[e & 1]), lv[mt]);
            } else {
              s[mt][j][e] = fmaf(s[mt][j][e], f[e & 1], lv[mt]);
            }
          }
        }
      if (partial) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = t0 + 16 * mt + g + ((e >> 1) << 3);
              const int pos = pos0 + (row0 + min(j * 8 + 2 * c + (e & 1), R - 1)) / G;
              if (tok < tok_lo || tok >= tok_hi || tok > pos || (p.window > 0 && tok <= pos - p.window))
                s[mt][j][e] = -INFINITY;
            }
      }
      bool grew = false;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float m = fmaxf(s[0][j][h], s[0][j][h + 2]);
#pragma unroll
          for (int mt = 1; mt < MT; ++mt) m = fmaxf(m, fmaxf(s[mt][j][h], s[mt][j][h + 2]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          mx[j][h] = m;
          grew |= m > m_run[j][h];
        }
      // the accumulators need rescaling only after a maximum rose somewhere in the warp
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          float alpha[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float m_new = fmaxf(m_run[j][h], mx[j][h]);
            alpha[h] = m_new == -INFINITY ? 1.f : ex2(m_run[j][h] - m_new);
            m_run[j][h] = m_new;
            l_run[j][h] *= alpha[h];
          }
#pragma unroll
          for (int i = 0; i < T::KS; ++i) {
            o[i][j][0] *= alpha[0];
            o[i][j][1] *= alpha[1];
            o[i][j][2] *= alpha[0];
            o[i][j][3] *= alpha[1];
          }
        }
      }
      uint32_t pb[MT][NJ][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float iv = ex2(-lv[mt]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          float mu[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) mu[h] = m_run[j][h] == -INFINITY ? 0.f : m_run[j][h] - kWeightBias;
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][j][e] = ex2(s[mt][j][e] - mu[e & 1]);
          l_run[j][0] = fmaf((s[mt][j][0] + s[mt][j][2]) * kDenScale, iv, l_run[j][0]);
          l_run[j][1] = fmaf((s[mt][j][1] + s[mt][j][3]) * kDenScale, iv, l_run[j][1]);
          pb[mt][j][0] = movmatrix_t(pack_f16x2(s[mt][j][0], s[mt][j][1]));
          pb[mt][j][1] = movmatrix_t(pack_f16x2(s[mt][j][2], s[mt][j][3]));
        }
      }

      // ---- O^T += V^T P^T over the codes ---------------------------------------
      const uint32_t vst_u = stage * T::STAGE + T::TILE;
      if constexpr (!I8 && MT > 1) {
        if (partial) clean(stage, t0);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int u = 0; u < T::KS; u += 2) {
          uint32_t w[4];               // of unit u: keys 0-7, 8-15; then of unit u + 1
          ldsm_x4_t(w, place_u[mt] + vst_u + T::unit(row, u + (mi >> 1)));
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
#pragma unroll
            for (int j = 0; j < NJ; ++j) mma_f16(o[u + v][j], a, pb[mt][j][0], pb[mt][j][1]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
    }
    };
    // (a tile with masked keys by itself: with one group of keys a warp the loop over the others holds fewer registers
    // without that code, 64 requests of heads of 256 with one to four rows 249 us for 263, with four 314 for 334; with two
    // groups one loop is better, heads of 128 113 for 117.  Rows beyond 8 are left out around the whole walk: inside it
    // their accumulators stay in registers, 249 us become 314)
    auto walk = [&](auto nj_tag) {
      if constexpr (I8 || MT > 1) {
        tiles(nj_tag, 0, n);
      } else {
        for (int k = 0, k1; k < n; k = k1) {
          const int t0 = (tile_begin + k) * TS + key0;
          if (t0 < full_lo || t0 + 16 > full_hi) {
            dead = dead || !__all_sync(0xffffffffu, mbar_wait(&full[it % NS], (it / NS) & 1, p.err));
            if (!dead) clean(it % NS, t0);
            k1 = k + 1;
          } else {
            k1 = min(n, (full_hi - 16 - key0) / TS - tile_begin + 1);          // up to the next with masked keys
          }
          tiles(nj_tag, k, k1);
        }
      }
    };
    if (NH8 == 2 && R <= 8) {
      walk(std::integral_constant<int, 1>{});
    } else {
      walk(std::integral_constant<int, NH8>{});
    }

    if (MT > 1) load_request<T>(p, b, TS, hgroups, r);   // (again, rather than in registers over the tiles)

    if (!I8 && __any_sync(0xffffffffu, nan_codes != 0)) {
      const int lo = max(r.lo, (r.tile0 + tile) * TS), hi = min(r.L, (r.tile0 + tile + n) * TS);
      const int seen_lo = max(lo, p.window > 0 ? r.L - p.window : 0), seen_hi = min(hi, r.L - r.n_new + 1);
      for (int tok = lo; tok < hi; ++tok) {
        if (tok >= seen_lo && tok < seen_hi) tok = seen_hi;              // (these codes were left as they are)
        if (tok >= hi) break;
        const int id = p.block_table[static_cast<int64_t>(b) * p.bt_stride + (tok >> ps_log2)];
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) continue;
        const uint8_t* vp = p.v + static_cast<int64_t>(id) * p.v_stride_page + (tok & (ps - 1)) * p.v_stride_tok +
                            static_cast<int64_t>(kvh) * p.v_stride_head + 2 * g;
        bool sees[NH8][2];
#pragma unroll
        for (int j = 0; j < NH8; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pos = r.L - r.n_new + (row0 + min(j * 8 + 2 * c + h, R - 1)) / G;
            sees[j][h] = tok <= pos && (p.window <= 0 || tok > pos - p.window);
          }
#pragma unroll
        for (int i = 0; i < T::KS; ++i) {
          const uint32_t w = e4m3_nan4(*reinterpret_cast<const uint16_t*>(vp + 16 * i));     // dims 16 i + 2 g and the next
#pragma unroll
          for (int j = 0; j < NH8; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (sees[j][h] && (w & 0xffu) != 0) o[i][j][h] = __uint_as_float(0x7fffffffu);
              if (sees[j][h] && (w & 0xff00u) != 0) o[i][j][h + 2] = __uint_as_float(0x7fffffffu);
            }
        }
      }
    }

    // ---- the rows' values, merged over a head's KW warps -----------------------------
    // the shares that hold parts of this (request, y): first .. last; a part that begins it goes to place
    // 2 share + 1, any other to 2 share
    const int first = share_of(pair0 + kStartWeight + r.weight - 1), last = share_of(pair0 + r.units() - 1);
    const bool direct = first == last;
    const int place = 2 * cta + (tile == 0 ? 1 : 0);
    float lse2[NH8][2];
#pragma unroll
    for (int j = 0; j < NH8; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = l_run[j][h];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        l_run[j][h] = l;
      }
    if (KW > 1) {
      // the states of a head's KW warps meet in shared memory, 8 rows at a time; each warp then has the units
      // of 16 dims i with i % KW == kw
#pragma unroll
      for (int j = 0; j < NH8; ++j) {
        compute_sync<W>();                               // (earlier states are read)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rr = 2 * c + h;
          if (g == 0) {
            wm[warp * T::HW + j * 8 + rr] = m_run[j][h];
            wl[warp * T::HW + j * 8 + rr] = l_run[j][h];
          }
#pragma unroll
          for (int i = 0; i < T::KS; ++i)
            *reinterpret_cast<float2*>(states + (warp * 8 + rr) * D + 16 * i + 2 * g) =
                make_float2(o[i][j][h], o[i][j][h + 2]);
        }
        compute_sync<W>();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rr = 2 * c + h;
          float M = -INFINITY, den = 0.f;
          for (int w = 0; w < KW; ++w) M = fmaxf(M, wm[((w << p.hg_log2) + hw) * T::HW + j * 8 + rr]);
          const float m_use = M == -INFINITY ? 0.f : M;
          m_run[j][h] = M;
#pragma unroll
          for (int i = 0; i < T::KS; ++i)
            if ((i & (KW - 1)) == kw) o[i][j][h] = o[i][j][h + 2] = 0.f;
          for (int w = 0; w < KW; ++w) {
            const int sw = (w << p.hg_log2) + hw;
            const float f = ex2(wm[sw * T::HW + j * 8 + rr] - m_use);
            den = fmaf(wl[sw * T::HW + j * 8 + rr], f, den);
#pragma unroll
            for (int i = 0; i < T::KS; ++i) {
              if ((i & (KW - 1)) != kw) continue;
              const float2 x = *reinterpret_cast<const float2*>(states + (sw * 8 + rr) * D + 16 * i + 2 * g);
              o[i][j][h] = fmaf(x.x, f, o[i][j][h]);
              o[i][j][h + 2] = fmaf(x.y, f, o[i][j][h + 2]);
            }
          }
          l_run[j][h] = den;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NH8; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rr = j * 8 + 2 * c + h;
        if (rr >= R) continue;
        // l = 2^-20 sum 2^(x - m + 14) / vs: the row's LSE is m - 14 + 20 + log2 l
        const float den = l_run[j][h];
        lse2[j][h] = den == 0.f ? -INFINITY : m_run[j][h] - (kWeightBias - kDenBias) + lg2_den(den);
        float f = den == 0.f ? 0.f : kDenScale / den;
        const bool lead = g == 0 && kw == 0;
        if (direct) {
          float sink;
          uint16_t* outp = finish_row(p, r.qs, kvh, row0 + rr, lse2[j][h], lead, sink) + 2 * g;
          f *= sink;
#pragma unroll
          for (int i = 0; i < T::KS; ++i)
            if ((i & (KW - 1)) == kw)
              *reinterpret_cast<uint32_t*>(outp + 16 * i) = pack_bf16x2(o[i][j][h] * f, o[i][j][h + 2] * f);
        } else {
          const int64_t pa = (static_cast<int64_t>(place) * HG + hw) * T::HW + rr;
          if (lead) p.lse_part[pa] = lse2[j][h];
          float* part = p.o_part + pa * D + 2 * g;
#pragma unroll
          for (int i = 0; i < T::KS; ++i)
            if ((i & (KW - 1)) == kw)
              *reinterpret_cast<float2*>(part + 16 * i) = make_float2(o[i][j][h] * f, o[i][j][h + 2] * f);
        }
      }
    if (!direct && cta == first && tid == 0)
      p.records[cta] = MergeRecord{last - first + 1, first, r.qs, kvh0, row0, R, {0, 0}};
  } while (advance());
}

// ---- rows in several shares, merged by their LSEs ------------------------------------
// One warp a row where rows have at most 32 parts, else all warps of a CTA.  (The last CTA of a row's
// shares as the merging one took 8 to 16 us: a few warps, each waiting for L2 row after row, often
// with tiles of the next request to come.)
constexpr int kMergeThreads = 256;
// The parts' weights count 2^-13 of themselves in the sum of values: of up to kMaxCtas parts next to fp32's largest
// number it stays finite.
constexpr float kPartScale = 0x1p-13f;

// Parts [i0, i1) of a row: v = kPartScale sum 2^(lse - M) part, Z = sum 2^(lse - M); U parts' loads in flight together.
template <int D, int U>
__device__ __forceinline__ void merge_range(const BlockParams& p, const MergeRecord& rec, int row_in_place, int place_rows,
                                            int i0, int i1, int lane, float& M, float& Z, float4 (&v)[(D + 127) / 128]) {
  constexpr int K = (D + 127) / 128;
  M = -INFINITY;
  Z = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int d = (lane * 4) % D;
  auto row_of = [&](int i) {
    return static_cast<int64_t>(2 * (rec.share + i) + (i == 0 ? 1 : 0)) * place_rows + row_in_place;
  };
  for (int base = i0; base < i1; base += U) {
    const int n = min(U, i1 - base);
    float l = __ldcg(p.lse_part + row_of(base + min(lane, n - 1)));
    if (lane >= n) l = -INFINITY;
    float4 o[U];
    auto fetch = [&](int k) {
#pragma unroll
      for (int i = 0; i < U; ++i)        // (behind the last part the last again, with weight 0)
        o[i] = __ldcg(reinterpret_cast<const float4*>(p.o_part + row_of(base + min(i, n - 1)) * D + d + 128 * k));
    };
    fetch(0);
    float m = l;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    const float top = fmaxf(M, m);
    const float old = M == -INFINITY ? 0.f : ex2(M - top);
    float w = l == -INFINITY ? 0.f : ex2(l - top);   // (a part with no key for this row)
    float z = w;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    Z = fmaf(Z, old, z);
    M = top;
    w *= kPartScale;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k > 0) fetch(k);
      v[k].x *= old; v[k].y *= old; v[k].z *= old; v[k].w *= old;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float f = __shfl_sync(0xffffffffu, w, i);
        v[k].x = fmaf(f, o[i].x, v[k].x);
        v[k].y = fmaf(f, o[i].y, v[k].y);
        v[k].z = fmaf(f, o[i].z, v[k].z);
        v[k].w = fmaf(f, o[i].w, v[k].w);
      }
    }
  }
}

template <int D, int HW>
__global__ void __launch_bounds__(kMergeThreads) block_merge_kernel(const BlockParams p, int ctas) {
  constexpr int K = (D + 127) / 128;
  constexpr int WARPS = kMergeThreads / 32;
  extern __shared__ int s_off[];         // [ctas + 1] rows of the records before
  __shared__ int s_sum[WARPS], s_most[WARPS];
  __shared__ float s_v[WARPS][D];
  __shared__ float s_m[WARPS], s_z[WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = 1 << p.hg_log2;
  pdl_wait_primary();
  const int per = (ctas + kMergeThreads - 1) / kMergeThreads;
  const int c0 = min(tid * per, ctas), c1 = min(c0 + per, ctas);
  int mine = 0, most = 0;
  for (int i = c0; i < c1; ++i) {
    const int n = p.records[i].n;
    if (n > 0) mine += p.records[i].rows << p.hg_log2;
    most = max(most, n);
  }
  int incl = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += x;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) s_sum[warp] = incl;
  if (lane == 0) s_most[warp] = most;
  __syncthreads();
  int run = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) run += s_sum[w];
    total += s_sum[w];
    most = max(most, s_most[w]);
  }
  for (int i = c0; i < c1; ++i) {
    s_off[i] = run;
    if (p.records[i].n > 0) run += p.records[i].rows << p.hg_log2;
  }
  if (tid == 0) s_off[ctas] = total;
  __syncthreads();
  const bool alone = most <= 32;         // a warp a row
  const int step = alone ? gridDim.x * WARPS : gridDim.x;
  for (int item = alone ? blockIdx.x * WARPS + warp : blockIdx.x; item < total; item += step) {
    int lo = 0, hi = ctas;               // the last record that begins at or before the item
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_off[mid] <= item) lo = mid;
      else hi = mid;
    }
    const MergeRecord rec = p.records[lo];
    const int hr = item - s_off[lo];
    const int head = hr / rec.rows;
    const int rr = hr - head * rec.rows;
    const int i0 = alone ? 0 : rec.n * warp / WARPS, i1 = alone ? rec.n : rec.n * (warp + 1) / WARPS;
    float M, Z;
    float4 v[K];
    // (most rows of many requests have two to four parts)
    if (i1 - i0 <= 4) {
      merge_range<D, 4>(p, rec, head * HW + rr, heads * HW, i0, i1, lane, M, Z, v);
    } else {
      merge_range<D, 16>(p, rec, head * HW + rr, heads * HW, i0, i1, lane, M, Z, v);
    }
    if (!alone) {
      __syncthreads();                   // (an earlier row's values are read)
      if (lane == 0) {
        s_m[warp] = M;
        s_z[warp] = Z;
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (lane * 4 < D) *reinterpret_cast<float4*>(&s_v[warp][lane * 4 + 128 * k]) = v[k];
      __syncthreads();
      if (warp != 0) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_m[w]);
      M = top;
      Z = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - top);
        Z = fmaf(s_z[w], f, Z);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(&s_v[w][(lane * 4) % D + 128 * k]);
          v[k].x = fmaf(x.x, f, v[k].x);
          v[k].y = fmaf(x.y, f, v[k].y);
          v[k].z = fmaf(x.z, f, v[k].z);
          v[k].w = fmaf(x.w, f, v[k].w);
        }
      }
    }
    float f;
    uint16_t* outp = finish_row(p, rec.qs, rec.kvh0 + head, rec.row0 + rr, Z == 0.f ? -INFINITY : M + lg2(Z), lane == 0, f);
    f = Z == 0.f ? 0.f : f / (Z * kPartScale);
    if (lane * 4 < D) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        uint32_t* w32 = reinterpret_cast<uint32_t*>(outp + lane * 4 + 128 * k);            // (rows are 4-byte aligned)
        w32[0] = pack_bf16x2(v[k].x * f, v[k].y * f);
        w32[1] = pack_bf16x2(v[k].z * f, v[k].w * f);
      }
    }
  }
}

struct Variant {
  int warps, smem, ctas, groups;        // groups: of 16 keys a warp and stage
};

template <int D, int NH8>
Variant variant() {
  using C = Choice<D, NH8>;
  return {C::W, Traits<D, NH8, C::W, C::NS, C::MT>::SMEM, C::CPS, C::MT};
}

Variant variant_of(int D, int nh8) {
  if (D == 64) return nh8 == 1 ? variant<64, 1>() : variant<64, 2>();
  if (D == 128) return nh8 == 1 ? variant<128, 1>() : variant<128, 2>();
  return nh8 == 1 ? variant<256, 1>() : variant<256, 2>();
}

template <int D, bool I8, int NH8>
cudaError_t launch_split(const CUtensorMap& tmk, const CUtensorMap& tmv, const BlockParams& p, dim3 grid,
                         cudaStream_t stream) {
  using C = Choice<D, NH8>;
  using T = Traits<D, NH8, C::W, C::NS, C::MT>;
  auto kern = p.cap_log2 > 0.f ? block_split_kernel<D, I8, NH8, C::W, C::NS, C::MT, true>
                               : block_split_kernel<D, I8, NH8, C::W, C::NS, C::MT, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<grid, T::THREADS, T::SMEM, stream>>>(tmk, tmv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid.x == 1) return e;         // (one share holds every row whole)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(std::min(grid.x, 304u));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = (grid.x + 1) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_merge_kernel<D, NH8 * 8>, p, static_cast<int>(grid.x));
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
  int num_pages, page_size, num_kv_heads, window, maxp, max_kv, max_new, total_q;
  uint16_t* kc;
  uint16_t* vc;
  float2* page_scales;        // [copy page][Hkv]: K scale, log2 of the V scale
  int32_t* bt_copy;           // a request's copy pages; the sign bit is set where a V code is NaN
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

// V codes without NaN, which a product would carry from its key's rows to all of a tile: NaN becomes minus zero, and
// minus zero zero.  Whether there was one.
__device__ __forceinline__ bool mark_nan(uint4& w) {
  uint32_t any = 0;
  uint32_t* x[4] = {&w.x, &w.y, &w.z, &w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t nan = e4m3_nan4(*x[k]), zero = __vcmpeq4(*x[k], 0x80808080u);
    *x[k] = (*x[k] & ~(nan | zero)) | (nan & 0x80808080u);
    any |= nan;
  }
  return any != 0;
}

// One CTA a (page of a request, request).
template <int D, bool I8>
__global__ void __launch_bounds__(256) block_copy_kernel(const CopyParams p) {
  const int i = blockIdx.x;
  const int b = blockIdx.y;
  const int64_t dst_page = static_cast<int64_t>(b) * p.maxp + i;
  if (threadIdx.x == 0) p.bt_copy[dst_page] = static_cast<int32_t>(dst_page);   // (the same thread marks it below)
  const int L = p.seq_lens[b];
  const int qs = p.qsl[b];
  const int n = packed_rows(qs, p.qsl[b + 1]);
  const int ctx = L - n;
  if (n <= 0 || n > p.max_new || ctx < 0 || L > p.max_kv || qs < 0 || static_cast<int64_t>(qs) + n > p.total_q) return;
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
  bool nan = false;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    const int tok = u / (p.num_kv_heads * UPH);
    const int rem = u - tok * (p.num_kv_heads * UPH);
    const int head = rem / UPH;
    const int64_t off = static_cast<int64_t>(src) * p.stride_page + static_cast<int64_t>(tok) * p.stride_tok +
                        static_cast<int64_t>(head) * p.stride_head + (rem - head * UPH) * 16;
    widen_unit<I8, true>(*reinterpret_cast<const uint4*>(p.k + off), kd + 2 * u);
    uint4 w = *reinterpret_cast<const uint4*>(p.v + off);
    if constexpr (!I8) nan |= mark_nan(w) && i * ps + tok >= first && i * ps + tok < L;       // (of a key of the request)
    widen_unit<I8, false>(w, vd + 2 * u);
  }
  if constexpr (!I8) {
    nan = __syncthreads_or(nan);
    if (nan && threadIdx.x == 0) p.bt_copy[dst_page] = static_cast<int32_t>(dst_page) | INT32_MIN;
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

// kv heads a CTA takes, as a log2: a power of two that divides Hkv, at most its warps
int heads_log2(const pa_block_shape& s, int warps) {
  int l = 0;
  while ((2 << l) <= warps && s.num_kv_heads % (2 << l) == 0) ++l;
  return l;
}

// Above this many rows a kv head (of one request) the chunked form is taken.  It copies the codes and has no
// parts of a context, so it wants requests enough to fill the card (two CTAs an SM).  Measured, split / chunked, groups
// of 4, heads of 128, us, e4m3 and int8: 64 requests of up to 8192 tokens, 12 rows each (48 a kv head) 323 / 485 and
// 348 / 485, 16 rows 423 / 489 and 454 / 486, 20 rows 518 / 487 and 562 / 488; 4 such requests, 32 rows (128 a kv head)
// 68 / 143 and 75 / 137; one of 131071 tokens, 32 rows, int8 376 / 1973.  (Between 48 and 64 rows the split form is
// ahead at heads of 128; 64 and 256 were not measured there.)
// One row a request is never chunked, whatever its group: such a plan's calls may leave query_start_loc out, which
// the chunked form's kernels read.
bool chunked_form(const pa_block_shape& s) {
  if (s.max_new == 1) return false;
  const bool fills = static_cast<int64_t>(s.max_batch) * s.num_kv_heads >= 2 * static_cast<int64_t>(s.num_sms);
  return rows_of(s) > (fills ? 48 : 128);
}

constexpr int64_t kMaxCtas = 4096;

// Fewest keys of one head that a CTA of the split kernel is given (four requests of 60 to 1000 tokens: 11.6 us with 128,
// 12.3 with 256, 15.1 with 512).
constexpr int kLeastKeys = 128;

int64_t split_scratch(const pa_block_shape& s, int64_t ctas, int hg) {
  const int64_t rows = 2 * ctas * nh8_of(s) * 8 << hg;
  return kScratchHeaderBytes + align_up(rows * s.head_dim * 4, 256) + align_up(rows * 4, 256) +
         ctas * static_cast<int64_t>(sizeof(MergeRecord));
}

pa_status validate(const pa_block_shape& s) {
  if (s.code != PA_CODE_E4M3 && s.code != PA_CODE_INT8) return PA_ERR_INVALID_ARG;
  if (s.max_new < 1 || s.num_ctas < 0) return PA_ERR_INVALID_ARG;
  const pa_status st = validate_shape(as_shape(s, PA_MODE_EXTEND));
  if (st != PA_OK) return st;
  if (s.max_batch > 65535) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

pa_status plan_split(const pa_block_shape& s, const int32_t* lens, int32_t batch, int num_sms, pa_block_plan_t* out) {
  const Variant v = variant_of(s.head_dim, nh8_of(s));
  const int hg = heads_log2(s, v.warps);
  const int TS = 16 * v.groups * (v.warps >> hg);
  const int groups = static_cast<int>(cdiv(rows_of(s), nh8_of(s) * 8));
  const int64_t ctas_y = static_cast<int64_t>(s.num_kv_heads >> hg) * groups;
  const int64_t max_n = static_cast<int64_t>(s.max_pages_per_seq) * s.page_size;
  auto tiles = [&](int64_t L) {
    return cdiv(s.window > 0 ? std::min<int64_t>(L, static_cast<int64_t>(s.window) + s.max_new - 1) : L, TS) +
           (s.window > 0 ? 1 : 0);
  };
  int64_t units = 0;
  if (lens) {
    for (int b = 0; b < batch; ++b) units += tiles(lens[b]) * ctas_y;
  } else {
    units = s.max_batch * ctas_y * tiles(max_n);
  }
  // one wave, or fewer CTAs where the lengths (or capacities) give none of them its least share
  const int64_t least = std::max<int64_t>(1, kLeastKeys / (v.warps * v.groups * 16));
  const int64_t wave = std::min<int64_t>(s.num_ctas > 0 ? s.num_ctas : static_cast<int64_t>(num_sms) * v.ctas,
                                         kMaxCtas);
  // (the kernel counts weighted tiles in 32 bits)
  if (s.max_batch * ctas_y * (tiles(max_n) * wide_weight(v.groups) + kStartWeight) > INT32_MAX) return PA_ERR_UNSUPPORTED;
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(wave, cdiv(units, least)));
  out->chunked = 0;
  out->tile_tokens = TS;
  out->min_tiles = static_cast<int32_t>(least);
  out->ctas = static_cast<int32_t>(ctas);
  out->row_groups = groups;
  out->head_group = 1 << hg;
  out->smem_bytes = v.smem;
  out->scratch_bytes = split_scratch(s, ctas, hg);
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
  out->tile_tokens = 64;
  out->scratch_bytes = chunk_scratch(s, group).end;
  return PA_OK;
}

template <int D>
cudaError_t launch_rows(bool i8, int nh8, const CUtensorMap& tmk, const CUtensorMap& tmv, const BlockParams& p,
                        dim3 grid, cudaStream_t st) {
  if (i8)
    return nh8 == 1 ? launch_split<D, true, 1>(tmk, tmv, p, grid, st) : launch_split<D, true, 2>(tmk, tmv, p, grid, st);
  return nh8 == 1 ? launch_split<D, false, 1>(tmk, tmv, p, grid, st) : launch_split<D, false, 2>(tmk, tmv, p, grid, st);
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
  st = chunked_form(p.shape) ? plan_chunks(*shape, &p) : plan_split(*shape, host_seq_lens, batch, num_sms, &p);
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
  if (chunked != chunked_form(s)) return PA_ERR_INVALID_ARG;
  const int NH = nh8_of(s) * 8;
  const int groups = static_cast<int>(cdiv(rows_of(s), NH));
  const Variant v = variant_of(s.head_dim, NH / 8);
  const int hg = heads_log2(s, v.warps);
  if (chunked) {
    if (plan->group_requests < 1 ||
        static_cast<int64_t>(plan->group_requests) * s.max_pages_per_seq > INT32_MAX ||
        plan->scratch_bytes < chunk_scratch(s, plan->group_requests).end)
      return PA_ERR_INVALID_ARG;
    if (!query_start_loc && batch > 0) return PA_ERR_INVALID_ARG;
  } else {
    if (plan->ctas < 1 || plan->ctas > kMaxCtas || plan->min_tiles < 1 || plan->row_groups != groups ||
        plan->head_group != 1 << hg || plan->tile_tokens != 16 * v.groups * (v.warps >> hg) || plan->smem_bytes != v.smem ||
        plan->scratch_bytes < split_scratch(s, plan->ctas, hg))
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
    if ((st = make_codes_map(&tmk, k_cache, s.head_dim, s.num_kv_heads, s.page_size, num_pages, kv_stride_page,
                             kv_stride_tok, kv_stride_head, box_rows, 1 << hg)) != PA_OK)
      return st;
    if ((st = make_codes_map(&tmv, v_cache, s.head_dim, s.num_kv_heads, s.page_size, num_pages, kv_stride_page,
                             kv_stride_tok, kv_stride_head, box_rows, 1 << hg)) != PA_OK)
      return st;
    BlockParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride_tok = q_stride_tok;
    p.q_stride_head = q_stride_head;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.scale_stride = scale_stride;
    p.v = static_cast<const uint8_t*>(v_cache);
    p.v_stride_page = kv_stride_page;
    p.v_stride_tok = kv_stride_tok;
    p.v_stride_head = kv_stride_head;
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
    const int64_t rows = static_cast<int64_t>(2) * plan->ctas * NH << hg;
    p.o_part = reinterpret_cast<float*>(sc + kScratchHeaderBytes);
    p.lse_part = reinterpret_cast<float*>(sc + kScratchHeaderBytes + align_up(rows * s.head_dim * 4, 256));
    p.records = reinterpret_cast<MergeRecord*>(reinterpret_cast<uint8_t*>(p.lse_part) + align_up(rows * 4, 256));
    p.min_tiles = plan->min_tiles;
    p.hg_log2 = hg;
    p.err = reinterpret_cast<uint32_t*>(sc);
    const dim3 grid(plan->ctas);
    cudaError_t e;
    switch (s.head_dim) {
      case 64: e = launch_rows<64>(i8, NH / 8, tmk, tmv, p, grid, strm); break;
      case 128: e = launch_rows<128>(i8, NH / 8, tmk, tmv, p, grid, strm); break;
      default: e = launch_rows<256>(i8, NH / 8, tmk, tmv, p, grid, strm); break;
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
  cp.max_new = s.max_new;
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
    st = extend_over_copy(as_shape(s, PA_MODE_EXTEND), tmq, cp.kc, cp.vc, cp.page_scales, static_cast<int32_t>(n * maxp),
                          cp.bt_copy, cp.seq_lens, cp.qsl, n, total_q, s.max_new, scale, sinks, out, out_stride_tok,
                          out_stride_head, lse, sc, sc + at.work, stream);
    if (st != PA_OK) return st;
  }
  return PA_OK;
}
