// Append to a paged cache of 8-bit codes with a scale for each page and kv head.
//
// A page's new tokens set its scale: max |x| / Q (Q = 448 for e4m3, 127 for int8),
// or the scale it has if older tokens stay in it and theirs is larger; a code is
// the quotient x / scale rounded to the nearest code.  Where older tokens' scale
// grew their codes are rounded again.  Only the first page a request's new tokens
// touch can hold older ones.
//
// The call reads 2 bytes and writes 1 an element, an HBM stream; but the scale is
// known only when all new rows of a (page, head) have been seen.  GT threads take one
// (page, head, K or V), GT * 8 vectors of 8 elements at a time, which stay in
// registers until they are quantised; where a page brings more rows than that they
// are read again (from L2).  The groups that touch a page are found without a prefix
// sum: request b with first row q_b has at most floor(q_b / ps) + 2 b pages before
// it, so page number j of the call belongs to the last b with that number <= j, and
// some groups stay idle.
//
// Codes are those of the exact quotient x / scale, ties to even.  Where the scale is the
// new tokens' own, fp32(max / Q), one product x m decides:  in x Q / max, whose x and
// max have 8 bits, a midpoint of two codes is either met exactly or at least 2^-16 (int8:
// 127 i against (2n + 1) j, both below 2^16) or 2^-13 (e4m3: 7 i against M j, M below 2^5)
// of it away.  The exact quotient by the rounded scale lies next to a met midpoint on the
// side that the scale's rounding gives, the same for all elements; so m is 1 / scale moved
// 2^-22 to that side, more than the products' rounding and less than what separates the
// other elements from their midpoints.  (With bf16 inputs one element in 40 meets one:
// telling them apart one by one took 32 us instead of 21 for 16380 tokens.)  Where the scale
// is max / Q exactly, quotients are taken to fp32 with one Newton step, exact at a midpoint.
// Under an older scale, a scale next to the smallest numbers, or beside infinities and NaN,
// the products with both neighbours of m are compared, and where their codes differ the
// sign of the remainder x - h scale at the midpoint h decides, which one fma has exactly.
//
// Measured (one GB300, CUDA-graph replay, 8 heads of 128): 16380 tokens into int8 pages of 16
// 20.4 us, 4.9 TB/s of the bytes it cannot do without (73 % of the copy bandwidth; issue slots
// 62 % busy); 250 requests of one to five tokens into e4m3 pages of 64 9.6 us, 64 of one token
// 4.1 us: launch and a chain of five dependent loads.
#include <cstdint>
#include <type_traits>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "blocks.cuh"
#include "pa.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kCta = 256;

struct BlockAppendParams {
  const uint16_t* x[2];          // K, V
  int64_t new_stride_tok, new_stride_head;
  uint8_t* cache[2];
  int64_t stride_page, stride_tok, stride_head;   // bytes
  int num_pages, num_kv_heads, ps_log2;
  float* scales[2];
  int64_t scale_stride;
  const int32_t* block_table;
  int64_t bt_stride;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* qsl;            // null: one token a request
  int batch, num_tokens;
  uint32_t* err;
};

template <bool I8>
__device__ __forceinline__ uint32_t two_codes(float lo, float hi) {
  if constexpr (I8) {
    // (NaN converts to 0, infinities to the ends)
    const int a = max(-127, min(127, __float2int_rn(lo)));
    const int b = max(-127, min(127, __float2int_rn(hi)));
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8);
  } else {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
  }
}

// The number of code next to (hi + lo) / s, exactly, given t = hi * (1 / s) within 2^-23 of it;
// infinities and NaN stay.
template <bool I8>
__device__ __forceinline__ float nearest_code(float t, float hi, float lo, float s) {
  float below, above;                    // the codes around t
  bool odd;                              // `below` is the odd one
  if constexpr (I8) {
    below = floorf(t);
    above = below + 1.f;
    odd = (static_cast<int>(below) & 1) != 0;
  } else {
    // magnitudes: subnormals are multiples of 2^-9, normals have three bits behind the first
    const float a = fabsf(t);
    float lower, step;
    bool lower_odd;
    if (a < 0x1p-6f) {
      step = 0x1p-9f;
      lower = floorf(a * 0x1p9f);
      lower_odd = (static_cast<int>(lower) & 1) != 0;
      lower *= step;
    } else {
      const uint32_t u = __float_as_uint(a);
      lower = __uint_as_float(u & 0xfff00000u);
      step = __uint_as_float((u & 0x7f800000u) - (3u << 23));
      lower_odd = ((u >> 20) & 1u) != 0;
    }
    below = t < 0.f ? -(lower + step) : lower;
    above = t < 0.f ? -lower : lower + step;
    odd = t < 0.f ? !lower_odd : lower_odd;
  }
  const float h = 0.5f * (below + above);
  const float r = fmaf(-h, s, hi) + lo;  // (both terms exact: hi is next to h s)
  const float x = r > 0.f || (r == 0.f && odd) ? above : below;
  return fabsf(hi) < INFINITY ? x : hi;
}

// Eight finite numbers to the codes next to x * m, or, NEWTON, to x / s.
template <bool I8, bool NEWTON>
__device__ __forceinline__ uint2 to_codes8(const float (&x)[8], float m, float s) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = make_float2(x[2 * k], x[2 * k + 1]);
    const float2 m2 = make_float2(m, m);
    if constexpr (I8) {
      // x m + 1.5 * 2^23 rounds to a whole number, whose two's complement is the sum's low byte
      const float2 a = __ffma2_rn(v, m2, make_float2(12582912.f, 12582912.f));
      w[2 * k] = __float_as_uint(a.x);
      w[2 * k + 1] = __float_as_uint(a.y);
    } else {
      float2 q = __fmul2_rn(v, m2);
      if constexpr (NEWTON) q = __ffma2_rn(__ffma2_rn(make_float2(-q.x, -q.y), make_float2(s, s), v), m2, q);
      w[k] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
  }
  if constexpr (I8)
    return make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410));
  else
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Eight numbers x * was to codes, exactly, one at a time where the products do not decide
// (PRODUCT false: was is 1; all: no product does).
template <bool I8, bool PRODUCT>
__device__ __forceinline__ uint2 exact8(const float (&x)[8], float m, float was, float s, bool all) {
  const float above = m * (1.f + 0x1p-22f), below = m * (1.f - 0x1p-22f);
  uint2 out = to_codes8<I8, false>(x, above, s);
  const uint2 other = to_codes8<I8, false>(x, below, s);
  const uint32_t off[2] = {all ? 0xffffffffu : out.x ^ other.x, all ? 0xffffffffu : out.y ^ other.y};
  if ((off[0] | off[1]) == 0) return out;
#pragma unroll 1
  for (int at = 0; at < 8; ++at) {
    const uint32_t sh = 8u * (at & 3);
    if (((at < 4 ? off[0] : off[1]) >> sh & 0xffu) == 0) continue;
    float v = x[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) v = at == k ? x[k] : v;
    const float hi = PRODUCT ? __fmul_rn(v, was) : v;
    const float lo = PRODUCT ? __fmaf_rn(v, was, -hi) : 0.f;
    const uint32_t code = two_codes<I8>(nearest_code<I8>(v * m, hi, lo, s), 0.f) & 0xffu;
    uint32_t& w = at < 4 ? out.x : out.y;
    w = (w & ~(0xffu << sh)) | (code << sh);
  }
  return out;
}

__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(in[k] << 16);
    x[2 * k + 1] = __uint_as_float(in[k] & 0xffff0000u);
  }
}

template <bool I8>
__device__ __forceinline__ void code_values8(const uint2& w, float (&x)[8]) {
  const uint32_t in[2] = {w.x, w.y};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h[2];
    if constexpr (I8) {
      h[0] = int8x2_to_f16x2<0x4140>(in[k] ^ 0x80808080u);
      h[1] = int8x2_to_f16x2<0x4342>(in[k] ^ 0x80808080u);
    } else {
      h[0] = e4m3x2_to_f16x2<0>(in[k]);
      h[1] = e4m3x2_to_f16x2<1>(in[k]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      x[4 * k + 2 * i] = f.x;
      x[4 * k + 2 * i + 1] = f.y;
    }
  }
}

// The largest magnitudes (bf16 bits) of the even and the odd elements; a NaN stays one.
__device__ __forceinline__ uint32_t most_of(const uint4& w, uint32_t most) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(most) : "r"(in[k] & 0x7fff7fffu));
  return most;
}

// The largest magnitude of the finite elements.
__device__ __forceinline__ uint32_t most_finite(const uint4& w, uint32_t most) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = in[k] & 0x7fffu, hi = (in[k] >> 16) & 0x7fffu;
    most = max(most, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
  }
  return most;
}

// The larger half, over the group's threads (all threads of the CTA call it).
template <int GT>
__device__ __forceinline__ uint32_t group_most(uint32_t most, uint32_t* s_most) {
  most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
  if constexpr (GT > 32) {
    __syncthreads();                       // (an earlier call's reads)
    if ((threadIdx.x & 31) == 0) s_most[threadIdx.x >> 5] = most;
    __syncthreads();
    const int w0 = (threadIdx.x / GT) * (GT / 32);
#pragma unroll
    for (int w = 0; w < GT / 32; ++w) most = max(most, s_most[w0 + w]);
  }
  return most;
}

// GT threads a (page, kv head, K or V).
template <int D, bool I8, int GT>
__global__ void __launch_bounds__(kCta, 4) block_append_kernel(const BlockAppendParams p) {
  constexpr int NV = 8;                    // vectors a thread holds
  constexpr int DV = D / 8;                // vectors a row
  constexpr int RPS = GT / DV;             // rows a step of the group
  constexpr int ROWS = RPS * NV;           // rows the group holds
  static_assert(GT % 32 == 0 && GT % DV == 0, "a step covers whole rows");
  __shared__ uint32_t s_most[kCta / 32];
  const int lane = threadIdx.x & 31;
  const int lt = threadIdx.x % GT;
  const int ps_log2 = p.ps_log2;
  const int ps = 1 << ps_log2;
  const uint32_t group = blockIdx.x * (kCta / GT) + threadIdx.x / GT;
  const uint32_t nh = static_cast<uint32_t>(p.num_kv_heads);
  const uint32_t half = group / nh;
  const int h = static_cast<int>(group - half * nh);
  const int kv = static_cast<int>(half & 1);
  const int item = static_cast<int>(half >> 1);

  // ---- the request and its page ------------------------------------------
  int b = item;
  if (p.qsl != nullptr) {
    // 32 requests compared at a time
    int lo = 0, n = p.batch;                          // the last one is in [lo, lo + n)
    while (n > 1) {
      const int step = (n + 31) >> 5;
      const int at = lane * step;
      const bool fits = at < n && (p.qsl[lo + at] >> ps_log2) + 2 * static_cast<int64_t>(lo + at) <= item;
      const unsigned m = __ballot_sync(0xffffffffu, fits);
      const int k = m != 0 ? 31 - __clz(m) : 0;
      lo += k * step;
      n = min(step, n - k * step);
    }
    b = lo;
  }
  int page = -1, first = 0, end = 0;       // new tokens lie in slots [first, end) of the page
  int64_t row0 = 0;                        // packed row of slot 0
  if (b < p.batch) {
    const int qs = p.qsl != nullptr ? p.qsl[b] : b;
    const int L = p.seq_lens[b];
    const int n = p.qsl != nullptr ? packed_rows(qs, p.qsl[b + 1]) : (L == 0 ? 0 : 1);      // (L 0: a padded batch's request)
    const int64_t k = p.qsl != nullptr ? item - ((qs >> ps_log2) + 2 * static_cast<int64_t>(b)) : 0;
    if (n != 0) {
      if (n < 0 || L < n || L > (static_cast<int64_t>(p.max_pages) << ps_log2) || qs < 0 ||
          static_cast<int64_t>(qs) + n > p.num_tokens) {
        if (p.err != nullptr && k == 0 && lt == 0) atomicOr(p.err, kErrCapacity);
      } else if (k >= 0 && k <= (n >> ps_log2) + 1) {
        const int ctx = L - n;
        const int at = (ctx >> ps_log2) + static_cast<int>(k);
        const int64_t slot0 = static_cast<int64_t>(at) << ps_log2;
        if (slot0 < L) {
          first = static_cast<int>(max(int64_t{0}, ctx - slot0));
          end = static_cast<int>(min(static_cast<int64_t>(ps), L - slot0));
          row0 = static_cast<int64_t>(qs) + (slot0 - ctx);
          page = p.block_table[static_cast<int64_t>(b) * p.bt_stride + at];
        }
      }
    }
  }

  // ---- new rows and their largest value (asked for before the page's id is looked at) ----
  const int r0 = first + lt / DV;
  const int col = (lt % DV) * 8;
  const int64_t step = RPS * p.new_stride_tok;
  const uint16_t* src = p.x[kv] + (row0 + r0) * p.new_stride_tok + static_cast<int64_t>(h) * p.new_stride_head + col;
  const bool held = end - first <= ROWS;   // all rows at once
  uint4 x[NV];
  auto load = [&](int base) {
    const uint16_t* at = src + (base - r0) * p.new_stride_tok;
#pragma unroll
    for (int v = 0; v < NV; ++v, at += step)
      x[v] = base + v * RPS < end ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
  };
  uint32_t most = 0;
  for (int base = r0; base < end; base += ROWS) {
    load(base);
#pragma unroll
    for (int v = 0; v < NV; ++v) most = most_of(x[v], most);
  }
  if (page >= 0 ? page >= p.num_pages : end > 0) {
    if (p.err != nullptr && lt == 0) atomicOr(p.err, kErrPageId);
    page = -1;
  }
  float was = 0.f;
  if (page >= 0 && first > 0) was = p.scales[kv][static_cast<int64_t>(page) * p.scale_stride + h];
  most = group_most<GT>(most, s_most);
  const bool odd = most >= 0x7f80u;        // infinities or NaN, which do not count
  if (GT > 32 ? __syncthreads_or(odd) : odd) {
    most = 0;
    for (int base = r0; base < end; base += ROWS) {
      load(base);
#pragma unroll
      for (int v = 0; v < NV; ++v) most = most_finite(x[v], most);
    }
    most = group_most<GT>(most, s_most);
  }
  if (page < 0) return;

  // ---- scale, codes ----------------------------------------------------------
  const float fresh = __fdiv_rn(__uint_as_float(most << 16), I8 ? 127.f : 448.f);
  const float scale = fmaxf(fresh, was);
  uint8_t* dst = p.cache[kv] + static_cast<int64_t>(page) * p.stride_page + static_cast<int64_t>(h) * p.stride_head + col;
  const float rounding = fmaf(-scale, I8 ? 127.f : 448.f, __uint_as_float(most << 16));   // of a scale of its own
  const bool own = scale == fresh && scale >= 0x1p-60f && !odd;
  if (own) {
    float m = __frcp_rn(scale);
    if (rounding != 0.f) m *= rounding > 0.f ? 1.f + 0x1p-22f : 1.f - 0x1p-22f;
    auto store = [&](auto newton_tag) {
      for (int base = r0; base < end; base += ROWS) {
        if (!held) load(base);
        uint8_t* to = dst + base * p.stride_tok;
#pragma unroll
        for (int v = 0; v < NV; ++v, to += RPS * p.stride_tok) {
          if (base + v * RPS < end) {
            float f[8];
            widen8(x[v], f);
            *reinterpret_cast<uint2*>(to) = to_codes8<I8, decltype(newton_tag)::value>(f, m, scale);
          }
        }
      }
    };
    // (127 divides a bf16 number to fp32 exactly only where the quotient is a power of two, whose m is exact)
    if (!I8 && rounding == 0.f) {
      store(std::true_type{});
    } else {
      store(std::false_type{});
    }
  }
  if (!own || (first > 0 && scale > was)) {
    // a scale next to the smallest numbers, and what it divides, times 2^80 (exact); scale 0: all finite elements are 0
    const float lift = scale < 0x1p-60f ? 0x1p80f : 1.f;
    const float s = scale > 0.f ? scale * lift : 1.f;
    const float wl = was * lift;
    const float mw = __fdiv_rn(wl, s), mx = __frcp_rn(s);
    for (int r = lt / DV; r < end; r += RPS) {
      uint2* w = reinterpret_cast<uint2*>(dst + r * p.stride_tok);
      float f[8];
      if (r < first) {
        if (!(scale > was)) continue;
        code_values8<I8>(*w, f);
        *w = exact8<I8, true>(f, mw, wl, s, false);
      } else {
        if (own) break;
        widen8(*reinterpret_cast<const uint4*>(src + (r - r0) * p.new_stride_tok), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= lift;
        *w = exact8<I8, false>(f, mx, 1.f, s, odd);
      }
    }
  }
  if (lt == 0) p.scales[kv][static_cast<int64_t>(page) * p.scale_stride + h] = scale;
}

// Threads a group: as many as hold the rows a page gets on average (at most all of a
// page's, at least a warp).
template <int D, bool I8>
cudaError_t launch(const BlockAppendParams& p, int64_t items, cudaStream_t st) {
  const int64_t groups = items * 2 * p.num_kv_heads;
  const int64_t mean = (static_cast<int64_t>(p.num_tokens) + p.batch - 1) / p.batch;
  const int rows = static_cast<int>(mean < (1 << p.ps_log2) ? mean : 1 << p.ps_log2);
  const int threads = rows * (D / 8) / 8;
#define PA_APPEND(GT) \
  block_append_kernel<D, I8, GT><<<static_cast<unsigned>((groups + kCta / GT - 1) / (kCta / GT)), kCta, 0, st>>>(p)
  if (threads <= 32) {
    PA_APPEND(32);
  } else if (threads <= 64) {
    PA_APPEND(64);
  } else if (D == 64 || threads <= 128) {
    PA_APPEND(128);
  } else {
    PA_APPEND(256);
  }
#undef PA_APPEND
  return cudaGetLastError();
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_append_blocks(const void* k_new, const void* v_new, int64_t new_stride_tok,
                                      int64_t new_stride_head, void* k_cache, void* v_cache, int64_t kv_stride_page,
                                      int64_t kv_stride_tok, int64_t kv_stride_head, int32_t num_pages,
                                      int32_t page_size, int32_t num_kv_heads, int32_t head_dim, int32_t code,
                                      float* k_scales, float* v_scales, int64_t scale_stride,
                                      const int32_t* block_table, int64_t bt_stride, int32_t max_pages_per_seq,
                                      const int32_t* seq_lens, const int32_t* query_start_loc, int32_t batch,
                                      int32_t num_tokens, void* scratch, void* stream) {
  using namespace pa;
  if (batch < 0 || num_tokens < 0 || num_kv_heads <= 0 || num_pages <= 0 || max_pages_per_seq < 0 || bt_stride < 0)
    return PA_ERR_INVALID_ARG;
  if (code != PA_CODE_E4M3 && code != PA_CODE_INT8) return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_pages_per_seq) * page_size > (int64_t{1} << 30)) return PA_ERR_UNSUPPORTED;
  if (!query_start_loc && num_tokens != batch) return PA_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0) return PA_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !k_scales || !v_scales || !block_table || !seq_lens)
    return PA_ERR_INVALID_ARG;
  if (new_stride_tok <= 0 || new_stride_head <= 0 || kv_stride_page <= 0 || kv_stride_tok <= 0 || kv_stride_head <= 0)
    return PA_ERR_INVALID_ARG;
  if (bt_stride < max_pages_per_seq && batch > 1) return PA_ERR_INVALID_ARG;
  if (scale_stride < num_kv_heads && num_pages > 1) return PA_ERR_INVALID_ARG;
  auto off = [](const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) != 0; };
  if (off(k_new, 16) || off(v_new, 16) || new_stride_tok % 8 || new_stride_head % 8) return PA_ERR_UNSUPPORTED;
  if (off(k_cache, 16) || off(v_cache, 16) || kv_stride_page % 16 || kv_stride_tok % 16 || kv_stride_head % 16)
    return PA_ERR_UNSUPPORTED;
  if (off(k_scales, 4) || off(v_scales, 4) || off(block_table, 4) || off(seq_lens, 4) || off(query_start_loc, 4) ||
      off(scratch, 4))
    return PA_ERR_UNSUPPORTED;
  // pages that hold new tokens: at most n / ps + 2 of a request, as the kernel counts them
  const int64_t items = query_start_loc ? num_tokens / page_size + 2 * static_cast<int64_t>(batch) : batch;
  if (items * 2 * num_kv_heads > (int64_t{1} << 31) - kCta) return PA_ERR_UNSUPPORTED;
  BlockAppendParams p{};
  p.x[0] = static_cast<const uint16_t*>(k_new);
  p.x[1] = static_cast<const uint16_t*>(v_new);
  p.new_stride_tok = new_stride_tok;
  p.new_stride_head = new_stride_head;
  p.cache[0] = static_cast<uint8_t*>(k_cache);
  p.cache[1] = static_cast<uint8_t*>(v_cache);
  p.stride_page = kv_stride_page;
  p.stride_tok = kv_stride_tok;
  p.stride_head = kv_stride_head;
  p.num_pages = num_pages;
  p.num_kv_heads = num_kv_heads;
  p.ps_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : 6;
  p.scales[0] = k_scales;
  p.scales[1] = v_scales;
  p.scale_stride = scale_stride;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.err = static_cast<uint32_t*>(scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = code == PA_CODE_INT8;
  cudaError_t e;
  switch (head_dim) {
    case 64: e = i8 ? launch<64, true>(p, items, st) : launch<64, false>(p, items, st); break;
    case 128: e = i8 ? launch<128, true>(p, items, st) : launch<128, false>(p, items, st); break;
    default: e = i8 ? launch<256, true>(p, items, st) : launch<256, false>(p, items, st); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
