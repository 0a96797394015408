// Append to a paged cache of 8-bit codes with a scale for each page and kv head.
//
// A page's new tokens set its scale: max |x| / Q (Q = 448 for e4m3, 127 for int8),
// or the scale it has if older tokens stay in it and theirs is larger; a code is
// the quotient x / scale rounded to the nearest code.  Where older tokens' scale
// grew their codes are rounded again.  Only the first page a request's new tokens
// touch can hold older ones.
//
// The call reads 2 bytes and writes 1 an element, an HBM stream; but the scale is
// known only when all of a (page, head) has been seen, so its new rows are held in
// registers (GT threads with NV vectors of 8 elements cover page_size rows of one
// head) from the one read to the quantisation.  The groups that touch a page are
// found without a prefix sum: request b with first row q_b has at most
// floor(q_b / ps) + 2 b groups of pages before it, so group j looks for the last b
// with that number <= j, and a few groups stay idle.
//
// Quotients are rounded exactly (ties to even): the fp32 quotient is made odd where
// it is inexact, which no tie of 8-bit codes survives, and rounds on to the code.
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

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
  int num_pages, num_kv_heads;
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

// x / s for s > 0 in fp32, rounded to odd: where it is inexact and the rounded
// quotient even, its neighbour on the exact quotient's side.  (The remainder of a
// rounded quotient is exact in an fma, or has the exact one's sign.)
__device__ __forceinline__ float quotient_odd(float x, float s) {
  const float q = __fdiv_rn(x, s);
  const float r = fmaf(-q, s, x);
  const int bits = __float_as_int(q);
  if ((bits & 1) == 0 && q != 0.f) {
    const bool out = q > 0.f ? r > 0.f : r < 0.f;      // the exact quotient is larger in magnitude
    const bool in = q > 0.f ? r < 0.f : r > 0.f;
    return __int_as_float(bits + (out ? 1 : 0) - (in ? 1 : 0));
  }
  return q;
}

// (fp32 rounded to odd of a 64-bit number)
__device__ __forceinline__ float odd_of(double q) {
  const float f = __double2float_rz(q);
  return static_cast<double>(f) != q ? __int_as_float(__float_as_int(f) | 1) : f;
}

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

template <bool I8>
__device__ __forceinline__ uint2 quantise8(const uint4& w, float scale) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo = __uint_as_float(in[k] << 16), hi = __uint_as_float(in[k] & 0xffff0000u);
    if (scale > 0.f) {                    // (0: every finite element is 0)
      lo = quotient_odd(lo, scale);
      hi = quotient_odd(hi, scale);
    }
    out[k >> 1] |= two_codes<I8>(lo, hi) << (16 * (k & 1));
  }
  return make_uint2(out[0], out[1]);
}

template <bool I8>
__device__ __forceinline__ double code_value(uint32_t byte) {
  if constexpr (I8) {
    return static_cast<double>(static_cast<int>(static_cast<int8_t>(byte)));
  } else {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    return static_cast<double>(__half2float(__half(h)));
  }
}

// Eight codes under a larger scale.
template <bool I8>
__device__ __forceinline__ uint2 requantise8(uint2 w, float was, float scale) {
  const uint32_t in[2] = {w.x, w.y};
  uint32_t out[2] = {0u, 0u};
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const uint32_t pair = in[k >> 1] >> (16 * (k & 1));
    // (the product of an 8-bit and a 24-bit number is exact)
    const double a = code_value<I8>(pair & 0xffu) * static_cast<double>(was);
    const double b = code_value<I8>((pair >> 8) & 0xffu) * static_cast<double>(was);
    out[k >> 1] |= two_codes<I8>(odd_of(a / static_cast<double>(scale)), odd_of(b / static_cast<double>(scale)))
                   << (16 * (k & 1));
  }
  return make_uint2(out[0], out[1]);
}

// GT threads a (page, kv head, K or V), NV vectors of 8 elements each.
template <int D, bool I8, int GT, int NV>
__global__ void __launch_bounds__(kCta) block_append_kernel(const BlockAppendParams p) {
  constexpr int DV = D / 8;                // vectors a row
  constexpr int PS = GT * NV / DV;         // page size
  constexpr int RPS = GT / DV;             // rows a step of the group (GT >= DV)
  static_assert(GT % 32 == 0 && GT % DV == 0 && PS * DV == GT * NV, "a group covers whole rows");
  __shared__ uint32_t s_most[kCta / 32];
  const int lt = threadIdx.x % GT;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * (kCta / GT) + threadIdx.x / GT;
  const int h = static_cast<int>(group % p.num_kv_heads);
  const int64_t rest = group / p.num_kv_heads;
  const int kv = static_cast<int>(rest & 1);
  const int64_t item = rest >> 1;

  // ---- the request and its page ------------------------------------------
  int b = 0, page = -1, first = 0, end = 0;    // new tokens lie in slots [first, end) of the page
  int64_t row0 = 0;                            // packed row of slot 0
  int at = 0;
  if (p.qsl == nullptr) {
    b = static_cast<int>(item);
  } else {
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.qsl[mid] / PS + 2 * static_cast<int64_t>(mid) <= item) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  if (b < p.batch) {
    const int qs = p.qsl != nullptr ? p.qsl[b] : b;
    const int n = p.qsl != nullptr ? p.qsl[b + 1] - qs : 1;
    const int L = p.seq_lens[b];
    const int64_t k = p.qsl != nullptr ? item - (qs / PS + 2 * static_cast<int64_t>(b)) : 0;
    if (n != 0) {
      if (n < 0 || L < n || L > static_cast<int64_t>(p.max_pages) * PS || qs < 0 ||
          static_cast<int64_t>(qs) + n > p.num_tokens) {
        if (p.err != nullptr && k == 0 && lt == 0) atomicOr(p.err, kErrCapacity);
      } else if (k >= 0 && k <= n / PS + 1) {
        const int ctx = L - n;
        at = ctx / PS + static_cast<int>(k);
        if (static_cast<int64_t>(at) * PS < L) {
          first = max(0, ctx - at * PS);
          end = min(PS, L - at * PS);
          row0 = static_cast<int64_t>(qs) + (static_cast<int64_t>(at) * PS - ctx);
          page = p.block_table[static_cast<int64_t>(b) * p.bt_stride + at];
          if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
            if (p.err != nullptr && lt == 0) atomicOr(p.err, kErrPageId);
            page = -1;
          }
        }
      }
    }
  }

  // ---- new rows and their largest value ------------------------------------
  const int r0 = lt / DV;
  const int col = (lt % DV) * 8;
  uint4 x[NV];
  uint32_t most = 0;
  float was = 0.f;
  if (page >= 0) {
    const uint16_t* src = p.x[kv] + static_cast<int64_t>(h) * p.new_stride_head + col;
    if (first > 0) was = p.scales[kv][static_cast<int64_t>(page) * p.scale_stride + h];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int r = r0 + v * RPS;
      x[v] = make_uint4(0, 0, 0, 0);
      if (r >= first && r < end)
        x[v] = *reinterpret_cast<const uint4*>(src + (row0 + r) * p.new_stride_tok);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t w[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
        if (lo < 0x7f80u) most = max(most, lo);      // infinities and NaN do not count
        if (hi < 0x7f80u) most = max(most, hi);
      }
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if constexpr (GT > 32) {
    if ((threadIdx.x & 31) == 0) s_most[threadIdx.x >> 5] = most;
    __syncthreads();
    const int w0 = (threadIdx.x / GT) * (GT / 32);
#pragma unroll
    for (int w = 0; w < GT / 32; ++w) most = max(most, s_most[w0 + w]);
  }
  if (page < 0) return;

  // ---- scale, codes ----------------------------------------------------------
  const float fresh = __fdiv_rn(__uint_as_float(most << 16), I8 ? 127.f : 448.f);
  const float scale = fmaxf(fresh, was);
  uint8_t* dst = p.cache[kv] + static_cast<int64_t>(page) * p.stride_page + static_cast<int64_t>(h) * p.stride_head + col;
  if (first > 0 && scale > was) {
#pragma unroll 1
    for (int r = r0; r < first; r += RPS) {
      uint2* w = reinterpret_cast<uint2*>(dst + r * p.stride_tok);
      *w = requantise8<I8>(*w, was, scale);
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int r = r0 + v * RPS;
    if (r >= first && r < end) *reinterpret_cast<uint2*>(dst + r * p.stride_tok) = quantise8<I8>(x[v], scale);
  }
  if (lt == 0) p.scales[kv][static_cast<int64_t>(page) * p.scale_stride + h] = scale;
}

template <int D, bool I8>
cudaError_t launch(int page_size, const BlockAppendParams& p, int64_t items, cudaStream_t st) {
  // threads a group: 8 vectors each, at least a warp
  const int64_t groups = items * 2 * p.num_kv_heads;
#define PA_APPEND(GT, NV)                                                                  \
  block_append_kernel<D, I8, GT, NV>                                                       \
      <<<static_cast<unsigned>((groups + kCta / GT - 1) / (kCta / GT)), kCta, 0, st>>>(p); \
  return cudaGetLastError()
  if constexpr (D == 64) {
    if (page_size == 16) { PA_APPEND(32, 4); }
    if (page_size == 32) { PA_APPEND(32, 8); }
    PA_APPEND(64, 8);
  } else if constexpr (D == 128) {
    if (page_size == 16) { PA_APPEND(32, 8); }
    if (page_size == 32) { PA_APPEND(64, 8); }
    PA_APPEND(128, 8);
  } else {
    if (page_size == 16) { PA_APPEND(64, 8); }
    if (page_size == 32) { PA_APPEND(128, 8); }
    PA_APPEND(256, 8);
  }
#undef PA_APPEND
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
    case 64: e = i8 ? launch<64, true>(page_size, p, items, st) : launch<64, false>(page_size, p, items, st); break;
    case 128: e = i8 ? launch<128, true>(page_size, p, items, st) : launch<128, false>(page_size, p, items, st); break;
    default: e = i8 ? launch<256, true>(page_size, p, items, st) : launch<256, false>(page_size, p, items, st); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
