// Key bounds of pages: per page, kv head and dim the smallest and the largest
// key value over the page's filled slots.  For any query q,
//   sum_d max(q_d lo_d, q_d hi_d) >= q . k   for every key k of the page,
// which is the score page selection ranks pages by.
//
// Minimum and maximum of bf16 values are values themselves, so the bounds are
// exact and do not depend on the order they are taken in: a page that changed
// is simply computed again.  e4m3 codes compare as f16 (exact) and the two
// winners alone are dequantised to bf16(float(code) * scale): one rounding is
// monotone, and a negative scale swaps the two.
//
// The kernel reads the changed pages' keys once and writes 2 D values per page
// and head: an HBM stream.  A thread owns 16 bytes of a (page, head) row and
// walks the page's slots, two batches of loads in flight; neighbouring threads own
// neighbouring bytes, so a slot of all heads is one contiguous read.  The pages
// to do lie in [first, last] of every request; a CTA lists them by a prefix sum
// over the requests and takes every gridDim-th group, so requests of any
// lengths share the machine evenly and the host needs to know none of them.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "pa.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

struct BoundsParams {
  const uint8_t* k_cache;
  int64_t stride_page, stride_tok, stride_head;   // bytes
  int num_pages, page_size, num_kv_heads;
  const int32_t* block_table;
  int64_t bt_stride;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* qsl;
  int batch;
  float k_scale;
  const float* k_scales;
  uint16_t* bounds;
  int64_t bounds_stride_page, bounds_stride_head;
  uint32_t* err;
};

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two e4m3 codes (the low or high half of w) as f16x2, exactly.
template <int HALF>
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (HALF == 0) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  }
  return r;
}

// bf16x2 of f16x2 * scale: the product in fp32, then one rounding.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t v, float scale) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return pack_bf16x2(f.x * scale, f.y * scale);
}

// E: bytes per element.  A 16-byte unit holds 16 / E elements of one head.
template <int D, int E>
__global__ void __launch_bounds__(kThreads) page_bounds_kernel(const BoundsParams p) {
  constexpr int UPH = D * E / 16;             // units per (page, head)
  constexpr int NE = 16 / E;                  // elements per unit
  // slots of a batch: fewer registers and more CTAs for bf16 (8 whole contexts 62.9
  // us with 4, 69.4 with 8), more in flight for the small e4m3 pages (8.8 / 11.6)
  constexpr int kUnroll = E == 2 ? 4 : 8;
  __shared__ int s_end[kThreads];             // pages of requests [base, base + i], summed
  __shared__ int s_first[kThreads];           // first page to do
  __shared__ int s_len[kThreads];
  __shared__ int s_warp[kThreads / 32];
  const int tid = threadIdx.x;
  const int ps = p.page_size;
  const int units = p.num_kv_heads * UPH;     // per page
  // a CTA takes `ppc` pages at a time (or a page in several rounds)
  const int ppc = units >= kThreads ? 1 : kThreads / units;
  int64_t skipped = 0;                        // groups of the requests before this chunk

  for (int base = 0; base < p.batch; base += kThreads) {
    // pages to do of up to kThreads requests, and their running sum
    int n = 0, first = 0, L = 0;
    const int b0 = base + tid;
    if (b0 < p.batch) {
      L = p.seq_lens[b0];
      const int fresh = p.qsl != nullptr ? p.qsl[b0 + 1] - p.qsl[b0] : L;
      if (L < 0 || fresh < 0 || fresh > L || L > static_cast<int64_t>(p.max_pages) * ps) {
        if (p.err != nullptr && blockIdx.x == 0) atomicOr(p.err, kErrCapacity);
      } else if (fresh > 0) {
        first = (L - fresh) / ps;
        n = (L + ps - 1) / ps - first;
      }
    }
    int sum = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, m);
      if ((tid & 31) >= m) sum += v;
    }
    if ((tid & 31) == 31) s_warp[tid >> 5] = sum;
    __syncthreads();
    for (int w = 0; w < (tid >> 5); ++w) sum += s_warp[w];
    s_end[tid] = sum;
    s_first[tid] = first;
    s_len[tid] = L;
    __syncthreads();
    const int total = s_end[kThreads - 1];
    const int groups = (total + ppc - 1) / ppc;

    // (the rotation by `skipped` continues the round robin of the chunk before)
    int g = static_cast<int>((static_cast<int64_t>(blockIdx.x) + gridDim.x - skipped % gridDim.x) % gridDim.x);
    for (; g < groups; g += gridDim.x) {
      for (int u0 = tid; u0 < ppc * units; u0 += kThreads) {
        const int item = g * ppc + u0 / units;
        if (item >= total) continue;
        int lo = 0, hi = kThreads - 1;        // first request whose running sum exceeds `item`
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s_end[mid] > item) hi = mid; else lo = mid + 1;
        }
        const int b = base + lo;
        const int pg = s_first[lo] + item - (lo > 0 ? s_end[lo - 1] : 0);
        const int u = u0 % units;
        const int h = u / UPH;
        const int part = u - h * UPH;
        const int id = p.block_table[b * p.bt_stride + pg];
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
          if (p.err != nullptr && u == 0) atomicOr(p.err, kErrPageId);
          continue;
        }
        const int filled = min(ps, s_len[lo] - pg * ps);
        const uint8_t* src = p.k_cache + id * p.stride_page + h * p.stride_head + part * 16;
        uint16_t* dst = p.bounds + id * p.bounds_stride_page + h * p.bounds_stride_head + part * NE;
        // Batches of kUnroll slots, the next one's loads ahead of this one's
        // comparisons; beyond the filled slots the last of them is read again.
        uint32_t mn[16 / E / 2], mx[16 / E / 2];
        uint4 w[2][kUnroll];
        auto load = [&](uint4 (&x)[kUnroll], int s0) {
#pragma unroll
          for (int k = 0; k < kUnroll; ++k)
            x[k] = *reinterpret_cast<const uint4*>(src + min(s0 + k, filled - 1) * p.stride_tok);
        };
        auto fold = [&](const uint4 (&x)[kUnroll]) {
#pragma unroll
          for (int k = 0; k < kUnroll; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v = (&x[k].x)[i];
              if constexpr (E == 2) {
                mn[i] = min_bf16x2(mn[i], v);
                mx[i] = max_bf16x2(mx[i], v);
              } else {
                const uint32_t y0 = e4m3x2_f16x2<0>(v), y1 = e4m3x2_f16x2<1>(v);
                mn[2 * i] = min_f16x2(mn[2 * i], y0);
                mx[2 * i] = max_f16x2(mx[2 * i], y0);
                mn[2 * i + 1] = min_f16x2(mn[2 * i + 1], y1);
                mx[2 * i + 1] = max_f16x2(mx[2 * i + 1], y1);
              }
            }
        };
        load(w[0], 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = (&w[0][0].x)[i];
          if constexpr (E == 2) {
            mn[i] = mx[i] = v;
          } else {
            mn[2 * i] = mx[2 * i] = e4m3x2_f16x2<0>(v);
            mn[2 * i + 1] = mx[2 * i + 1] = e4m3x2_f16x2<1>(v);
          }
        }
        for (int s0 = 0; s0 < filled; s0 += 2 * kUnroll) {
          if (s0 + kUnroll < filled) load(w[1], s0 + kUnroll);
          fold(w[0]);
          if (s0 + kUnroll >= filled) break;
          if (s0 + 2 * kUnroll < filled) load(w[0], s0 + 2 * kUnroll);
          fold(w[1]);
        }
        if constexpr (E == 2) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
          *reinterpret_cast<uint4*>(dst + D) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
        } else {
          const float scale = p.k_scales != nullptr ? p.k_scales[b] : p.k_scale;
          uint32_t a[8], z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t l = scale_f16x2(mn[i], scale), r = scale_f16x2(mx[i], scale);
            a[i] = scale < 0.f ? r : l;
            z[i] = scale < 0.f ? l : r;
          }
          uint4* lo4 = reinterpret_cast<uint4*>(dst);
          uint4* hi4 = reinterpret_cast<uint4*>(dst + D);
          lo4[0] = make_uint4(a[0], a[1], a[2], a[3]);
          lo4[1] = make_uint4(a[4], a[5], a[6], a[7]);
          hi4[0] = make_uint4(z[0], z[1], z[2], z[3]);
          hi4[1] = make_uint4(z[4], z[5], z[6], z[7]);
        }
      }
    }
    skipped += groups;
    __syncthreads();   // the tables are rewritten for the next chunk
  }
}

template <int D>
cudaError_t launch(const BoundsParams& p, bool fp8, int ctas, cudaStream_t st) {
  if (fp8) {
    page_bounds_kernel<D, 1><<<ctas, kThreads, 0, st>>>(p);
  } else {
    page_bounds_kernel<D, 2><<<ctas, kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_page_bounds(const void* k_cache, int64_t kv_stride_page, int64_t kv_stride_tok,
                                    int64_t kv_stride_head, int32_t num_pages, int32_t page_size,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t kv_dtype,
                                    const int32_t* block_table, int64_t bt_stride, int32_t max_pages_per_seq,
                                    const int32_t* seq_lens, const int32_t* query_start_loc, int32_t batch,
                                    float k_scale, const float* k_scales, void* bounds, int64_t bounds_stride_page,
                                    int64_t bounds_stride_head, void* scratch, void* stream) {
  using namespace pa;
  if (batch < 0 || num_kv_heads <= 0 || num_pages <= 0 || max_pages_per_seq < 0) return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64) return PA_ERR_UNSUPPORTED;
  if (num_kv_heads > (1 << 16) || static_cast<int64_t>(max_pages_per_seq) * page_size > (int64_t{1} << 30))
    return PA_ERR_UNSUPPORTED;
  const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
  if (fp8 && !std::isfinite(k_scale)) return PA_ERR_INVALID_ARG;
  if (batch == 0) return PA_OK;
  // a CTA sums the pages of 256 requests in 32 bits
  if (static_cast<int64_t>(max_pages_per_seq) * std::min(batch, kThreads) > (int64_t{1} << 30)) return PA_ERR_UNSUPPORTED;
  if (!k_cache || !block_table || !seq_lens || !bounds || bt_stride < max_pages_per_seq) return PA_ERR_INVALID_ARG;
  if (kv_stride_page <= 0 || kv_stride_tok <= 0 || kv_stride_head <= 0 || bounds_stride_page <= 0 ||
      bounds_stride_head <= 0)
    return PA_ERR_INVALID_ARG;
  const int e = fp8 ? 1 : 2;
  auto a16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
  if (!a16(k_cache) || (kv_stride_page * e) % 16 || (kv_stride_tok * e) % 16 || (kv_stride_head * e) % 16 ||
      !a16(bounds) || bounds_stride_page % 8 || bounds_stride_head % 8 || reinterpret_cast<uintptr_t>(scratch) % 4)
    return PA_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  BoundsParams p{};
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.stride_page = kv_stride_page * e;
  p.stride_tok = kv_stride_tok * e;
  p.stride_head = kv_stride_head * e;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.num_kv_heads = num_kv_heads;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.batch = batch;
  p.k_scale = k_scale;
  p.k_scales = fp8 ? k_scales : nullptr;
  p.bounds = static_cast<uint16_t*>(bounds);
  p.bounds_stride_page = bounds_stride_page;
  p.bounds_stride_head = bounds_stride_head;
  p.err = static_cast<uint32_t*>(scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int ctas = sms * 4;   // as many as the registers let share an SM (5 would take a second wave: 74.7 us for 62.9)
  const cudaError_t r = head_dim == 64 ? launch<64>(p, fp8, ctas, st)
                        : head_dim == 128 ? launch<128>(p, fp8, ctas, st) : launch<256>(p, fp8, ctas, st);
  return r == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
