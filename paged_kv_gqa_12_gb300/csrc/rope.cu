// Norm, rotate and append: the queries and keys of new tokens take a per-head
// RMS norm and their rotation on the way from the projection to q_out and the
// paged cache; the values go along unchanged.
//
// Per (token, head) row x of D elements, in fp32:
//   y = x * rsqrt(sum x^2 / D + eps) * (w + offset)            (where w is given)
//   (a, b) <- (a cos - b sin, b cos + a sin)                   per rotated pair
// and one rounding at the end, to bf16 or to e4m3(y / scale).
//
// Every byte is touched once (read q, k, v; write q_out and two slots), so the
// kernel is an HBM stream.  D / 8 lanes share a row; lane j holds the four
// pairs 4j .. 4j+3, i.e. two 4-element vectors: the two halves' when pairs lie
// rot_dim / 2 apart, neighbours when they are interleaved or do not rotate.  A
// pair's two elements are therefore always in one lane and the rotation needs
// no exchange; the norm needs log2(D / 8) shuffles.  A CTA takes one token's
// rows: cosines and sines are read once per lane and used for all its rows.
#include <cmath>
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "pa.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

struct RopeParams {
  const uint16_t* q;
  int64_t q_stride_tok, q_stride_head;
  uint16_t* q_out;
  int64_t qo_stride_tok, qo_stride_head;
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t new_stride_tok, new_stride_head;
  const int32_t* positions;
  int64_t positions_stride;
  const float* cos_sin;
  int64_t cos_sin_stride;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  float norm_eps, norm_offset;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t stride_page, stride_tok, stride_head;   // bytes
  int num_pages, page_size, ps_log2, num_q_heads, num_kv_heads, num_tokens;   // ps_log2: -1, no power of two
  int half;              // rot_dim / 2
  int interleaved, num_axes, max_position;
  int axis_end[4];       // first pair behind each axis
  const int64_t* slot_mapping;
  float k_scale, v_scale;
  uint32_t* err;         // optional error word
};

__device__ __forceinline__ void unpack4(uint2 w, float* x) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xffff0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xffff0000u);
}

__device__ __forceinline__ uint32_t quant4(const float* x, float scale) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)),
                                               __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <int D, bool FP8, int U>
__global__ void __launch_bounds__(kThreads) append_rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 8;                  // lanes per row
  constexpr int ROWS = kThreads / LPR;        // rows a CTA holds at a time
  const int t = blockIdx.x;
  const int lane = threadIdx.x % LPR;
  const int sub = threadIdx.x / LPR;
  // this lane's two 4-element vectors of a row
  const bool turns = 4 * lane < p.half;
  const bool apart = turns && !p.interleaved;
  const int da = apart ? 4 * lane : 8 * lane;
  const int db = apart ? p.half + 4 * lane : 8 * lane + 4;

  // U rows at a time, their loads ahead of everything else
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  uint2 wa[U], wb[U];
  auto kind_of = [&](int r) { return r < p.num_q_heads ? 0 : (r < p.num_q_heads + p.num_kv_heads ? 1 : 2); };   // q, k, v
  auto head_of = [&](int r, int kind) { return kind == 0 ? r : r - p.num_q_heads - (kind - 1) * p.num_kv_heads; };
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * ROWS + sub;
      wa[u] = wb[u] = make_uint2(0u, 0u);
      if (r < rows) {
        const int kind = kind_of(r), h = head_of(r, kind);
        const uint16_t* src = kind == 0 ? p.q + t * p.q_stride_tok + h * p.q_stride_head
                              : (kind == 1 ? p.k_new : p.v_new) + t * p.new_stride_tok + h * p.new_stride_head;
        wa[u] = *reinterpret_cast<const uint2*>(src + da);
        wb[u] = *reinterpret_cast<const uint2*>(src + db);
      }
    }
  };
  load(0);

  const int64_t slot = p.slot_mapping[t];
  if (slot < 0) return;                       // padding token
  const int64_t page = p.ps_log2 >= 0 ? slot >> p.ps_log2 : slot / p.page_size;
  if (page >= p.num_pages) {                  // outside the pool: nothing written
    if (p.err != nullptr && threadIdx.x == 0) atomicOr(p.err, kErrPageId);
    return;
  }
  int pos[4] = {0, 0, 0, 0};
  bool bad = false;
  if (p.half > 0) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (a < p.num_axes) {
        pos[a] = p.positions[a * p.positions_stride + t];
        bad |= static_cast<unsigned>(pos[a]) >= static_cast<unsigned>(p.max_position);
      }
  }
  if (bad) {
    if (p.err != nullptr && threadIdx.x == 0) atomicOr(p.err, PA_DEVICE_POSITION);
    return;
  }

  // the cosines and sines of this lane's four pairs
  float cs[4], sn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) cs[e] = 1.f, sn[e] = 0.f;
  if (turns) {
    if (p.num_axes == 1) {
      const float* row = p.cos_sin + pos[0] * p.cos_sin_stride + 4 * lane;
      const float4 c = __ldg(reinterpret_cast<const float4*>(row));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + p.half));
      cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
      sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int pair = 4 * lane + e;
        const int ps = pair < p.axis_end[0] ? pos[0]
                       : pair < p.axis_end[1] ? pos[1] : pair < p.axis_end[2] ? pos[2] : pos[3];
        const float* row = p.cos_sin + ps * p.cos_sin_stride + pair;
        cs[e] = __ldg(row);
        sn[e] = __ldg(row + p.half);
      }
    }
  }

  const int64_t cell = page * p.stride_page + (slot - page * p.page_size) * p.stride_tok;
  const bool norms = p.q_norm != nullptr || p.k_norm != nullptr;
  for (int r0 = 0; r0 < rows; r0 += U * ROWS) {
    if (r0 > 0) load(r0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * ROWS + sub;
      const int kind = kind_of(r), h = head_of(r, kind);
      float a[4], b[4];
      unpack4(wa[u], a);
      unpack4(wb[u], b);
      if (norms) {   // (the same for the whole CTA: every lane of the warp shuffles)
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const uint16_t* w = kind == 0 ? p.q_norm : (kind == 1 ? p.k_norm : nullptr);
        if (w != nullptr) {
          const float rs = rsqrtf(ss * (1.f / D) + p.norm_eps);
          float x[4], y[4];
          unpack4(__ldg(reinterpret_cast<const uint2*>(w + da)), x);
          unpack4(__ldg(reinterpret_cast<const uint2*>(w + db)), y);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] *= rs * (x[e] + p.norm_offset);
            b[e] *= rs * (y[e] + p.norm_offset);
          }
        }
      }
      if (r >= rows) continue;
      if (turns && kind != 2) {
        if (p.interleaved) {   // pairs (a0, a1), (a2, a3), (b0, b1), (b2, b3)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float x = a[e], y = b[e];
            a[e] = x * cs[e / 2] - a[e + 1] * sn[e / 2];
            a[e + 1] = a[e + 1] * cs[e / 2] + x * sn[e / 2];
            b[e] = y * cs[2 + e / 2] - b[e + 1] * sn[2 + e / 2];
            b[e + 1] = b[e + 1] * cs[2 + e / 2] + y * sn[2 + e / 2];
          }
        } else {               // pairs (a_e, b_e)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = a[e];
            a[e] = x * cs[e] - b[e] * sn[e];
            b[e] = b[e] * cs[e] + x * sn[e];
          }
        }
      }
      if (FP8 && kind != 0) {
        uint8_t* dst = (kind == 1 ? p.k_cache : p.v_cache) + cell + h * p.stride_head;
        const float scale = kind == 1 ? p.k_scale : p.v_scale;
        *reinterpret_cast<uint32_t*>(dst + da) = quant4(a, scale);
        *reinterpret_cast<uint32_t*>(dst + db) = quant4(b, scale);
      } else {
        uint16_t* dst = kind == 0 ? p.q_out + t * p.qo_stride_tok + h * p.qo_stride_head
                                  : reinterpret_cast<uint16_t*>((kind == 1 ? p.k_cache : p.v_cache) + cell +
                                                                h * p.stride_head);
        if (kind != 2) {       // (values keep their bits)
          wa[u] = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
          wb[u] = make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
        }
        *reinterpret_cast<uint2*>(dst + da) = wa[u];
        *reinterpret_cast<uint2*>(dst + db) = wb[u];
      }
    }
  }
}

template <int D, bool FP8>
cudaError_t launch_rows(const RopeParams& p, cudaStream_t st) {
  const int passes = (p.num_q_heads + 2 * p.num_kv_heads + kThreads / (D / 8) - 1) / (kThreads / (D / 8));
  auto kern = passes == 1 ? append_rope_kernel<D, FP8, 1> : passes == 2 ? append_rope_kernel<D, FP8, 2>
              : passes == 3 ? append_rope_kernel<D, FP8, 3> : append_rope_kernel<D, FP8, 4>;
  kern<<<p.num_tokens, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const RopeParams& p, bool fp8, cudaStream_t st) {
  return fp8 ? launch_rows<D, true>(p, st) : launch_rows<D, false>(p, st);
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_append_rope_kv(const pa_rope* rope, const void* q, int64_t q_stride_tok,
                                       int64_t q_stride_head, void* q_out, int64_t q_out_stride_tok,
                                       int64_t q_out_stride_head, int32_t num_q_heads, const void* k_new,
                                       const void* v_new, int64_t new_stride_tok, int64_t new_stride_head,
                                       const int32_t* positions, int64_t positions_stride, void* k_cache,
                                       void* v_cache, int64_t kv_stride_page, int64_t kv_stride_tok,
                                       int64_t kv_stride_head, int32_t num_pages, int32_t page_size,
                                       int32_t num_kv_heads, int32_t head_dim, int32_t kv_dtype,
                                       const int64_t* slot_mapping, int32_t num_tokens, float k_scale, float v_scale,
                                       void* scratch, void* stream) {
  using namespace pa;
  if (!rope || num_tokens < 0 || num_kv_heads <= 0 || num_q_heads < 0 || page_size <= 0 || num_pages <= 0)
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_q_heads) + 2 * static_cast<int64_t>(num_kv_heads) > (1 << 20)) return PA_ERR_UNSUPPORTED;
  const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
  if (fp8 && !(k_scale > 0.f && v_scale > 0.f)) return PA_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr) || (q != nullptr) != (num_q_heads > 0)) {
    if (num_tokens > 0) return PA_ERR_INVALID_ARG;
  }
  const int rot = rope->rot_dim;
  if (rot < 0 || rot > head_dim) return PA_ERR_INVALID_ARG;
  if (rot % 8) return PA_ERR_UNSUPPORTED;
  if (rope->interleaved != 0 && rope->interleaved != 1) return PA_ERR_INVALID_ARG;
  if (!(rope->norm_eps >= 0.f) || !std::isfinite(rope->norm_eps) || !std::isfinite(rope->norm_offset))
    return PA_ERR_INVALID_ARG;
  if (rot > 0) {
    if (rope->num_axes < 1 || rope->num_axes > 4 || rope->max_position <= 0) return PA_ERR_INVALID_ARG;
    if (rope->num_axes > 1) {
      int64_t sum = 0;
      for (int a = 0; a < rope->num_axes; ++a) {
        if (rope->sections[a] < 0) return PA_ERR_INVALID_ARG;
        sum += rope->sections[a];
      }
      if (sum != rot / 2) return PA_ERR_INVALID_ARG;
    }
  }
  if (num_tokens == 0) return PA_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
  if (new_stride_tok <= 0 || new_stride_head <= 0 || kv_stride_page <= 0 || kv_stride_tok <= 0 || kv_stride_head <= 0)
    return PA_ERR_INVALID_ARG;
  if (q && (q_stride_tok <= 0 || q_stride_head <= 0 || q_out_stride_tok <= 0 || q_out_stride_head <= 0))
    return PA_ERR_INVALID_ARG;
  const int e = fp8 ? 1 : 2;
  auto at = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0; };
  if (rot > 0) {
    if (!rope->cos_sin || !positions || rope->cos_sin_stride < rot) return PA_ERR_INVALID_ARG;
    if (rope->num_axes > 1 && positions_stride < num_tokens) return PA_ERR_INVALID_ARG;
    if (!at(rope->cos_sin, 16) || rope->cos_sin_stride % 4 || !at(positions, 4)) return PA_ERR_UNSUPPORTED;
  }
  // 8-byte vectors of the new rows, 8-byte (bf16) or 4-byte (e4m3) stores into pages
  if (!at(k_new, 8) || !at(v_new, 8) || (new_stride_tok % 4) || (new_stride_head % 4)) return PA_ERR_UNSUPPORTED;
  if (q && (!at(q, 8) || !at(q_out, 8) || (q_stride_tok % 4) || (q_stride_head % 4) || (q_out_stride_tok % 4) ||
            (q_out_stride_head % 4)))
    return PA_ERR_UNSUPPORTED;
  if (!at(rope->q_norm, 8) || !at(rope->k_norm, 8) || !at(slot_mapping, 8)) return PA_ERR_UNSUPPORTED;
  if (!at(k_cache, 16) || !at(v_cache, 16) || (kv_stride_page * e) % 16 || (kv_stride_tok * e) % 16 ||
      (kv_stride_head * e) % 16)
    return PA_ERR_UNSUPPORTED;
  RopeParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.qo_stride_tok = q_out_stride_tok;
  p.qo_stride_head = q_out_stride_head;
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.new_stride_tok = new_stride_tok;
  p.new_stride_head = new_stride_head;
  p.positions = positions;
  p.positions_stride = positions_stride;
  p.cos_sin = rope->cos_sin;
  p.cos_sin_stride = rope->cos_sin_stride;
  p.q_norm = q ? static_cast<const uint16_t*>(rope->q_norm) : nullptr;
  p.k_norm = static_cast<const uint16_t*>(rope->k_norm);
  p.norm_eps = rope->norm_eps;
  p.norm_offset = rope->norm_offset;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.stride_page = kv_stride_page * e;
  p.stride_tok = kv_stride_tok * e;
  p.stride_head = kv_stride_head * e;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.ps_log2 = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(page_size)) : -1;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_tokens = num_tokens;
  p.half = rot / 2;
  p.interleaved = rope->interleaved;
  p.num_axes = rope->num_axes;
  p.max_position = rope->max_position;
  for (int a = 0, end = 0; a < 4; ++a) {
    if (a < rope->num_axes) end += rope->num_axes == 1 ? rot / 2 : rope->sections[a];
    p.axis_end[a] = end;
  }
  p.slot_mapping = slot_mapping;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err = static_cast<uint32_t*>(scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t r = head_dim == 64 ? launch<64>(p, fp8, st)
                        : head_dim == 128 ? launch<128>(p, fp8, st) : launch<256>(p, fp8, st);
  return r == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
