// Norm, rotate and append: the queries and keys of new tokens take a per-head
// RMS norm and their rotation on the way from the projection to q_out and the
// paged cache; the values go along unchanged.
//
// Per (token, head) row x of D elements, in fp32:
//   y = x * rsqrt(sum x^2 / D + eps) * (w + offset)            (where w is given)
//   (a, b) <- (a cos - b sin, b cos + a sin)                   per rotated pair
// and one rounding at the end, to bf16 or to e4m3(y / scale).
//
// Every byte is touched once (read q, k, v and the angles; write q_out and two
// slots): the floor is HBM's.  D / 8 lanes share a row; lane j holds the four
// pairs 4j .. 4j+3, i.e. two 4-element vectors: the two halves' when pairs lie
// rot_dim / 2 apart, neighbours when they are interleaved or do not rotate.  A
// pair's two elements are therefore always in one lane and the rotation needs
// no exchange; the norm needs log2(D / 8) shuffles.
//
// Measured (411 MB: 16381 tokens, 32 + 2 x 8 heads of 128, norms, three axes):
// 76.4 us, 5.4 TB/s, 79 % of the copy bandwidth.  With eight warps a token 85 us:
// half of its 547 warp instructions a lane were the token's own (slot, positions,
// angles, 64-bit addresses); one warp a token leaves 386.  Packed fp32 arithmetic
// and 32-bit byte strides took a fifth off before that (119 -> 93 us).  Slower: one
// persistent CTA loop with hoisted rows (120 us), the rows through a cp.async ring (141
// us), 16-byte vectors (101 us), rows prefetched into L2 (no change).  Nor does it pay to
// prefetch the angles of tokens further on: 512 / 1024 / 2432 / 4864 ahead 77.2 / 76.9 /
// 77.9 / 77.8 us, 8191 tokens of heads of 256 61 us for 54.1 without.
#include <algorithm>
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
constexpr int kWarps = kThreads / 32;

// Strides are in bytes and below 2^32: an address is one 32 x 32 + 64 bit product.
struct RopeParams {
  const uint8_t* q;
  uint8_t* q_out;
  const uint8_t* k_new;
  const uint8_t* v_new;
  uint32_t q_tok, q_head, qo_tok, qo_head, new_tok, new_head;
  const int32_t* positions;
  int64_t positions_stride;
  const float* cos_sin;
  uint32_t cos_sin_row;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  float norm_eps, norm_offset;
  uint8_t* k_cache;
  uint8_t* v_cache;
  uint32_t page_bytes, tok_bytes, head_bytes;
  int num_pages, page_size, ps_log2, num_q_heads, num_kv_heads, num_tokens;   // ps_log2: -1, no power of two
  int token_warps;       // warps per token: 1, 2, 4 or 8
  int half;              // rot_dim / 2
  int interleaved, num_axes, max_position;
  int axis_end[4];       // first pair behind each axis
  const int64_t* slot_mapping;
  float k_scale, v_scale;
  uint32_t* err;         // optional error word
};

__device__ __forceinline__ uint64_t offset(uint32_t i, uint32_t stride) { return static_cast<uint64_t>(i) * stride; }

// Two floats as one operand of the packed fp32 instructions: half as many issue
// slots as single ones.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 floats(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 bf16x2_floats(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t floats_bf16x2(F2 a) {
  const float2 f = floats(a);
  return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ uint32_t quant4(F2 lo, F2 hi, float scale) {
  const float2 a = floats(lo), b = floats(hi);
  const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a.x, scale), __fdiv_rn(a.y, scale)),
                                              __NV_SATFINITE, __NV_E4M3);
  const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(b.x, scale), __fdiv_rn(b.y, scale)),
                                              __NV_SATFINITE, __NV_E4M3);
  return l | (h << 16);
}

// A token takes `token_warps` warps (1, 2, 4 or 8 of the CTA's eight): what is worked
// out once a token (slot, positions, angles, addresses: half the instructions when
// eight warps each do it) is shared by more rows the fewer they are, and the rows
// run at the same time the more they are.  kQ query rows and kKv key or value rows
// per lane group are in flight at a time, the first ones' loads ahead of the token's
// slot and positions.
// CTAs an SM: four of bf16, which spill (bytes stored: heads of 64 and 128 40, 92 to 100
// where pairs are interleaved, of 256 136 and 104), three of e4m3, which hardly do.  us with
// three / four: 16381 tokens bf16 78.9 / 76.4, interleaved 77.5 / 78.6, e4m3 90.3 / 88.4; 8191
// tokens of heads of 256 58.1 / 54.2; 250 e4m3 tokens 3.8 / 4.0.
template <int D, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, FP8 ? 3 : 4) append_rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 8;                  // lanes per row
  constexpr int kQ = 4, kKv = 2;
  const int warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (kWarps / p.token_warps) + warp / p.token_warps;
  if (t >= p.num_tokens) return;
  const int lane = threadIdx.x % LPR;
  const int lead = (warp & (p.token_warps - 1)) * (32 / LPR);    // the warp's first row
  const int row = lead + (threadIdx.x & 31) / LPR;               // this lane's first row
  const int step = p.token_warps * (32 / LPR);                   // from a warp's rows to its next
  // this lane's two 4-element vectors of a row, as bytes of a bf16 row
  const bool turns = 4 * lane < p.half;
  const bool apart = turns && !INTERLEAVED;
  const uint32_t da = apart ? 8 * lane : 16 * lane;
  const uint32_t db = apart ? 2 * p.half + 8 * lane : 16 * lane + 8;
  const int nq = p.num_q_heads, nk = p.num_kv_heads;

  const uint8_t* q_src = p.q + offset(t, p.q_tok);
  const uint64_t new_at = offset(t, p.new_tok);
  uint2 qa[kQ], qb[kQ], na[kKv], nb[kKv];
  auto load_q = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int h = r0 + u * step;
      if (h < nq) {
        qa[u] = *reinterpret_cast<const uint2*>(q_src + da + offset(h, p.q_head));
        qb[u] = *reinterpret_cast<const uint2*>(q_src + db + offset(h, p.q_head));
      }
    }
  };
  auto load_kv = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kKv; ++u) {
      const int r = r0 + u * step;
      if (r < 2 * nk) {
        const uint8_t* x = (r < nk ? p.k_new : p.v_new) + new_at + offset(r < nk ? r : r - nk, p.new_head);
        na[u] = *reinterpret_cast<const uint2*>(x + da);
        nb[u] = *reinterpret_cast<const uint2*>(x + db);
      }
    }
  };
  load_q(row);
  load_kv(row);

  const int64_t slot = p.slot_mapping[t];
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
  if (slot < 0) return;                       // padding token
  const int64_t page = p.ps_log2 >= 0 ? slot >> p.ps_log2 : slot / p.page_size;
  if (page >= p.num_pages || bad) {           // outside the pool or the table: nothing written
    if (p.err != nullptr && (threadIdx.x & 31) == 0)
      atomicOr(p.err, page >= p.num_pages ? kErrPageId : PA_DEVICE_POSITION);
    return;
  }

  // the cosines and sines of this lane's four pairs
  float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turns) {
    const int pair = 4 * lane;
    auto at = [&](int i) {
      return i < p.axis_end[0] ? pos[0] : i < p.axis_end[1] ? pos[1] : i < p.axis_end[2] ? pos[2] : pos[3];
    };
    auto end = [&](int i) {
      return i < p.axis_end[0] ? p.axis_end[0] : i < p.axis_end[1] ? p.axis_end[1]
             : i < p.axis_end[2] ? p.axis_end[2] : p.axis_end[3];
    };
    const float* row = p.cos_sin + offset(at(pair), p.cos_sin_row) + pair;
    if (end(pair) >= pair + 4) {              // all on one axis
      cs = __ldg(reinterpret_cast<const float4*>(row));
      sn = __ldg(reinterpret_cast<const float4*>(row + p.half));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        row = p.cos_sin + offset(at(pair + e), p.cos_sin_row) + pair + e;
        (&cs.x)[e] = __ldg(row);
        (&sn.x)[e] = __ldg(row + p.half);
      }
    }
  }

  // norm (where the head kind has weights: x, y) and rotation of one row
  auto turn = [&](uint2 wa, uint2 wb, bool norm, uint2 x, uint2 y, F2 (&a)[2], F2 (&b)[2]) {
    a[0] = bf16x2_floats(wa.x), a[1] = bf16x2_floats(wa.y);
    b[0] = bf16x2_floats(wb.x), b[1] = bf16x2_floats(wb.y);
    if (norm) {
      const float2 s2 = floats(fma2(a[0], a[0], fma2(a[1], a[1], fma2(b[0], b[0], b[1] * b[1]))));
      float ss = s2.x + s2.y;
#pragma unroll
      for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float rs = rsqrtf(ss * (1.f / D) + p.norm_eps);
      const F2 r2 = f2(rs, rs), off = f2(rs * p.norm_offset, rs * p.norm_offset);   // rs (w + offset)
      a[0] = a[0] * fma2(r2, bf16x2_floats(x.x), off);
      a[1] = a[1] * fma2(r2, bf16x2_floats(x.y), off);
      b[0] = b[0] * fma2(r2, bf16x2_floats(y.x), off);
      b[1] = b[1] * fma2(r2, bf16x2_floats(y.y), off);
    }
    if (!turns) return;
    if constexpr (INTERLEAVED) {              // pairs (a0, a1), (a2, a3), (b0, b1), (b2, b3)
      auto one = [](F2 v, float c, float s) {
        const float2 f = floats(v);
        return fma2(v, f2(c, c), f2(f.y, f.x) * f2(-s, s));
      };
      a[0] = one(a[0], cs.x, sn.x);
      a[1] = one(a[1], cs.y, sn.y);
      b[0] = one(b[0], cs.z, sn.z);
      b[1] = one(b[1], cs.w, sn.w);
    } else {                                  // pairs (a_e, b_e)
      const F2 c[2] = {f2(cs.x, cs.y), f2(cs.z, cs.w)}, s[2] = {f2(sn.x, sn.y), f2(sn.z, sn.w)};
      const F2 n[2] = {f2(-sn.x, -sn.y), f2(-sn.z, -sn.w)};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const F2 v = a[i];
        a[i] = fma2(v, c[i], b[i] * n[i]);
        b[i] = fma2(b[i], c[i], v * s[i]);
      }
    }
  };
  auto weights = [&](const uint16_t* w, uint2& x, uint2& y) {
    if (w == nullptr) return;
    x = __ldg(reinterpret_cast<const uint2*>(w + da / 2));
    y = __ldg(reinterpret_cast<const uint2*>(w + db / 2));
  };
  uint2 x = make_uint2(0u, 0u), y = x;
  weights(p.q_norm, x, y);

  uint8_t* q_dst = p.q_out + offset(t, p.qo_tok);
  for (int r0 = 0; r0 + lead < nq; r0 += kQ * step) {
    if (r0 > 0) load_q(r0 + row);
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      if (r0 + u * step + lead >= nq) break;  // (the same for the warp: whole warps shuffle)
      const int h = r0 + u * step + row;
      F2 a[2], b[2];
      turn(qa[u], qb[u], p.q_norm != nullptr, x, y, a, b);
      if (h < nq) {
        *reinterpret_cast<uint2*>(q_dst + da + offset(h, p.qo_head)) =
            make_uint2(floats_bf16x2(a[0]), floats_bf16x2(a[1]));
        *reinterpret_cast<uint2*>(q_dst + db + offset(h, p.qo_head)) =
            make_uint2(floats_bf16x2(b[0]), floats_bf16x2(b[1]));
      }
    }
  }
  const uint64_t cell = offset(static_cast<uint32_t>(page), p.page_bytes) +
                        offset(static_cast<uint32_t>(slot - page * p.page_size), p.tok_bytes);
  weights(p.k_norm, x, y);
  for (int r0 = 0; r0 + lead < 2 * nk; r0 += kKv * step) {
    if (r0 > 0) load_kv(r0 + row);
#pragma unroll
    for (int u = 0; u < kKv; ++u) {
      if (r0 + u * step + lead >= 2 * nk) break;
      const int r = r0 + u * step + row;
      const bool k = r < nk;
      F2 a[2], b[2];
      // (a warp of values alone has nothing to turn)
      if (FP8 || r0 + u * step + lead < nk) turn(na[u], nb[u], p.k_norm != nullptr, x, y, a, b);
      if (r >= 2 * nk) continue;
      uint8_t* dst = (k ? p.k_cache : p.v_cache) + cell + offset(k ? r : r - nk, p.head_bytes);
      if constexpr (FP8) {
        if (!k) {                             // values go as they are
          a[0] = bf16x2_floats(na[u].x), a[1] = bf16x2_floats(na[u].y);
          b[0] = bf16x2_floats(nb[u].x), b[1] = bf16x2_floats(nb[u].y);
        }
        const float scale = k ? p.k_scale : p.v_scale;
        *reinterpret_cast<uint32_t*>(dst + da / 2) = quant4(a[0], a[1], scale);
        *reinterpret_cast<uint32_t*>(dst + db / 2) = quant4(b[0], b[1], scale);
      } else {
        if (k) {
          na[u] = make_uint2(floats_bf16x2(a[0]), floats_bf16x2(a[1]));
          nb[u] = make_uint2(floats_bf16x2(b[0]), floats_bf16x2(b[1]));
        }
        *reinterpret_cast<uint2*>(dst + da) = na[u];
        *reinterpret_cast<uint2*>(dst + db) = nb[u];
      }
    }
  }
}

template <int D>
cudaError_t launch(const RopeParams& p, bool fp8, cudaStream_t st) {
  auto kern = p.interleaved ? (fp8 ? append_rope_kernel<D, true, true> : append_rope_kernel<D, false, true>)
                            : (fp8 ? append_rope_kernel<D, true, false> : append_rope_kernel<D, false, false>);
  const int per_cta = kWarps / p.token_warps;
  kern<<<(p.num_tokens - 1) / per_cta + 1, kThreads, 0, st>>>(p);
  return cudaGetLastError();
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
  if (static_cast<int64_t>(num_q_heads) + 2 * static_cast<int64_t>(num_kv_heads) > (1 << 16)) return PA_ERR_UNSUPPORTED;
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
    int64_t sum = 0;
    for (int a = 0; a < rope->num_axes; ++a) {
      if (rope->sections[a] < 0) return PA_ERR_INVALID_ARG;
      sum += rope->sections[a];
    }
    if (sum != rot / 2 && !(rope->num_axes == 1 && sum == 0)) return PA_ERR_INVALID_ARG;
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
  if (!at(rope->q_norm, 8) || !at(rope->k_norm, 8) || !at(slot_mapping, 8) || !at(scratch, 4))
    return PA_ERR_UNSUPPORTED;
  if (!at(k_cache, 16) || !at(v_cache, 16) || (kv_stride_page * e) % 16 || (kv_stride_tok * e) % 16 ||
      (kv_stride_head * e) % 16)
    return PA_ERR_UNSUPPORTED;
  // strides below 2^32 bytes (a token's and a page's own; whole arrays may be larger)
  const int64_t widest = std::max({q ? std::max(std::max(q_stride_tok, q_stride_head),
                                                std::max(q_out_stride_tok, q_out_stride_head)) : int64_t{0},
                                   new_stride_tok, new_stride_head});
  if (widest > (UINT32_MAX >> 1) || std::max({kv_stride_page, kv_stride_tok, kv_stride_head}) > UINT32_MAX / e ||
      rope->cos_sin_stride > UINT32_MAX)
    return PA_ERR_UNSUPPORTED;
  RopeParams p{};
  p.q = static_cast<const uint8_t*>(q);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.k_new = static_cast<const uint8_t*>(k_new);
  p.v_new = static_cast<const uint8_t*>(v_new);
  if (q) {
    p.q_tok = static_cast<uint32_t>(q_stride_tok * 2);
    p.q_head = static_cast<uint32_t>(q_stride_head * 2);
    p.qo_tok = static_cast<uint32_t>(q_out_stride_tok * 2);
    p.qo_head = static_cast<uint32_t>(q_out_stride_head * 2);
  }
  p.new_tok = static_cast<uint32_t>(new_stride_tok * 2);
  p.new_head = static_cast<uint32_t>(new_stride_head * 2);
  p.positions = positions;
  p.positions_stride = positions_stride;
  p.cos_sin = rope->cos_sin;
  p.cos_sin_row = static_cast<uint32_t>(rope->cos_sin_stride);
  p.q_norm = q ? static_cast<const uint16_t*>(rope->q_norm) : nullptr;
  p.k_norm = static_cast<const uint16_t*>(rope->k_norm);
  p.norm_eps = rope->norm_eps;
  p.norm_offset = rope->norm_offset;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.page_bytes = static_cast<uint32_t>(kv_stride_page * e);
  p.tok_bytes = static_cast<uint32_t>(kv_stride_tok * e);
  p.head_bytes = static_cast<uint32_t>(kv_stride_head * e);
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.ps_log2 = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(page_size)) : -1;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.half = rot / 2;
  p.interleaved = rope->interleaved;
  p.num_axes = rope->num_axes;
  p.max_position = rot > 0 ? rope->max_position : 1;
  for (int a = 0, end = 0; a < 4; ++a) {
    if (a < rope->num_axes) end += rope->num_axes == 1 ? rot / 2 : rope->sections[a];
    p.axis_end[a] = end;
  }
  p.num_tokens = num_tokens;
  p.slot_mapping = slot_mapping;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err = static_cast<uint32_t*>(scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  // Warps per token: as many as leave the SMs no more than 32 warps each to run (us
  // for 8 / 4 / 2 / 1 warps, bf16: 300 tokens 3.8 / 4.2 / 6.1 / 10.0, 1200 tokens 10.6 /
  // 8.1 / 9.6 / 14.0, 2400 tokens 20.0 / 16.2 / 15.1 / 17.9, 4800 tokens 36.0 / 28.0 /
  // 26.3 / 25.5).
  p.token_warps = kWarps;
  while (p.token_warps > 1 && static_cast<int64_t>(num_tokens) * p.token_warps > static_cast<int64_t>(sms) * 32)
    p.token_warps /= 2;
  const cudaError_t r = head_dim == 64 ? launch<64>(p, fp8, st)
                        : head_dim == 128 ? launch<128>(p, fp8, st) : launch<256>(p, fp8, st);
  return r == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
