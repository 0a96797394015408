// Verification of drafted tokens against the target's probabilities, and the draw
// of the token after them, from given random numbers.
//
// A request's drafts are tested in order, u q(x) < p(x) (products of two floats,
// exact in 64 bits); only the row where they end is read whole: the token there is
// the first v with  C_v > w C,  C_v the running sum of y = max(p - q, 0).  So a call
// reads one row of p (and of q) a request and is bound by HBM, or for few requests
// by the latency of its steps.
//
// Which v the sum crosses at depends on sums next to a border: in 32 bits a row of
// 10^5 entries has errors of the order of an entry.  The differences p - q and all
// sums are therefore pairs of floats (Knuth's two-sum, Dekker's pairs).  With u = 2^-24 the
// k-th addition of a sum begun at zero is off by at most (k + 5) u^2 of it, so a lane's 32 of
// a block by 700 u^2; a block's or eight entries' sum joins the others for 5 u^2, and where the
// running sum crosses is off by less than 3000 u^2, 2^-36, of the whole for 2^20 entries and
// one CTA a request.
// The card adds 64-bit numbers 64 times slower than floats: with the sums over lanes
// and parts in 64 bits the call of 64 rows of 131072 entries took 44 us.
//
// A request has a cluster of CTAs: every warp sums a contiguous part of the row, the
// parts' sums go to all CTAs over distributed shared memory, and the CTA whose warp
// holds the crossing sums that part again, a few entries a thread.
//
// Measured (one GB300, CUDA-graph replay): 64 requests of up to four drafts, 131072
// entries, 46 MB read on average (a request whose drafts are all accepted needs no q)
// 16.4 us (16.0 without blocks); 19.8 with one entry an instruction instead of two.  One request of 32000
// entries 6.2 us: what is left is latency (lengths, tokens, their probabilities, the
// row, two cluster barriers).
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pa.h"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;             // CTAs a request (portable cluster size)
constexpr int kUnit = 128;              // entries a warp takes at a time
constexpr int kBlock = 2048;            // entries whose sum a warp begins at zero
constexpr unsigned kAll = 0xffffffffu;

struct VerifyParams {
  const int32_t* tokens;
  const float* target;
  int64_t target_stride;
  const float* draft;          // null: drafts are certain
  int64_t draft_stride;
  int vocab;
  const int32_t* qsl;
  int batch, total_rows;
  const float* accept_u;
  const float* sample_u;
  int32_t* out;
  int64_t out_stride;
  int out_width;
  int32_t* num;
  uint32_t* err;
};

// A number held as two floats, hi + lo.
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float y) {
    const float s = __fadd_rn(hi, y);
    const float t = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(y, t)));
    hi = s;
  }
  __device__ __forceinline__ void add(const Pair& y) {
    add(y.hi);
    lo = __fadd_rn(lo, y.lo);
  }
  // lo at most half a step of hi: pairs then compare by hi first
  __device__ __forceinline__ Pair normal() const {
    Pair r;
    r.hi = __fadd_rn(hi, lo);
    r.lo = __fsub_rn(lo, __fsub_rn(r.hi, hi));
    return r;
  }
  __device__ __forceinline__ bool above(const Pair& y) const {
    const Pair a = normal(), b = y.normal();
    return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
  }
  __device__ __forceinline__ Pair from(unsigned m, int lane) const {
    Pair r;
    r.hi = __shfl_sync(m, hi, lane);
    r.lo = __shfl_sync(m, lo, lane);
    return r;
  }
  __device__ __forceinline__ Pair up(int n) const {
    Pair r;
    r.hi = __shfl_up_sync(kAll, hi, n);
    r.lo = __shfl_up_sync(kAll, lo, n);
    return r;
  }
  __device__ __forceinline__ Pair minus() const {
    Pair r;
    r.hi = -hi;
    r.lo = -lo;
    return r;
  }
};

// The running sum over the lanes, this one's included.
__device__ __forceinline__ Pair lane_sums(Pair x, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const Pair y = x.up(m);
    if (lane >= m) x.add(y);
  }
  return x;
}

// NaN and what is below 0 count as 0.
__device__ __forceinline__ float weight(float x) { return fmaxf(x, 0.f); }

// Two sums side by side, in packed arithmetic (each instruction does both).
struct Pairs {
  float2 hi = {0.f, 0.f}, lo = {0.f, 0.f};
  // adds max(p - q, 0) = max(p, q) - q (q >= 0): the difference and its rounding error, then both to the sum
  __device__ __forceinline__ void add(float2 p, float2 q) {
    const float2 m = make_float2(fmaxf(p.x, q.x), fmaxf(p.y, q.y));
    const float2 nq = make_float2(-q.x, -q.y);
    const float2 d = __fadd2_rn(m, nq);
    const float2 t = __fadd2_rn(d, make_float2(-m.x, -m.y));                                   // -q as it was taken
    const float2 e = __fadd2_rn(__fadd2_rn(m, sub(t, d)), sub(nq, t));
    const float2 s = __fadd2_rn(hi, d);
    const float2 u = sub(s, hi);
    lo = __fadd2_rn(lo, __fadd2_rn(__fadd2_rn(sub(hi, sub(s, u)), sub(d, u)), e));
    hi = s;
  }
  static __device__ __forceinline__ float2 sub(float2 a, float2 b) { return __fadd2_rn(a, make_float2(-b.x, -b.y)); }
  __device__ __forceinline__ Pair both() const {
    Pair r;
    r.hi = hi.x;
    r.lo = lo.x;
    Pair o;
    o.hi = hi.y;
    o.lo = lo.y;
    r.add(o);
    return r;
  }
};

// How a row's entries become weights y = max(p - q, 0).
struct Row {
  const float* p;
  const float* q;       // null: nothing is taken off
  int taken;            // the certain draft whose entry loses 1, or -1

  __device__ __forceinline__ float less(int v) const {
    return q != nullptr ? weight(__ldg(q + v)) : (v == taken ? 1.f : 0.f);
  }
  // a lane's sum of a warp's entries [v, v1), at most kBlock of them, v a multiple of kUnit; Q: there is a q
  template <bool Q>
  __device__ __forceinline__ Pair block(int v, int v1, int lane) const {
    Pairs s;
    if (((reinterpret_cast<uintptr_t>(p) | (Q ? reinterpret_cast<uintptr_t>(q) : 0)) & 15u) == 0) {
      constexpr int U = 4;               // 16 entries of p and q a lane in flight
      for (; v + U * kUnit <= v1; v += U * kUnit) {
        float4 a[U], c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = v + u * kUnit + lane * 4;
          a[u] = __ldg(reinterpret_cast<const float4*>(p + at));
          if constexpr (Q) c[u] = __ldg(reinterpret_cast<const float4*>(q + at));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if constexpr (Q) {
            x = make_float4(weight(c[u].x), weight(c[u].y), weight(c[u].z), weight(c[u].w));
          } else {
            const int at = taken - (v + u * kUnit + lane * 4);
            if (static_cast<unsigned>(at) < 4u)
              x = make_float4(at == 0 ? 1.f : 0.f, at == 1 ? 1.f : 0.f, at == 2 ? 1.f : 0.f, at == 3 ? 1.f : 0.f);
          }
          s.add(make_float2(a[u].x, a[u].y), make_float2(x.x, x.y));
          s.add(make_float2(a[u].z, a[u].w), make_float2(x.z, x.w));
        }
      }
    }
    for (v += lane; v < v1; v += 8 * 32) {
      float a[8], x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = v + 32 * u;
        a[u] = at < v1 ? __ldg(p + at) : 0.f;
        x[u] = at < v1 ? less(at) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; u += 2) s.add(make_float2(a[u], a[u + 1]), make_float2(x[u], x[u + 1]));
    }
    return s.both();
  }
  // and of any number: the lower part of a pair collects what the upper one rounds off, so its own rounding grows with
  // the additions it has seen (over 2000 of them, from one large entry on, a sum was off by 2^-28 of itself)
  template <bool Q>
  __device__ __forceinline__ Pair sum(int v, int v1, int lane) const {
    Pair s;
    for (; v < v1; v += kBlock) {
      s.add(block<Q>(v, min(v + kBlock, v1), lane));
      s = s.normal();
    }
    return s;
  }
  // entry v to a sum; whether it weighs anything
  __device__ __forceinline__ bool add(Pair& sum, int v) const {
    Pairs one;
    const float a = __ldg(p + v), x = less(v);
    one.add(make_float2(a, 0.f), make_float2(x, 0.f));
    sum.add(one.hi.x);
    sum.lo = __fadd_rn(sum.lo, one.lo.x);
    return a > x;
  }
};

__global__ void __launch_bounds__(kThreads, 4) verify_tokens_kernel(const VerifyParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ float2 s_part[2][kMaxCtas * kWarps];   // sums of the parts, all of the cluster
  __shared__ float2 s_scan[kWarps];
  __shared__ float2 s_rest;
  __shared__ int s_kept, s_mine, s_best, s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / C;
  const int qs = p.qsl[b];
  const int n = packed_rows(qs, p.qsl[b + 1]);
  int32_t* out = p.out + static_cast<int64_t>(b) * p.out_stride;
  // (the same in all threads of the cluster)
  if (n < 0 || n > p.out_width || qs < 0 || static_cast<int64_t>(qs) + n > p.total_rows) {
    if (p.err != nullptr && rank == 0 && tid == 0) atomicOr(p.err, kErrCapacity);
    return;
  }
  if (n == 0) {
    if (rank == 0) {
      for (int i = tid; i < p.out_width; i += kThreads) out[i] = -1;
      if (tid == 0) p.num[b] = 0;
    }
    return;
  }

  // (no CTA's shared memory is written before it runs: the wait is before the first write)
  cluster.barrier_arrive();

  // ---- the drafts, in order ------------------------------------------------
  if (warp == 0) {
    int kept = n - 1;
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
      const int i = i0 + lane;
      bool no = false;
      if (i < n - 1) {
        const int64_t r = qs + i;
        const int x = p.tokens[r + 1];
        const bool in = static_cast<unsigned>(x) < static_cast<unsigned>(p.vocab);
        const float pv = in ? weight(p.target[r * p.target_stride + x]) : 0.f;
        const float qv = p.draft == nullptr ? 1.f : in ? weight(p.draft[r * p.draft_stride + x]) : 0.f;
        no = !(static_cast<double>(p.accept_u[r]) * qv < static_cast<double>(pv));
      }
      const unsigned m = __ballot_sync(0xffffffffu, no);
      if (m != 0) {
        kept = i0 + __ffs(m) - 1;
        break;
      }
    }
    if (lane == 0) s_kept = kept;
  }
  __syncthreads();
  const int kept = s_kept;
  const bool rejected = kept < n - 1;
  const int64_t r = qs + kept;
  Row row;
  row.p = p.target + r * p.target_stride;
  row.q = rejected && p.draft != nullptr ? p.draft + r * p.draft_stride : nullptr;
  row.taken = rejected && p.draft == nullptr ? p.tokens[r + 1] : -1;
  if (rank == 0) {
    for (int i = tid; i < p.out_width; i += kThreads)
      if (i != kept) out[i] = i < kept ? p.tokens[qs + i + 1] : -1;
    if (tid == 0) p.num[b] = kept + 1;
  }

  // ---- the parts' sums -------------------------------------------------------
  const int units = (p.vocab + kUnit - 1) / kUnit;
  const int parts = C * kWarps;
  auto part_begin = [&](int w) { return static_cast<int>(static_cast<int64_t>(units) * w / parts) * kUnit; };
  for (int pass = 0; pass < 2; ++pass) {
    const int v0 = part_begin(rank * kWarps + warp), v1 = min(part_begin(rank * kWarps + warp + 1), p.vocab);
    Pair sum = row.q != nullptr ? row.sum<true>(v0, v1, lane) : row.sum<false>(v0, v1, lane);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      Pair y;
      y.hi = __shfl_xor_sync(kAll, sum.hi, m);
      y.lo = __shfl_xor_sync(kAll, sum.lo, m);
      sum.add(y);
    }
    sum = sum.from(kAll, 0);
    if (pass == 0) cluster.barrier_wait();
    if (lane < C) *cluster.map_shared_rank(&s_part[pass][rank * kWarps + warp], lane) = make_float2(sum.hi, sum.lo);
    cluster.sync();

    // the total, and the part whose running sum first exceeds w * total
    if (warp == 0) {
      constexpr int K = kMaxCtas * kWarps / 32;
      Pair part[K], own;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (lane * K + k < parts) {
          const float2 x = s_part[pass][lane * K + k];
          part[k].hi = x.x;
          part[k].lo = x.y;
        }
        own.add(part[k]);
      }
      const Pair incl = lane_sums(own, lane);
      const Pair total = incl.from(kAll, 31).normal();
      int mine = -1;
      Pair rest;
      if (total.hi > 0.f) {
        const float w = p.sample_u[b];
        Pair target;                     // w * total: the product of the upper parts exactly
        target.hi = __fmul_rn(w, total.hi);
        target.lo = __fmaf_rn(w, total.lo, __fmaf_rn(w, total.hi, -target.hi));
        Pair before = incl.up(1);
        if (lane == 0) before = Pair();
        int found = -1, last = -1;       // last: where rounding leaves the sum short of the target
        Pair left;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (part[k].hi > 0.f) {
            last = lane * K + k;
            Pair to = before;
            to.add(part[k]);
            if (found < 0 && to.above(target)) {
              found = last;
              left = target;
              left.add(before.minus());
            }
            before = to;
          }
        }
        const unsigned m = __ballot_sync(kAll, found >= 0);
        if (m != 0) {
          mine = __shfl_sync(kAll, found, __ffs(m) - 1);
          rest = left.from(kAll, __ffs(m) - 1);
        } else {
          mine = __reduce_max_sync(kAll, last);
          rest = total;
        }
      }
      if (lane == 0) {
        s_mine = mine;
        s_rest = make_float2(rest.hi, rest.lo);
        s_best = 0x7fffffff;
        s_last = -1;
      }
    }
    __syncthreads();
    if (s_mine >= 0 || (row.q == nullptr && row.taken < 0)) break;      // found, or nothing to draw from
    row.q = nullptr;                                                    // p <= q everywhere: from p itself
    row.taken = -1;
  }
  const int mine = s_mine;
  if (mine < 0) {
    if (rank == 0 && tid == 0) out[kept] = -1;
    return;
  }
  if (mine / kWarps != rank) return;

  // ---- the entry, within the part: some consecutive ones a thread ---------------
  Pair rest;
  rest.hi = s_rest.x;
  rest.lo = s_rest.y;
  const int v0 = part_begin(mine), v1 = min(part_begin(mine + 1), p.vocab);
  const int per = (v1 - v0 + kThreads - 1) / kThreads;
  const int a0 = min(v0 + tid * per, v1), a1 = min(a0 + per, v1);
  Pair own;
  int last = -1;
  for (int v = a0; v < a1; v += 8) {       // (eight from zero, as a block's)
    Pair eight;
    const int v1 = min(v + 8, a1);
#pragma unroll 4
    for (int u = v; u < v1; ++u)
      if (row.add(eight, u)) last = u;
    own.add(eight);
    own = own.normal();
  }
  const Pair incl = lane_sums(own, lane);
  if (lane == 31) s_scan[warp] = make_float2(incl.hi, incl.lo);
  __syncthreads();
  Pair before = incl.up(1);
  if (lane == 0) before = Pair();
  for (int w = 0; w < warp; ++w) {
    Pair y;
    y.hi = s_scan[w].x;
    y.lo = s_scan[w].y;
    before.add(y);
  }
  Pair to = before;
  to.add(own);
  if (last >= 0) {
    atomicMax(&s_last, last);
    if (to.above(rest)) atomicMin(&s_best, tid);
  }
  __syncthreads();
  // the first thread whose running sum exceeds the rest; none (rounding): the last entry that weighs
  const int best = s_best;
  if (best == 0x7fffffff) {
    if (tid == 0) out[kept] = s_last;
  } else if (tid == best) {
    int pick = -1;
    rest.add(before.minus());              // what is left of it for this thread's entries
    for (int v = a0; v < a1 && pick < 0; v += 8) {
      rest = rest.normal();
      Pair eight;
      const int v1 = min(v + 8, a1);
      for (int u = v; u < v1; ++u) {
        if (row.add(eight, u) && eight.above(rest)) {
          pick = u;
          break;
        }
      }
      rest.add(eight.minus());
    }
    if (pick < 0) pick = last;
    out[kept] = pick;
  }
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_verify_tokens(const int32_t* tokens, const float* target_probs, int64_t target_stride,
                                      const float* draft_probs, int64_t draft_stride, int32_t vocab,
                                      const int32_t* query_start_loc, int32_t batch, int32_t total_rows,
                                      const float* accept_u, const float* sample_u, int32_t* out_tokens,
                                      int64_t out_stride, int32_t out_width, int32_t* num_tokens, void* scratch,
                                      void* stream) {
  using namespace pa;
  if (batch < 0 || total_rows < 0 || vocab <= 0 || out_width < 0) return PA_ERR_INVALID_ARG;
  if (vocab > (1 << 20)) return PA_ERR_UNSUPPORTED;
  if (batch == 0) return PA_OK;
  if (!query_start_loc || !sample_u || !num_tokens || (out_width > 0 && !out_tokens)) return PA_ERR_INVALID_ARG;
  if (total_rows > 0 && (!tokens || !target_probs || !accept_u)) return PA_ERR_INVALID_ARG;
  if (total_rows > 1 && (target_stride < vocab || (draft_probs && draft_stride < vocab))) return PA_ERR_INVALID_ARG;
  if (batch > 1 && out_stride < out_width) return PA_ERR_INVALID_ARG;
  auto off = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3u) != 0; };
  if (off(tokens) || off(target_probs) || off(draft_probs) || off(query_start_loc) || off(accept_u) || off(sample_u) ||
      off(out_tokens) || off(num_tokens) || off(scratch))
    return PA_ERR_UNSUPPORTED;
  VerifyParams p{};
  p.tokens = tokens;
  p.target = target_probs;
  p.target_stride = target_stride;
  p.draft = draft_probs;
  p.draft_stride = draft_stride;
  p.vocab = vocab;
  p.qsl = query_start_loc;
  p.batch = batch;
  p.total_rows = total_rows;
  p.accept_u = accept_u;
  p.sample_u = sample_u;
  p.out = out_tokens;
  p.out_stride = out_stride;
  p.out_width = out_width;
  p.num = num_tokens;
  p.err = static_cast<uint32_t*>(scratch);
  // CTAs a request: up to eight while the call is about one wave of CTAs (four an SM) and each
  // still has 2048 entries
  int ctas = kMaxCtas;
  while (ctas > 1 && (static_cast<int64_t>(ctas) * batch > 608 || static_cast<int64_t>(ctas) * 2048 > vocab)) ctas /= 2;
  if (static_cast<int64_t>(ctas) * batch > INT32_MAX) return PA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * batch));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_tokens_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
