// Block tables, slot maps and positions of a step, from the requests' lengths.
//
// The pool's free pages are a stack S: free_pages[0 .. count), then the pages of
// the requests that end in this step.  With o_b the running sum of the pages the
// requests before b need, the k-th page request b is given is S[top - 1 - o_b - k].
// Everything follows from three prefix sums over the requests (new tokens, pages
// needed, pages returned), so no thread waits for another request's turn.
//
// A call moves kilobytes: what bounds it is the launch and two trips to memory
// (the lengths, then the tables).  So it is one kernel whose CTAs (one, or a
// cluster of eight where there are many tokens) each make all prefix sums for
// themselves in shared memory and then share tokens and pages; a thread finds the
// request of four consecutive tokens by bisection.  The counts and lengths are
// written behind a cluster barrier, because they may lie where the inputs do.
//
// Measured (one GB300, CUDA-graph replay): 4 requests of one token 4.1 us (an empty
// launch is about 2.5), 250 requests with 40 prompts, 10214 tokens, 8.9 us; there a CTA
// takes 26 us of searches for all tokens, so clusters of 4 / 2 / 1 take 13.7 / 19 / 30.
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pa.h"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kMaxRequests = 8192;
constexpr uint32_t kErrNoPages = PA_DEVICE_NO_PAGES;

struct TablesParams {
  const int32_t* ctx;
  const int32_t* fresh;
  int batch, page_size;
  int ps_log2;                 // log2(page_size) where it is a power of two, else -1
  const int32_t* held;
  int32_t* held_out;
  int32_t* free_pages;
  int free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  int num_pages;
  int32_t* block_table;
  int64_t bt_stride;
  int max_pages;
  int32_t* seq_lens;
  int32_t* qsl;
  int64_t* slots;
  int32_t* positions;
  int max_tokens;
  uint32_t* err;
};

// The last i with off[i] <= x (off ascending, off[0] = 0 <= x < off[n]).
__device__ __forceinline__ int find(const int* off, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Sums stop at 2^30, which no limit of the call reaches: such a step is refused.
constexpr int kFull = 1 << 30;
__device__ __forceinline__ int capped(int a, int b) {
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), static_cast<unsigned>(kFull)));
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) step_tables_kernel(const TablesParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int B = p.batch;
  extern __shared__ int smem[];
  int* tok_off = smem;                   // [B + 1] new tokens of the requests before
  int* need_off = tok_off + B + 1;       // [B + 1] pages they need
  int* back_off = need_off + B + 1;      // [B + 1] pages they return
  int* ctx_s = back_off + B + 1;
  int* held_s = ctx_s + B;
  __shared__ int s_sum[3][kThreads / 32];

  // ---- lengths and their prefix sums -------------------------------------
  const int count = *p.free_count;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  int sum[3] = {0, 0, 0};
  uint32_t bad = count < 0 || count > p.free_capacity ? kErrCapacity : 0u;
  for (int b = b0; b < b1; ++b) {
    const int ctx = p.ctx[b], fresh = p.fresh[b], held = p.held[b];
    ctx_s[b] = ctx;
    held_s[b] = held;
    int n = 0, need = 0, back = 0;
    if (held < 0 || held > p.max_pages || fresh < -1 || ctx < 0) {
      bad = kErrCapacity;
    } else if (fresh == -1) {
      back = held;
    } else {
      const long long len = static_cast<long long>(ctx) + fresh;
      if (ctx > static_cast<long long>(held) * p.page_size ||
          len > static_cast<long long>(p.max_pages) * p.page_size || fresh > p.max_tokens) {
        bad = kErrCapacity;
      } else {
        n = fresh;
        need = max(0, static_cast<int>((len + p.page_size - 1) / p.page_size) - held);
      }
    }
    tok_off[b] = n;
    need_off[b] = need;
    back_off[b] = back;
    sum[0] = capped(sum[0], n);
    sum[1] = capped(sum[1], need);
    sum[2] = capped(sum[2], back);
  }
  int incl[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
  for (int m = 1; m < 32; m <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int v = __shfl_up_sync(0xffffffffu, incl[k], m);
      if (lane >= m) incl[k] = capped(incl[k], v);
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) s_sum[k][warp] = incl[k];
  __syncthreads();
  int total[3] = {0, 0, 0};
  int run[3] = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int v = s_sum[k][w];
      if (w < warp) run[k] = capped(run[k], v);
      total[k] = capped(total[k], v);
    }
#pragma unroll
  for (int k = 0; k < 3; ++k) run[k] += incl[k] - sum[k];
  // (count and the sums are at most 2^30: 64 bits for their sum)
  const long long top_l = static_cast<long long>(count) + total[2];
  if (total[0] > p.max_tokens || max(total[1], total[2]) >= kFull || top_l - total[1] > p.free_capacity)
    bad |= kErrCapacity;
  if (total[1] > top_l) bad |= kErrNoPages;
  bad = __syncthreads_or(bad & kErrCapacity) ? kErrCapacity : (bad & kErrNoPages);   // (the rest is the same in all threads)
  const bool ok = bad == 0;
  if (ok) {
    // lengths in place become the sums before them (all fit: they are at most the totals checked above)
    for (int b = b0; b < b1; ++b) {
      const int n = tok_off[b], need = need_off[b], back = back_off[b];
      tok_off[b] = run[0];
      need_off[b] = run[1];
      back_off[b] = run[2];
      run[0] += n;
      run[1] += need;
      run[2] += back;
    }
    if (tid == 0) {
      tok_off[B] = total[0];
      need_off[B] = total[1];
      back_off[B] = total[2];
    }
  } else if (tid == 0 && cluster.block_rank() == 0 && p.err != nullptr) {
    atomicOr(p.err, bad);
  }
  // this CTA has read the lengths and counts; behind the wait all have
  cluster.barrier_arrive();
  __syncthreads();

  const int gt = static_cast<int>(cluster.block_rank()) * kThreads + tid;
  const int stride = static_cast<int>(cluster.num_blocks()) * kThreads;
  const int tokens = ok ? total[0] : 0;
  if (ok) {
    const int need = total[1];
    const int top = static_cast<int>(top_l);
    // where entry `at` of the stack lies: what ended requests held is in their rows, which this call does not write
    auto stack = [&](int at) -> const int32_t* {
      if (at < count) return p.free_pages + at;
      const int e = at - count;
      const int b = find(back_off, B, e);
      return p.block_table + static_cast<int64_t>(b) * p.bt_stride + (e - back_off[b]);
    };
    // four consecutive tokens a thread: one search, and mostly one page
    constexpr int U = 4;
    for (int t0 = gt * U; t0 < tokens; t0 += stride * U) {
      int b = find(tok_off, B, t0);
      const int32_t* where[U];
      int pos[U], rest[U];
      int last_pg = -1, last_b = -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = min(t0 + u, tokens - 1);
        while (t >= tok_off[b + 1]) ++b;
        pos[u] = ctx_s[b] + (t - tok_off[b]);
        const int pg = p.ps_log2 >= 0 ? pos[u] >> p.ps_log2 : pos[u] / p.page_size;
        rest[u] = pos[u] - pg * p.page_size;
        if (u > 0 && pg == last_pg && b == last_b) {
          where[u] = where[u - 1];
        } else {
          where[u] = pg < held_s[b] ? p.block_table + static_cast<int64_t>(b) * p.bt_stride + pg
                                    : stack(top - 1 - (need_off[b] + pg - held_s[b]));
        }
        last_pg = pg;
        last_b = b;
      }
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) id[u] = *where[u];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + u >= tokens) break;
        const bool in = static_cast<unsigned>(id[u]) < static_cast<unsigned>(p.num_pages);
        if (!in && p.err != nullptr) atomicOr(p.err, kErrPageId);
        p.slots[t0 + u] = in ? static_cast<int64_t>(id[u]) * p.page_size + rest[u] : -1;
        p.positions[t0 + u] = pos[u];
      }
    }
    for (int k = gt; k < need; k += stride) {
      const int b = find(need_off, B, k);
      p.block_table[static_cast<int64_t>(b) * p.bt_stride + held_s[b] + (k - need_off[b])] = *stack(top - 1 - k);
    }
    // what is left of the returned pages goes behind the entries that stay (entries below `count` are only read)
    for (int at = count + gt; at < top - need; at += stride) p.free_pages[at] = *stack(at);
  }
  for (int t = tokens + gt; t < p.max_tokens; t += stride) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }

  cluster.barrier_wait();
  for (int b = gt; b < B; b += stride) {
    const int ctx = ctx_s[b], held = held_s[b];
    int len = ctx, now = held;
    if (ok) {
      const bool ended = p.fresh[b] == -1;
      const int n = tok_off[b + 1] - tok_off[b];
      len = ended ? 0 : ctx + n;
      now = ended ? 0 : held + (need_off[b + 1] - need_off[b]);
    }
    p.seq_lens[b] = len;
    p.held_out[b] = now;
  }
  for (int b = gt; b <= B; b += stride) p.qsl[b] = ok ? tok_off[b] : 0;
  if (gt == 0) *p.free_count_out = ok ? static_cast<int>(top_l - total[1]) : count;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_step_tables(const int32_t* context_lens, const int32_t* new_lens, int32_t batch,
                                    int32_t page_size, const int32_t* page_counts, int32_t* page_counts_out,
                                    int32_t* free_pages, int32_t free_capacity, const int32_t* free_count,
                                    int32_t* free_count_out, int32_t num_pages, int32_t* block_table,
                                    int64_t bt_stride, int32_t max_pages_per_seq, int32_t* seq_lens,
                                    int32_t* query_start_loc, int64_t* slots, int32_t* positions, int32_t max_tokens,
                                    void* scratch, void* stream) {
  using namespace pa;
  if (batch < 0 || page_size <= 0 || free_capacity < 0 || num_pages <= 0 || max_pages_per_seq < 0 || max_tokens < 0)
    return PA_ERR_INVALID_ARG;
  if (batch > kMaxRequests) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_pages_per_seq) * page_size > (int64_t{1} << 30)) return PA_ERR_UNSUPPORTED;
  // (a stack entry's index is at most free_capacity and the pages of max_tokens: 32 bits hold it)
  if (max_tokens > (1 << 29) || free_capacity > (1 << 30)) return PA_ERR_UNSUPPORTED;
  if (batch > 0 && (!context_lens || !new_lens || !page_counts || !page_counts_out || !seq_lens || !block_table))
    return PA_ERR_INVALID_ARG;
  if (!free_count || !free_count_out || !query_start_loc || (free_capacity > 0 && !free_pages) ||
      (max_tokens > 0 && (!slots || !positions)))
    return PA_ERR_INVALID_ARG;
  if (bt_stride < max_pages_per_seq && batch > 1) return PA_ERR_INVALID_ARG;
  auto off = [](const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) != 0; };
  if (off(context_lens, 4) || off(new_lens, 4) || off(page_counts, 4) || off(page_counts_out, 4) ||
      off(free_pages, 4) || off(free_count, 4) || off(free_count_out, 4) || off(block_table, 4) || off(seq_lens, 4) ||
      off(query_start_loc, 4) || off(slots, 8) || off(positions, 4) || off(scratch, 4))
    return PA_ERR_UNSUPPORTED;
  TablesParams p{};
  p.ctx = context_lens;
  p.fresh = new_lens;
  p.batch = batch;
  p.page_size = page_size;
  p.ps_log2 = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(page_size)) : -1;
  p.held = page_counts;
  p.held_out = page_counts_out;
  p.free_pages = free_pages;
  p.free_capacity = free_capacity;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.slots = slots;
  p.positions = positions;
  p.max_tokens = max_tokens;
  p.err = static_cast<uint32_t*>(scratch);
  // few requests and tokens: one small CTA, whose barriers are short; many: a cluster of eight
  const bool small = batch <= 128 && max_tokens <= 512;
  const int ctas = max_tokens + batch > 4096 ? 8 : 1;
  auto kern = small ? step_tables_kernel<128> : step_tables_kernel<512>;
  // (a kernel's limit is set to its most, and only by calls that need more than 48 KB)
  constexpr int kMaxSmem = (5 * kMaxRequests + 3) * 4;
  const size_t smem = static_cast<size_t>(5 * batch + 3) * 4;
  if (smem > 49152 - 512 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess)
    return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(small ? 128 : 512);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
