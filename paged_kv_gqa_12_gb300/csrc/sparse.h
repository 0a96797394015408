// Shared by page selection (select.cu) and sparse attention (sparse.cu): the
// checks of a sparse shape, the layout of its scratch workspace, and the map
// from a packed query row to its request and position.
#pragma once

#include <cstdint>

#include "pa.h"
#include "pa_internal.h"

namespace pa {

constexpr int kMaxTopPages = 4096;
constexpr int kMaxSparsePages = 65536;        // block-table width
constexpr int kScorePagesMin = 64;            // pages a score CTA covers at least
constexpr int64_t kScoreBytes = int64_t{256} << 20;   // scores held at a time (at least one row's)

// Pages per row of the score buffer: whole 32-page words.
inline int64_t score_pages(const pa_sparse_shape& s) {
  return (static_cast<int64_t>(s.max_pages_per_seq) + 31) / 32 * 32;
}
// Chunk maxima kept per (row, kv head).
inline int64_t score_chunks(const pa_sparse_shape& s) {
  return (score_pages(s) + kScorePagesMin - 1) / kScorePagesMin;
}

pa_status validate_sparse(const pa_sparse_shape& s);

// KV splits of each row in a call of `rows` query rows.
int sparse_splits(const pa_sparse_shape& s, int64_t rows);
// CTAs per kv head of the attention (16 heads each).
inline int sparse_head_groups(const pa_sparse_shape& s) {
  return (s.num_q_heads / s.num_kv_heads + 15) / 16;
}
int64_t sparse_partial_bytes(const pa_sparse_shape& s, int64_t partial_rows);
int64_t sparse_score_bytes(const pa_sparse_shape& s, int64_t score_rows);

// The checks every call of a plan makes before anything is enqueued.
pa_status check_sparse_call(const pa_sparse_plan_t* plan, const int32_t* block_table, int64_t bt_stride,
                            const int32_t* seq_lens, const int32_t* qsl, int32_t batch, int32_t total_q,
                            const void* scratch, int64_t scratch_bytes);

#ifdef __CUDACC__
// Where a packed query row belongs.
struct RowPlace {
  int b;        // request, or -1: a row behind the last request
  int pos;      // position in the sequence; -1: the request has no keys
  bool bad;     // length beyond the capacity, or more rows than tokens
};

// By a whole CTA of N threads (contains barriers).  query_start_loc is
// non-decreasing, so a row's request is the number of requests that end at or
// before it.
template <int N>
__device__ __forceinline__ RowPlace find_row(const int32_t* seq_lens, const int32_t* qsl, int batch, int row,
                                             int64_t max_len) {
  RowPlace r{-1, -1, false};
  int b = row;
  int L;
  if (qsl != nullptr) {
    b = 0;
    for (int base = 0; base < batch; base += N) {
      const int i = base + static_cast<int>(threadIdx.x);
      b += __syncthreads_count(i < batch && qsl[i + 1] <= row);
    }
    if (b >= batch) return r;
    const int begin = qsl[b], end = qsl[b + 1];
    L = seq_lens[b];
    r.b = b;
    r.bad = row < begin || L < 0 || L > max_len || end - begin > L;
    r.pos = L - (end - row);
    return r;
  }
  if (b >= batch) return r;
  L = seq_lens[b];
  r.b = b;
  r.bad = L < 0 || L > max_len;
  r.pos = L - 1;
  return r;
}
#endif

}  // namespace pa
