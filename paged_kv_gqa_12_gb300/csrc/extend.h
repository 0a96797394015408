// Extend (prefix-prefill) planning, shared between the C-ABI and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa.h"

namespace pa {

pa_status plan_extend(const pa_shape& s, int num_sms, pa_plan_t* out);

// Work items (32 bytes each) an extend call of this shape has room for.
int64_t extend_work_capacity(const pa_shape& s);

// Tensor map of an extend call's queries.
pa_status extend_q_map(CUtensorMap* map, const pa_shape& s, const void* q, int64_t q_stride_tok,
                       int64_t q_stride_head, int32_t total_q);

// Extend over a dense copy of the codes in the requests' pages, K as bf16 and V as f16 (page i of
// request b at copy page table[b * max_pages_per_seq + i] = b * max_pages_per_seq + i), with
// page_scales [copy page][Hkv] = (K scale, log2 of the V scale); a NaN of V is minus zero in the copy,
// and its page's entry of the table has the sign bit set: the scheduler and the attention
// kernel.  `work` holds the work list, `header` is a scratch header.
pa_status extend_over_copy(const pa_shape& s, const CUtensorMap& tmq, const void* k_copy, const void* v_copy,
                           const float2* page_scales, int32_t copy_pages, const int32_t* table,
                           const int32_t* seq_lens, const int32_t* query_start_loc, int32_t batch, int32_t total_q,
                           int32_t max_new, float scale, const float* sinks, void* out, int64_t out_stride_tok,
                           int64_t out_stride_head, float* lse, void* header, void* work, void* stream);

}  // namespace pa
