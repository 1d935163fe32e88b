// Internal declarations shared by the translation units of libpagedattn.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/pagedattn.h"

// Rows of every tile-routine MMA (M): (query token, head-in-group) pairs of one KV head.
#define PA_ROWS 128

namespace pa_detail {

// Records a failed CUDA call for pa_last_cuda_error(); returns PA_OK or PA_ERR_CUDA.
int32_t note_cuda(cudaError_t e);
// Shape support check (see pa_shape in pagedattn.h).
int32_t check_shape(const pa_shape* s);
// cu_seqlens_q / ctx_lens consistency: cu[0] == 0, non-decreasing, 0 <= n_q <= ctx.
int32_t check_step_meta(int32_t B, const int32_t* cu, const int32_t* ctx);

// paged_attention_step with its rows' log-sum-exps and decode rows' raw scores (attention.cu).
int32_t attention_step_stats(const void* q, const void* k_pool, const void* v_pool,
                             const int32_t* block_table, int32_t max_blocks,
                             const int32_t* cu_seqlens_q, const int32_t* ctx_lens, int32_t B,
                             int32_t T, int32_t max_ctx, const pa_work_item* items,
                             int32_t n_items, bool fp8, float k_scale, float v_scale,
                             void* workspace, size_t ws_bytes, void* out, float* lse,
                             float* scores, int64_t scores_ld, const pa_shape* shape,
                             int32_t* err_flag, cudaStream_t stream);

}  // namespace pa_detail
