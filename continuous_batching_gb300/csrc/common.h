// Internal declarations shared by the translation units of libpagedattn.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/pagedattn.h"

// Rows of every tile-routine MMA (M): (query token, head-in-group) pairs of one KV head.
#define PA_ROWS 128

// Most rows (query tokens times heads of a group) of a sequence that the default reads from the codes. Where the
// GPU is full the two ways meet at about 60 rows (8 sequences of 4,000 keys, 32 / 8 heads of 128: 40 us against
// 69 with 32 rows, 77 against 70 with 64; 32 of 3,000 keys, 8 / 8 heads: 110 against 159, 206 against 160); a
// single sequence is faster read from the codes up to 250 rows, but the choice may not depend on the batch.
#define PA_Q4_DIRECT_ROWS 48

namespace pa_detail {

// Keys of a split of a row read from the codes, by its sequence's context alone. A split is the work of two warps:
// short ones where there are few, so that a single sequence spreads over the GPU, and longer ones where
// what a split costs beyond its keys (its start, its result written and read once more) would add up.
// Multiples of 32. (64 sequences of median 2,048 keys / 12 of 700 to 6,000 / one of 16,001: 72.8 / 13.7 / 20.5 us; with 512
// keys up to 32,768 78.4 / 13.7 / 15.2, half of each length 80.9 / 12.7 / 15.2, 640 up to 6,144 71.0 / 15.4 / 20.5. At the
// borders, 1 / 8 / 32 sequences of 32 / 8 heads, caches cold, with the shorter split and, a key further, with the longer
// one: 6,144 keys 20 / 29 / 75 and 24 / 34 / 75 us; 12,288 24 / 50 / 125 and 28 / 42 / 126; 32,768 30 / 95 / 276 and 42 / 106 / 287: a
// longer split costs where sequences are few, with one exception.)
__host__ __device__ constexpr int64_t q4_split_keys(int32_t ctx) {
    return ctx <= 6144 ? 512 : ctx <= 12288 ? 768 : ctx <= 32768 ? 1024 : 2048;
}
// The longest context of one split.
constexpr int64_t q4_one_split() { return 512; }
// The longest context: the keys that a warp looks up ahead of a split's, up to 3,000 behind its first, are counted
// in 32 bits.
constexpr int32_t kQ4MaxCtx = INT32_MAX - 4096;
// Most splits of any context up to max_ctx.
inline int64_t q4_max_splits(int64_t max_ctx) {
    const auto n = [](int64_t c) { return c <= 0 ? 1 : (c + q4_split_keys(int32_t(c)) - 1) / q4_split_keys(int32_t(c)); };
    int64_t most = n(max_ctx);
    for (const int64_t c : {6144, 12288, 32768})                // the last context of every length
        if (max_ctx > c && n(c) > most) most = n(c);
    return most;
}

// Rows of a tile read from the codes, 8 or 16, by the plan's sizes. A row's bits do not depend on it. 16 where sequences
// bring several tokens, so that they share a tile; 8 where a tile would mostly hold one token's rows: where there are
// no more rows than sequences, and where the step's chunks account for the rest. (32 / 8 heads of 128, contexts of
// 1,000 to 8,000, caches cold, tiles of 8 / 16 rows: 64 single tokens 91 / 138 us; 32, a prompt's last 5 and a chunk of
// 512 108 / 136; 32 times 4 drafted tokens and a chunk 136 / 127; 64 / 8 heads, 32 times 2 tokens 261 / 95.)
inline int32_t q4_tile_rows(int32_t g, const pa_q4_plan& p) {
    return p.direct_rows > 8 && (g > 8 || (p.T > p.B && p.n_chunk == 0)) ? 16 : 8;
}

// Where the parts of a plan's words begin (see pa_q4_plan).
struct Q4Words {
    int64_t direct, lists, fold, chunk, expand, table, total;
};
inline Q4Words q4_words(const pa_q4_plan& p) {
    constexpr int64_t item = sizeof(pa_work_item) / 4;
    Q4Words w;
    w.direct = 0;
    w.lists = w.direct + item * p.n_direct;
    w.fold = w.lists + (p.n_direct > 0 ? PA_PLAN_CTAS + 1 : 0);
    w.chunk = w.fold + p.n_fold;
    w.expand = w.chunk + item * p.n_chunk;
    w.table = w.expand + 2 * int64_t(p.n_expand);
    w.total = w.table + int64_t(p.n_chunk > 0 ? p.B : 0) * p.expand_cols;
    return w;
}
// PA_OK, or what is wrong with a plan's sizes.
int32_t check_q4_plan(const pa_shape* shape, const pa_q4_plan& p);

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

// paged_attention_step over the contexts that a 4-bit step has expanded (attention.cu), blocks of 128 keys: K in bf16, V
// in f16 where v16 [num_blocks][num_kv_heads] is 1, in bf16 where it is 0. partials: as the workspace of
// paged_attention_step, or NULL where no single token is among the rows.
int32_t attention_step_expanded(const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_table, int32_t max_blocks,
                                const int32_t* cu_seqlens_q, const int32_t* ctx_lens, int32_t B,
                                int32_t T, int32_t max_ctx, const uint8_t* v16,
                                const pa_work_item* items, int32_t n_items, void* partials, void* out, const pa_shape* shape,
                                int32_t* err_flag, cudaStream_t stream);

}  // namespace pa_detail
