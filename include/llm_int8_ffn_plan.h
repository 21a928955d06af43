/*
 * llm_int8_ffn_plan.h - which kernels the feed-forward operators
 * (llm_int8_ffn.h) run at a shape.  Introspection for tests and benchmarks, as
 * llm_int8_plan is for llm_int8_linear: sizes alone decide, nothing is enqueued,
 * and no result depends on it beyond the order of fp32 sums.
 *
 * N is the number of the weight's rows, 2F for a pair (gated != 0, N even).
 * Both return LI8_ERR_SHAPE for a shape that the operators refuse and
 * LI8_ERR_INVALID_ARG for a null pointer or a pair of odd N.
 */
#ifndef LLM_INT8_FFN_PLAN_H
#define LLM_INT8_FFN_PLAN_H

#include "llm_int8_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * llm_int8_linear_epilogue, llm_int8_gated_linear:
 *   path            an LI8_PATH_* of llm_int8.h;
 *   tile_m, tile_n  tokens and weight rows of a workgroup's tile (few tokens: T, 16);
 *   fold_lo, _hi    a call of fold_lo < n <= fold_hi outlier columns copies their
 *                   codes out of the stages of the weight; else they are gathered
 *                   (both 0: always gathered, or read by index);
 *   ranges          of K, in workgroups of their own whose sums a second launch adds
 *                   on tiles of 32 x 64 (1: none);
 *   per_cu          workgroups that share a compute unit (2: tiles of 64 x 128 that
 *                   are more than the compute units).
 */
typedef struct li8_epilogue_plan {
    int32_t path, tile_m, tile_n, fold_lo, fold_hi, ranges, per_cu;
} li8_epilogue_plan;

li8_status llm_int8_epilogue_plan(int64_t T, int64_t K, int64_t N, int32_t gated,
                                  li8_epilogue_plan *plan);

/*
 * llm_int8_linear_backward, llm_int8_gated_backward:
 *   path         LI8_BACKWARD_EMPTY  no weight rows or no tokens: zeros at most;
 *                LI8_BACKWARD_FEW    one kernel from dY to sums of dX;
 *                LI8_BACKWARD_TILED  dZ row by row, then the tiled product;
 *                LI8_BACKWARD_ROWS   K = 0, dZ alone;
 *   tile         rows of a tile of dX (its columns are 256; 0 without a product);
 *   ranges       of the weight's rows, whose sums a last launch adds (1: none);
 *   row_threads  threads that form a row of dZ (64 or 512; 0 on the path of few);
 *   row_rounds   rounds of eight features a thread that stay in registers (0: rows
 *                of any length, formed twice);
 *   strips       of the tokens for dbias, whose sums the last launch adds (1: none).
 */
enum { LI8_BACKWARD_EMPTY = 0, LI8_BACKWARD_FEW = 1, LI8_BACKWARD_TILED = 2, LI8_BACKWARD_ROWS = 3 };
typedef struct li8_backward_plan {
    int32_t path, tile, ranges, row_threads, row_rounds, strips;
} li8_backward_plan;

li8_status llm_int8_backward_plan(int64_t T, int64_t K, int64_t N, int32_t gated,
                                  li8_backward_plan *plan);

#ifdef __cplusplus
}
#endif

#endif /* LLM_INT8_FFN_PLAN_H */
