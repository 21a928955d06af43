// Host side of the C ABI declared in include/llm_int8_ffn.h and llm_int8_ffn_plan.h:
// argument checks and kernel launches.  No allocation, no host sync.
#include <math.h>

#include "li8_internal.h"
#include "llm_int8_ffn.h"
#include "llm_int8_ffn_plan.h"

using namespace li8;

namespace {

bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }

li8_status from_hip(hipError_t e) { return e == hipSuccess ? LI8_OK : LI8_ERR_HIP; }

bool known_act(int32_t act) { return act >= LI8_ACT_NONE && act <= LI8_ACT_GELU_TANH; }

// A forward call's shape; N: rows of the weight (2F for a pair).  Grids stay below
// 2^32 work-items: 512 threads a tile of 256 x 128 at least.  Tiles of 64 x 128 are as
// many where T <= 64; past that they are taken only while a few rounds of the compute
// units hold them (two of them cost 0.66 of a round, half a 256x256 tile 0.5).
li8_status forward_shape(int64_t T, int64_t K, int64_t N)
{
    const li8_status st = check_shape(T, K, N);
    return st == LI8_OK && ((T + 255) / 256) * ((N + 127) / 128) >= (int64_t)1 << 23 ? LI8_ERR_SHAPE : st;
}

li8_status forward(const void *X, const int8_t *Wq, const float *sW, float threshold, int64_t T, int64_t K,
                   int64_t N, const void *bias, int32_t act, const void *residual, void *Y, void *pre, bool gated,
                   void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    li8_status st = check_shape(T, K, N);
    if (st != LI8_OK)
        return st;
    if (isnan(threshold) || threshold < 0.0f || !known_act(act))
        return LI8_ERR_INVALID_ARG;
    if (T == 0 || N == 0)
        return LI8_OK;
    if (forward_shape(T, K, N) != LI8_OK)
        return LI8_ERR_SHAPE;
    if ((K > 0 && (!X || !Wq)) || !sW || !Y)
        return LI8_ERR_INVALID_ARG;
    for (const void *p : {X, (const void *)Wq, (const void *)sW, bias, residual, (const void *)Y, (const void *)pre,
                          (const void *)workspace})
        if (misaligned(p))
            return LI8_ERR_ALIGN;
    const size_t need = llm_int8_linear_workspace_bytes(T, K, N);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return LI8_ERR_WORKSPACE;
    const EpiParams epi{static_cast<const uint16_t *>(bias), static_cast<const uint16_t *>(residual),
                        static_cast<uint16_t *>(pre), act_params(act), gated};
    const uint16_t *x = static_cast<const uint16_t *>(X);
    uint16_t *y = static_cast<uint16_t *>(Y);
    char *ws = static_cast<char *>(workspace);
    const uint16_t thr = threshold_magnitude(threshold);
    if (decode_shape(T, K))
        return from_hip(launch_decode_epi(x, Wq, sW, thr, T, K, N, y, epi, stream));
    if (split_shape(T, K))
        return from_hip(launch_split_fused(x, Wq, sW, nullptr, thr, T, K, N, y, ws, stream, &epi));
    const WsLayout L = ws_layout(T, K, N);
    const hipError_t e = launch_prepare(x, Wq, nullptr, thr, T, K, N, ws, L, stream, nullptr,
                                        GatherSkip{kFoldMin, epi_plan(T, K, N, gated).fold});
    if (e != hipSuccess)
        return LI8_ERR_HIP;
    return from_hip(launch_gemm_epi(Wq, sW, T, K, N, y, ws, L, epi, stream));
}

li8_status backward_shape(int64_t T, int64_t K, int64_t N)
{
    const li8_status st = check_shape(T, K, N);
    return st == LI8_OK && (N > kMaxGradN || T > kMaxGradT) ? LI8_ERR_SHAPE : st;
}

li8_status backward(const void *dY, const void *pre, int32_t act, const int8_t *Wq, const float *sW, int64_t T,
                    int64_t K, int64_t N, void *dX, void *grad_pre, float *dbias, bool gated, void *workspace,
                    size_t workspace_bytes, hipStream_t stream)
{
    li8_status st = backward_shape(T, K, N);
    if (st != LI8_OK)
        return st;
    if (!known_act(act))
        return LI8_ERR_INVALID_ARG;
    if (T > 0 && N > 0 && (!dY || !sW || (K > 0 && !Wq) || ((gated || act != LI8_ACT_NONE) && !pre)))
        return LI8_ERR_INVALID_ARG;
    if (T > 0 && K > 0 && !dX)
        return LI8_ERR_INVALID_ARG;
    for (const void *p : {dY, pre, (const void *)Wq, (const void *)sW, (const void *)dX, (const void *)grad_pre,
                          (const void *)dbias, (const void *)workspace})
        if (misaligned(p))
            return LI8_ERR_ALIGN;
    const size_t need = llm_int8_backward_workspace_bytes(T, K, N);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return LI8_ERR_WORKSPACE;
    if (N == 0 ? T == 0 || K == 0 : T == 0 && !dbias)   // nothing to write
        return LI8_OK;
    return from_hip(launch_backward(static_cast<const uint16_t *>(dY),
                                    gated || act != LI8_ACT_NONE ? static_cast<const uint16_t *>(pre) : nullptr,
                                    act_params(act), gated, Wq, sW, T, K, N, static_cast<uint16_t *>(dX),
                                    static_cast<uint16_t *>(grad_pre), dbias, static_cast<char *>(workspace), stream));
}

// Rows of a pair's weight, or a number that no check passes.
int64_t pair_rows(int64_t F) { return F < 0 || F >= ((int64_t)1 << 30) ? -1 : 2 * F; }

} // namespace

extern "C" {

li8_status llm_int8_linear_epilogue(const void *X, const int8_t *Wq, const float *sW, float threshold, int64_t T,
                                    int64_t K, int64_t N, const void *bias, int32_t act, const void *residual,
                                    void *Y, void *pre, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return forward(X, Wq, sW, threshold, T, K, N, bias, act, residual, Y, pre, false, workspace, workspace_bytes,
                   stream);
}

li8_status llm_int8_gated_linear(const void *X, const int8_t *Wq, const float *sW, float threshold, int64_t T,
                                 int64_t K, int64_t F, const void *bias, int32_t act, void *H, void *pre,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return forward(X, Wq, sW, threshold, T, K, pair_rows(F), bias, act, nullptr, H, pre, true, workspace,
                   workspace_bytes, stream);
}

li8_status llm_int8_epilogue_plan(int64_t T, int64_t K, int64_t N, int32_t gated, li8_epilogue_plan *plan)
{
    const li8_status st = forward_shape(T, K, N);
    if (st != LI8_OK)
        return st;
    if (!plan || (gated && N % 2))
        return LI8_ERR_INVALID_ARG;
    *plan = li8_epilogue_plan{LI8_PATH_EMPTY, 0, 0, 0, 0, 1, 1};
    if (T == 0 || N == 0)
        return LI8_OK;
    const bool few = decode_shape(T, K);
    if (few || split_shape(T, K)) {
        plan->path = few ? LI8_PATH_FEW_TOKENS : LI8_PATH_FEW_TOKENS_SPLIT;
        plan->tile_m = (int32_t)T;
        plan->tile_n = 16;
        return LI8_OK;
    }
    const GemmPlan p = epi_plan(T, K, N, gated != 0);
    *plan = li8_epilogue_plan{LI8_PATH_TILED, p.bm, p.bn, 0, 0, p.ranges, p.two ? 2 : 1};
    if (p.fold > kFoldMin) {
        plan->fold_lo = kFoldMin;
        plan->fold_hi = p.fold;
    }
    return LI8_OK;
}

size_t llm_int8_backward_workspace_bytes(int64_t T, int64_t K, int64_t N)
{
    if (backward_shape(T, K, N) != LI8_OK || T == 0 || N == 0)
        return 0;
    return backward_layout(T, K, N).total;
}

li8_status llm_int8_backward_plan(int64_t T, int64_t K, int64_t N, int32_t gated, li8_backward_plan *plan)
{
    const li8_status st = backward_shape(T, K, N);
    if (st != LI8_OK)
        return st;
    if (!plan || (gated && N % 2))
        return LI8_ERR_INVALID_ARG;
    *plan = li8_backward_plan{LI8_BACKWARD_EMPTY, 0, 1, 0, 0, 1};
    if (T == 0 || N == 0)
        return LI8_OK;
    const BackwardPlan p = backward_plan(T, K, N);
    if (p.few && K > 0) {
        *plan = li8_backward_plan{LI8_BACKWARD_FEW, p.bm, p.splits, 0, 0, 1};
        return LI8_OK;
    }
    const int64_t F = gated ? N / 2 : N;
    const RowPlan r = row_plan(F);
    *plan = li8_backward_plan{K > 0 ? LI8_BACKWARD_TILED : LI8_BACKWARD_ROWS, K > 0 ? p.bm : 0, K > 0 ? p.splits : 1,
                              r.threads, r.rounds, col_strips(T, F)};
    return LI8_OK;
}

li8_status llm_int8_linear_backward(const void *dY, const void *pre, int32_t act, const int8_t *Wq, const float *sW,
                                    int64_t T, int64_t K, int64_t N, void *dX, void *grad_pre, float *dbias,
                                    void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return backward(dY, pre, act, Wq, sW, T, K, N, dX, grad_pre, dbias, false, workspace, workspace_bytes, stream);
}

li8_status llm_int8_gated_backward(const void *dH, const void *pre, int32_t act, const int8_t *Wq, const float *sW,
                                   int64_t T, int64_t K, int64_t F, void *dX, void *grad_pre, float *dbias,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return backward(dH, pre, act, Wq, sW, T, K, pair_rows(F), dX, grad_pre, dbias, true, workspace, workspace_bytes,
                    stream);
}

} // extern "C"
