// Host side of the C ABI declared in include/llm_int8_kv.h: argument checks
// and kernel launches.  No allocation, no host sync.
#include <algorithm>

#include "kv_internal.h"

using namespace li8;

namespace {

constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;
constexpr float kMaxScale = 1.0e29f;     // below it the kernels' log2(e) times the scale is finite
constexpr int32_t kMaxKeys = 1 << 30;   // positions and a step past them stay below 2^31

bool off_by(const void *p, uintptr_t align) { return ((uintptr_t)p & (align - 1)) != 0; }

li8_status from_hip(hipError_t e) { return e == hipSuccess ? LI8_OK : LI8_ERR_HIP; }

// Sizes alone: what the plan and the workspace query need.
li8_status check_sizes(const li8_kv_batch *b, const li8_kv_cache *c)
{
    if (!b || !c)
        return LI8_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128)
        return LI8_ERR_SHAPE;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return LI8_ERR_SHAPE;
    if (c->heads < 1 || c->heads > 65535 || c->pages < 0 || c->pages > kMaxGrid)
        return LI8_ERR_SHAPE;
    if (b->seqs < 0 || b->tokens < 0 || b->max_q < 0 || b->max_kv < 0 || b->max_kv > kMaxKeys ||
        b->table_width < 0 ||
        b->table_stride < b->table_width)
        return LI8_ERR_SHAPE;
    if (b->max_kv > (int64_t)b->table_width * c->page_size)
        return LI8_ERR_SHAPE;
    // with pages none of which exists there is nothing the kernels could
    // read in a missing page's place
    if (b->max_kv > 0 && c->pages == 0)
        return LI8_ERR_SHAPE;
    return LI8_OK;
}

bool empty(const li8_kv_batch *b) { return b->seqs == 0 || b->tokens == 0 || b->max_q == 0; }

li8_status check_pointers(const li8_kv_batch *b, const li8_kv_cache *c)
{
    if (!b->q_start || !b->kv_len)
        return LI8_ERR_INVALID_ARG;
    if (off_by(b->q_start, 4) || off_by(b->kv_len, 4) || off_by(b->table, 4))
        return LI8_ERR_ALIGN;
    if (b->max_kv > 0 && (!b->table || !c->k || !c->v || !c->k_scale || !c->v_scale))
        return LI8_ERR_INVALID_ARG;
    if (off_by(c->k, 16) || off_by(c->v, 16) || off_by(c->k_scale, 4) || off_by(c->v_scale, 4))
        return LI8_ERR_ALIGN;
    return LI8_OK;
}

li8_status check_tokens(const void *p, int64_t stride, int64_t heads, int64_t dim)
{
    if (!p)
        return LI8_ERR_INVALID_ARG;
    if (off_by(p, 16) || stride % 8 != 0)
        return LI8_ERR_ALIGN;
    if (stride < heads * dim || stride > ((int64_t)1 << 31))
        return LI8_ERR_SHAPE;
    return LI8_OK;
}

li8_status check_rope(const li8_rope *r, const li8_kv_batch *b, const li8_kv_cache *c, KvRope *out)
{
    *out = KvRope{nullptr, nullptr, 0, 0};
    if (!r)
        return LI8_OK;
    if (r->dims <= 0 || r->dims % 16 != 0 || r->dims > c->head_dim || r->rows < b->max_kv)
        return LI8_ERR_SHAPE;
    if (r->interleaved != 0 && r->interleaved != 1)
        return LI8_ERR_INVALID_ARG;
    if (b->max_kv == 0)
        return LI8_OK;   // every position is out of range: nothing is rotated
    if (!r->cos || !r->sin)
        return LI8_ERR_INVALID_ARG;
    if (off_by(r->cos, 16) || off_by(r->sin, 16))
        return LI8_ERR_ALIGN;
    *out = KvRope{r->cos, r->sin, r->dims / 2, r->interleaved};
    return LI8_OK;
}

bool bad_dtype(li8_dtype d) { return d != LI8_F16 && d != LI8_BF16; }

// Query heads and the grid of the attention.
li8_status check_heads(const li8_kv_batch *b, const li8_kv_cache *c, int32_t q_heads, int32_t causal,
                       int32_t window)
{
    if (q_heads < 1 || q_heads > (1 << 20) || q_heads % c->heads != 0)
        return LI8_ERR_SHAPE;
    if (window < 0 || (causal != 0 && causal != 1))
        return LI8_ERR_INVALID_ARG;
    const int64_t rows = std::min(b->max_q, b->tokens), group = q_heads / c->heads;
    if (rows * group > kMaxGrid)
        return LI8_ERR_SHAPE;
    // (256 columns and work-items for a workgroup at least: with more, no plan
    // fits, and the plan's own products need not be looked at)
    if ((double)b->seqs * c->heads * ((rows * group + 255) / 256) * 256 > kKvMaxItems)
        return LI8_ERR_SHAPE;
    const KvPlan p = kv_plan(*b, *c, q_heads, causal != 0, window);
    if (kv_attention_items(*b, *c, p) > kKvMaxItems)
        return LI8_ERR_SHAPE;
    return LI8_OK;
}

#define LI8_TRY(call)                    \
    do {                                 \
        const li8_status try_st = (call); \
        if (try_st != LI8_OK)            \
            return try_st;               \
    } while (0)

} // namespace

extern "C" {

li8_status int8_kv_append(const void *K, int64_t k_stride, const void *V, int64_t v_stride,
                          li8_dtype dtype, const li8_rope *rope, const li8_kv_batch *batch,
                          const li8_kv_cache *cache, hipStream_t stream)
{
    LI8_TRY(check_sizes(batch, cache));
    if (bad_dtype(dtype))
        return LI8_ERR_INVALID_ARG;
    KvRope r;
    LI8_TRY(check_rope(rope, batch, cache, &r));
    if (empty(batch) || batch->max_kv == 0)
        return LI8_OK;
    LI8_TRY(check_pointers(batch, cache));
    LI8_TRY(check_tokens(K, k_stride, cache->heads, cache->head_dim));
    LI8_TRY(check_tokens(V, v_stride, cache->heads, cache->head_dim));
    if (kv_append_items(*batch, *cache) > kKvMaxItems)
        return LI8_ERR_SHAPE;
    return from_hip(launch_kv_append(KvTokens{static_cast<const uint16_t *>(K), k_stride},
                                     KvTokens{static_cast<const uint16_t *>(V), v_stride},
                                     dtype == LI8_BF16, r, *batch, *cache, stream));
}

li8_status int8_kv_read(const li8_kv_cache *cache, const li8_kv_batch *batch, li8_dtype dtype,
                        void *K, int64_t k_stride, void *V, int64_t v_stride, hipStream_t stream)
{
    LI8_TRY(check_sizes(batch, cache));
    if (bad_dtype(dtype))
        return LI8_ERR_INVALID_ARG;
    if (empty(batch))
        return LI8_OK;
    LI8_TRY(check_pointers(batch, cache));
    LI8_TRY(check_tokens(K, k_stride, cache->heads, cache->head_dim));
    LI8_TRY(check_tokens(V, v_stride, cache->heads, cache->head_dim));
    if (kv_read_items(*batch) > kKvMaxItems)
        return LI8_ERR_SHAPE;
    return from_hip(launch_kv_read(*cache, *batch, dtype == LI8_BF16, static_cast<uint16_t *>(K),
                                   k_stride, static_cast<uint16_t *>(V), v_stride, stream));
}

size_t int8_kv_attention_workspace_bytes(const li8_kv_batch *batch, const li8_kv_cache *cache,
                                         int32_t q_heads)
{
    if (check_sizes(batch, cache) != LI8_OK || check_heads(batch, cache, q_heads, 1, 0) != LI8_OK)
        return 0;
    return kv_workspace(*batch, *cache, q_heads);
}

li8_status int8_kv_attention_plan(const li8_kv_batch *batch, const li8_kv_cache *cache,
                                  int32_t q_heads, int32_t causal, int32_t window, int32_t *path,
                                  int32_t *splits)
{
    LI8_TRY(check_sizes(batch, cache));
    LI8_TRY(check_heads(batch, cache, q_heads, causal, window));
    if (!path || !splits)
        return LI8_ERR_INVALID_ARG;
    const KvPlan p = kv_plan(*batch, *cache, q_heads, causal != 0, window);
    *path = p.path;
    *splits = p.splits;
    return LI8_OK;
}

li8_status int8_kv_attention(const void *Q, int64_t q_stride, li8_dtype dtype, int32_t q_heads,
                             float scale, const li8_rope *rope, int32_t causal, int32_t window,
                             const li8_kv_batch *batch, const li8_kv_cache *cache, void *O,
                             int64_t o_stride, float *lse, void *workspace,
                             size_t workspace_bytes, hipStream_t stream)
{
    LI8_TRY(check_sizes(batch, cache));
    LI8_TRY(check_heads(batch, cache, q_heads, causal, window));
    if (bad_dtype(dtype) || !(scale >= 0.0f && scale < kMaxScale))   // (NaN is refused too)
        return LI8_ERR_INVALID_ARG;
    KvRope r;
    LI8_TRY(check_rope(rope, batch, cache, &r));
    if (empty(batch))
        return LI8_OK;
    LI8_TRY(check_pointers(batch, cache));
    LI8_TRY(check_tokens(Q, q_stride, q_heads, cache->head_dim));
    LI8_TRY(check_tokens(O, o_stride, q_heads, cache->head_dim));
    if (O == Q)   // (workgroups that share a row's keys read its query at different times)
        return LI8_ERR_INVALID_ARG;
    if (off_by(lse, 4) || off_by(workspace, 16))
        return LI8_ERR_ALIGN;
    const size_t need = kv_workspace(*batch, *cache, q_heads);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return LI8_ERR_WORKSPACE;
    return from_hip(launch_kv_attention(KvTokens{static_cast<const uint16_t *>(Q), q_stride},
                                        dtype == LI8_BF16, q_heads, scale, r, causal != 0, window,
                                        *batch, *cache, static_cast<uint16_t *>(O), o_stride, lse,
                                        static_cast<char *>(workspace), stream));
}

} // extern "C"
