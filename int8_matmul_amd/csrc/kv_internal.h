// Internal declarations of the int8 key/value cache (include/llm_int8_kv.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "li8_internal.h"
#include "llm_int8_kv.h"

namespace li8 {

// One sequence of a batch as the kernels see it.  Every number comes from
// device memory that the host has not looked at, so each is brought into the
// range that the tensors have: whatever q_start and kv_len hold, q0 .. q0+n-1
// are rows of the packed tensors and positions below len have a table entry.
struct KvSeq {
    int q0, n;   // first row, rows
    int len;     // tokens
    int begin;   // position of row q0: len - n (negative: more rows than tokens)
};

__host__ __device__ inline int kv_clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

__host__ __device__ inline KvSeq kv_sequence(int start, int end, int kv_len, int tokens, int max_q,
                                             int max_kv)
{
    KvSeq q;
    q.q0 = kv_clamp(start, 0, tokens);
    q.n = kv_clamp(end, q.q0, tokens) - q.q0;
    q.len = kv_clamp(kv_len, 0, max_kv);
    q.begin = q.len - q.n;             // (before the cut: row q0 keeps its position)
    q.n = q.n < max_q ? q.n : max_q;
    return q;
}

// Keys that a block of rows at positions first .. last reaches: [lo, hi).
// The steps of a block count from base, lo rounded down to 32.
struct KvSpan {
    int lo, hi, base;
};

__host__ __device__ inline KvSpan kv_span(int first, int last, int len, bool causal, int window)
{
    KvSpan s;
    s.hi = causal && last + 1 < len ? last + 1 : len;
    const int64_t lo = window > 0 ? (int64_t)first + 1 - window : 0;
    s.lo = lo < 0 ? 0 : (int)lo;       // first < 2^31, window >= 1: fits
    s.hi = s.hi < s.lo ? s.lo : s.hi;  // (nothing is seen)
    s.base = s.lo & ~31;
    return s;
}

constexpr int kKvCols = 16;        // query columns of a few-column workgroup, or twice as many

// `parts` workgroups share all blocks' keys (0: one workgroup for each block).
struct KvPlan {
    int path;       // LI8_KV_*
    int cols;       // query columns of a workgroup
    int blocks;     // column blocks of the longest chunk
    int used;       // columns in use in the fullest block
    int splits;     // most parts of a block
    int parts;
};
KvPlan kv_plan(const li8_kv_batch &b, const li8_kv_cache &c, int q_heads, bool causal, int window);
size_t kv_workspace(const li8_kv_batch &b, const li8_kv_cache &c, int q_heads);

// A rotation table, or cos == nullptr for none.
struct KvRope {
    const float *cos, *sin;
    int half;        // pairs of a row
    int interleaved;
};

struct KvTokens {    // strided rows of 16-bit values
    const uint16_t *p;
    int64_t stride;
};

// Work-items of a call's largest launch along x (as numbers that no sizes
// overflow): past 2^32 - 1 the runtime refuses the launch, so the checks refuse
// the call.
constexpr double kKvMaxItems = 4294967295.0;
double kv_append_items(const li8_kv_batch &b, const li8_kv_cache &c);
double kv_read_items(const li8_kv_batch &b);
double kv_attention_items(const li8_kv_batch &b, const li8_kv_cache &c, const KvPlan &p);

hipError_t launch_kv_append(KvTokens K, KvTokens V, bool bf16, KvRope rope, const li8_kv_batch &b,
                            const li8_kv_cache &c, hipStream_t s);
hipError_t launch_kv_read(const li8_kv_cache &c, const li8_kv_batch &b, bool bf16, uint16_t *K,
                          int64_t ks, uint16_t *V, int64_t vs, hipStream_t s);
hipError_t launch_kv_attention(KvTokens Q, bool bf16, int q_heads, float scale, KvRope rope,
                               bool causal, int window, const li8_kv_batch &b,
                               const li8_kv_cache &c, uint16_t *O, int64_t os, float *lse,
                               char *ws, hipStream_t s);

} // namespace li8
