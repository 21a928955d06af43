// Device helpers shared by the key/value cache kernels.
#pragma once

#include "kv_internal.h"

namespace li8 {

typedef _Float16 kv_h2 __attribute__((ext_vector_type(2)));
typedef __bf16 kv_b2 __attribute__((ext_vector_type(2)));

// Batch and cache as the kernels take them (by value).
struct KvArgs {
    const int32_t *q_start, *kv_len, *table;
    int64_t table_stride;
    int table_width, tokens, max_q, max_kv;
    int8_t *k, *v;
    float *ks, *vs;
    int pages, heads, page_shift;
};

inline KvArgs kv_args(const li8_kv_batch &b, const li8_kv_cache &c)
{
    KvArgs a;
    a.q_start = b.q_start; a.kv_len = b.kv_len; a.table = b.table;
    a.table_stride = b.table_stride; a.table_width = b.table_width;
    a.tokens = b.tokens; a.max_q = b.max_q; a.max_kv = b.max_kv;
    a.k = c.k; a.v = c.v; a.ks = c.k_scale; a.vs = c.v_scale;
    a.pages = (int)c.pages; a.heads = c.heads;
    a.page_shift = __builtin_ctz((unsigned)c.page_size);
    return a;
}

__device__ __forceinline__ KvSeq kv_sequence_of(const KvArgs &a, int s)
{
    return kv_sequence(a.q_start[s], a.q_start[s + 1], a.kv_len[s], a.tokens, a.max_q, a.max_kv);
}

template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 v, float x[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (BF16) {
            x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
        } else {
            const kv_h2 h = __builtin_bit_cast(kv_h2, w[i]);
            x[2 * i] = (float)h.x;
            x[2 * i + 1] = (float)h.y;
        }
    }
}

// 8 floats to 16 bits, round to nearest even.
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float x[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (BF16) {
            kv_b2 b;
            b.x = (__bf16)x[2 * i];
            b.y = (__bf16)x[2 * i + 1];
            w[i] = __builtin_bit_cast(uint32_t, b);
        } else {
            kv_h2 h;
            h.x = (_Float16)x[2 * i];
            h.y = (_Float16)x[2 * i + 1];
            w[i] = __builtin_bit_cast(uint32_t, h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 load_u4(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }

// Values 8c .. 8c+7 of one head's row, rotated as of position pos >= 0.
// Products and sums are rounded one by one (the file is compiled without
// contraction), so that the stored codes are those of the definition bit for
// bit.
template <bool BF16>
__device__ __forceinline__ void load_rotated8(const uint16_t *row, int c, const KvRope &r, int pos,
                                              float x[8])
{
    unpack8<BF16>(load_u4(row + 8 * c), x);
    if (!r.cos || 4 * c >= r.half)
        return;
    const int64_t t = (int64_t)pos * r.half;
    if (r.interleaved) {
        const float4 cs = *reinterpret_cast<const float4 *>(r.cos + t + 4 * c);
        const float4 sn = *reinterpret_cast<const float4 *>(r.sin + t + 4 * c);
        const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cv[i] - b * sv[i];
            x[2 * i + 1] = b * cv[i] + a * sv[i];
        }
        return;
    }
    const int hc = r.half >> 3;              // chunks of each half
    const bool first = c < hc;
    const int i0 = 8 * (first ? c : c - hc);
    float y[8];
    unpack8<BF16>(load_u4(row + 8 * (first ? c + hc : c - hc)), y);
    float cv[8], sv[8];
    *reinterpret_cast<float4 *>(cv) = *reinterpret_cast<const float4 *>(r.cos + t + i0);
    *reinterpret_cast<float4 *>(cv + 4) = *reinterpret_cast<const float4 *>(r.cos + t + i0 + 4);
    *reinterpret_cast<float4 *>(sv) = *reinterpret_cast<const float4 *>(r.sin + t + i0);
    *reinterpret_cast<float4 *>(sv + 4) = *reinterpret_cast<const float4 *>(r.sin + t + i0 + 4);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float p = y[i] * sv[i];
        x[i] = x[i] * cv[i] + (first ? -p : p);
    }
}

} // namespace li8
