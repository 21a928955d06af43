// Device helpers shared by the key/value cache kernels.
#pragma once

#include <type_traits>

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

// How a row is rotated: not, in pairs (i, i + half), in pairs (2i, 2i + 1).
enum { ROT_NONE = 0, ROT_HALVES = 1, ROT_PAIRS = 2 };

inline int rotation_of(const KvRope &r) { return !r.cos ? ROT_NONE : r.interleaved ? ROT_PAIRS : ROT_HALVES; }

// Values 8c .. 8c+7 of one head's row and what their rotation takes: loads
// without branches, so that a caller can have several rows in flight.  (A
// chunk past the rotated values loads itself and the table's first numbers.)
struct RowChunk {
    uint4 own, partner;
    float4 c[2], s[2];
};

template <int ROT>
__device__ __forceinline__ void fetch_row(RowChunk &w, const uint16_t *row, int c, const KvRope &r, int pos)
{
    w.own = load_u4(row + 8 * c);
    const int64_t t = (int64_t)pos * r.half;
    const bool turned = 4 * c < r.half;
    if constexpr (ROT == ROT_HALVES) {
        const int hc = r.half >> 3;              // chunks of each half
        w.partner = load_u4(row + 8 * (!turned ? c : c < hc ? c + hc : c - hc));
        const int i0 = !turned ? 0 : 8 * (c < hc ? c : c - hc);
        const float4 *pc = reinterpret_cast<const float4 *>(r.cos + t + i0);
        const float4 *ps = reinterpret_cast<const float4 *>(r.sin + t + i0);
        w.c[0] = pc[0]; w.c[1] = pc[1];
        w.s[0] = ps[0]; w.s[1] = ps[1];
    } else if constexpr (ROT == ROT_PAIRS) {
        w.c[0] = *reinterpret_cast<const float4 *>(r.cos + t + (turned ? 4 * c : 0));
        w.s[0] = *reinterpret_cast<const float4 *>(r.sin + t + (turned ? 4 * c : 0));
    }
}

// The rotated values.  Products and sums are rounded one by one (the files
// are compiled without contraction), so that the stored codes are those of
// the definition bit for bit.
template <bool BF16, int ROT>
__device__ __forceinline__ void rotate_row(const RowChunk &w, int c, const KvRope &r, float x[8])
{
    unpack8<BF16>(w.own, x);
    const bool turned = 4 * c < r.half;
    if constexpr (ROT == ROT_HALVES) {
        // chunk c of the first half takes -sin times its partner, of the
        // second +sin: the partner's sign bits carry it
        const uint32_t flip = c < (r.half >> 3) ? 0x80008000u : 0u;
        float y[8];
        unpack8<BF16>(make_uint4(w.partner.x ^ flip, w.partner.y ^ flip, w.partner.z ^ flip, w.partner.w ^ flip), y);
        const float cv[8] = {w.c[0].x, w.c[0].y, w.c[0].z, w.c[0].w, w.c[1].x, w.c[1].y, w.c[1].z, w.c[1].w};
        const float sv[8] = {w.s[0].x, w.s[0].y, w.s[0].z, w.s[0].w, w.s[1].x, w.s[1].y, w.s[1].z, w.s[1].w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float z = x[i] * cv[i] + y[i] * sv[i];
            x[i] = turned ? z : x[i];
        }
    } else if constexpr (ROT == ROT_PAIRS) {
        const float cv[4] = {w.c[0].x, w.c[0].y, w.c[0].z, w.c[0].w};
        const float sv[4] = {w.s[0].x, w.s[0].y, w.s[0].z, w.s[0].w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a = x[2 * i], b = x[2 * i + 1];
            const float za = a * cv[i] - b * sv[i], zb = b * cv[i] + a * sv[i];
            x[2 * i] = turned ? za : a;
            x[2 * i + 1] = turned ? zb : b;
        }
    }
}

// Runs f with the rotation's mode as a constant.
template <class F>
__device__ __forceinline__ void with_rotation(const KvRope &r, F f)
{
    if (!r.cos)
        f(std::integral_constant<int, ROT_NONE>());
    else if (r.interleaved)
        f(std::integral_constant<int, ROT_PAIRS>());
    else
        f(std::integral_constant<int, ROT_HALVES>());
}

} // namespace li8
