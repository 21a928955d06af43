// The epilogue variants of the few-token kernels (decode.hip,
// decode_split.hip): which weight rows a row group of 16 holds, and what the
// finishing wave does with them.  In that wave lane (kg, tok) = (lane / 16,
// lane % 16) holds token tok's results of rows 4 kg .. 4 kg + 3.
//
// EPI_GATED: rows 0..7 of a group are 8 features' gate rows and rows 8..15
// the same features' up rows, so the lanes of the wave's upper half hold the
// up values of the features whose gate values are 32 lanes below: one lane
// exchange joins them, and the groups are as many as for 2F plain rows.
#pragma once

#include "act_math.h"
#include "li8_internal.h"
#include "quant_math.h"

namespace li8 {

// Weight row of row i (0..15) of group rg < ceil(N / 16); rows past the last
// repeat it.
template <int EPI>
__device__ __forceinline__ int few_row(int rg, int i, int N)
{
    if constexpr (EPI == EPI_GATED) {
        const int F = N >> 1, f = min(rg * 8 + (i & 7), F - 1);
        return i < 8 ? f : F + f;
    } else {
        return min(rg * 16 + i, N - 1);
    }
}

// Bias and residual of a lane's four rows: loaded ahead of the products, raw
// (the conversions would wait for them), used by finish().  The loads are
// unconditional at clamped addresses but for the two uniform null tests.
template <int EPI>
struct FewOperands {
    uint16_t b[4], r[4];

    __device__ __forceinline__ void load(const EpiParams &p, int rg, int kg, int tok, int T, int N)
    {
#pragma unroll
        for (int j = 0; j < 4; j++)
            b[j] = r[j] = 0;
        if (p.bias)
#pragma unroll
            for (int j = 0; j < 4; j++)
                b[j] = p.bias[few_row<EPI>(rg, 4 * kg + j, N)];
        if constexpr (EPI == EPI_LINEAR)
            if (p.residual)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    r[j] = p.residual[(int64_t)min(tok, T - 1) * N + few_row<EPI>(rg, 4 * kg + j, N)];
    }

    // z: fl32(D * sW) of the lane's four rows.  Every lane of the wave calls.
    __device__ __forceinline__ void finish(const EpiParams &p, float (&z)[4], uint16_t *Y, int rg, int kg,
                                           int tok, int T, int N) const
    {
        // `n` of four values at element `at` of a row, 8 bytes if it may
        auto store = [](uint16_t *dst, const float (&v)[4], int n, bool vec) {
            const uint32_t h01 = pack_f16x2(v[0], v[1]), h23 = pack_f16x2(v[2], v[3]);
            if (vec && n >= 4) {
                *reinterpret_cast<uint2 *>(dst) = make_uint2(h01, h23);
            } else {
                const uint32_t w[2] = {h01, h23};
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (j < n)
                        dst[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            }
        };
#pragma unroll
        for (int j = 0; j < 4; j++)
            z[j] += h2f(b[j]);
        if constexpr (EPI == EPI_GATED) {
            const int F = N >> 1, f = rg * 8 + 4 * (kg & 1);
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const auto q = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, z[j]),
                                                                __builtin_bit_cast(uint32_t, z[j]), false, false);
                // (q[1]: every lane's value from the upper half, its up value)
                y[j] = value(p.act, z[j]) * __builtin_bit_cast(float, (uint32_t)q[1]);
            }
            if (tok >= T)
                return;
            if (p.pre)
                store(p.pre + (int64_t)tok * N + (kg < 2 ? f : F + f), z, F - f, (F & 3) == 0);
            if (kg < 2)
                store(Y + (int64_t)tok * F + f, y, F - f, (F & 3) == 0);
        } else {
            const int n = rg * 16 + 4 * kg;
            if (tok >= T)
                return;
            if (p.pre)
                store(p.pre + (int64_t)tok * N + n, z, N - n, (N & 3) == 0);
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; j++)
                y[j] = value(p.act, z[j]) + h2f(r[j]);
            store(Y + (int64_t)tok * N + n, y, N - n, (N & 3) == 0);
        }
    }

private:
    static __device__ __forceinline__ float value(const ActParams &a, float z)
    {
        return a.kind == 0 ? act_value<0>(z, a) : a.kind == 1 ? act_value<1>(z, a) : act_value<2>(z, a);
    }
};

template <>
struct FewOperands<EPI_PLAIN> {};

} // namespace li8
