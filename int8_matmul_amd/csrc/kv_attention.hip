// Attention over the int8 key/value cache, for gfx950.
//
//   z[t] = scale (rotated q).(k code) k scale       over the keys a row sees
//   O    = sum_t exp(z[t]) v code v scale / sum_t exp(z[t])
//
// The query rows of one key/value head, tokens x heads of its group, are the
// columns of the products.  For a block of keys
//   S^T[key, col] = K Q^T    int8 MFMA: q is split into two int8 parts, a
//                            15-bit integer of its row's largest magnitude,
//                            q = f (128 qh + ql); the sums are exact
//   O^T[d, col]  += V^T P^T  fp16 MFMA: the codes are exact in fp16, the
//                            probabilities are rounded to it (11 bits)
// The transposed form leaves a column in the lanes that hold it as the next
// product's operand: with the keys of a step of 32 numbered so that lane
// group g has keys 4g..4g+3 and 16+4g..16+4g+3, the scores' accumulator
// registers are the probabilities' operand registers, and neither goes
// through LDS.
#include <float.h>

#include <algorithm>

#include "kv_device.h"

namespace li8 {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kNone = -1.0e30f;      // a running maximum over nothing yet
constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;
constexpr float kQMax = 16256.0f;      // 127 * 128: the largest 15-bit query integer
constexpr int kFewWaves = 4;

struct AttnArgs {
    KvTokens Q;
    KvRope rope;
    uint16_t *O;
    int64_t os;
    float *lse;
    float *part_o, *part_m;            // [item][split][used][D], [item][split][used]
    float scale;                       // scale * log2(e)
    int group, causal, window;
    int cols, blocks, used, splits, chunk;
};

// Where a workgroup's columns lie.
struct Block {
    KvSeq q;
    KvSpan span;
    int s, h, c0, nc;                  // sequence, head, first column, columns
};

__device__ __forceinline__ bool locate(const KvArgs &a, const AttnArgs &t, int item, int cols, Block &b)
{
    const int cb = item % t.blocks;
    const int sh = item / t.blocks;
    b.h = sh % a.heads;
    b.s = sh / a.heads;
    b.q = kv_sequence_of(a, b.s);
    const int64_t ncol = (int64_t)b.q.n * t.group;
    if ((int64_t)cb * cols >= ncol)
        return false;
    b.c0 = cb * cols;
    b.nc = (int)min((int64_t)cols, ncol - b.c0);
    b.span = kv_span(b.q.begin + b.c0 / t.group, b.q.begin + (b.c0 + b.nc - 1) / t.group, b.q.len,
                     t.causal != 0, t.window);
    return true;
}

// One row's 8 query values (a chunk of D) as two int8 parts; f is the
// factor of the row's integers, without the softmax scale.  The lanes of a
// row are D/8 neighbours.
template <int D>
__device__ __forceinline__ void split_query(const float x[8], uint2 &hi, uint2 &lo, float &f)
{
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++)
        m = fmaxf(m, fabsf(x[e]));
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1)
        m = fmaxf(m, __shfl_xor(m, o, 64));
    const float inv = m > 0.0f ? fminf(kQMax / m, FLT_MAX) : 0.0f;
    f = m * (1.0f / kQMax);
    uint32_t h[2] = {0, 0}, l[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const int qi = (int)fminf(fmaxf(rintf(x[e] * inv), -kQMax), kQMax);
        const int qh = (qi + 64) >> 7;   // -127 .. 127, and the rest -64 .. 63
        h[e >> 2] |= ((uint32_t)qh & 0xffu) << (8 * (e & 3));
        l[e >> 2] |= ((uint32_t)(qi - 128 * qh) & 0xffu) << (8 * (e & 3));
    }
    hi = make_uint2(h[0], h[1]);
    lo = make_uint2(l[0], l[1]);
}

// Codes of byte `byte` of two keys' words (already offset by 128: 0..255) as
// fp16: 0x6400 | u is 1024 + u, and 1024 + u - 1152 is the code, exactly.
template <int BYTE>
__device__ __forceinline__ uint32_t codes_f16(uint32_t a, uint32_t b)
{
    const uint32_t w = __builtin_amdgcn_perm(b, a, 0x0c000c00u | BYTE | ((4 + BYTE) << 16)) | 0x64006400u;
    const kv_h2 h = __builtin_bit_cast(kv_h2, w) - (kv_h2){(_Float16)1152.0f, (_Float16)1152.0f};
    return __builtin_bit_cast(uint32_t, h);
}

// Keys and values of a step of 32 keys, two tiles of 16.
template <int D>
struct Step {
    v4i k[2][D / 64];
    uint32_t v[8][D / 64];
    float ks[2], vs[2];
    bool ok[2];
};

template <int D>
__device__ __forceinline__ void load_step(Step<D> &st, const KvArgs &a, const int32_t *table, int h,
                                          int t0, int lo, int te, int lane)
{
    const int r = lane & 15, g = lane >> 4, page = 1 << a.page_shift;
#pragma unroll
    for (int tt = 0; tt < 2; tt++) {
        const int t = t0 + 16 * tt;
        const int pid = table[min(t >> a.page_shift, a.table_width - 1)];
        // a tile past the end, before the first key seen or in no page is
        // masked; page 0 is read in its place
        st.ok[tt] = (unsigned)pid < (unsigned)a.pages && t < te && t + 16 > lo;
        const int64_t ph = (int64_t)(st.ok[tt] ? pid : 0) * a.heads + h;
        const int64_t base = ((ph * D) << a.page_shift) + (t & (page - 1)) * D;
        const int8_t *kp = a.k + base;
        const int8_t *vp = a.v + base;
#pragma unroll
        for (int ks = 0; ks < D / 64; ks++)
            st.k[tt][ks] = *reinterpret_cast<const v4i *>(kp + r * D + 64 * ks + 16 * g);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int8_t *p = vp + (4 * g + j) * D + r * (D / 16);
            if constexpr (D == 128)
                *reinterpret_cast<uint2 *>(st.v[4 * tt + j]) = *reinterpret_cast<const uint2 *>(p);
            else
                st.v[4 * tt + j][0] = *reinterpret_cast<const uint32_t *>(p);
        }
        const float ksc = a.ks[ph], vsc = a.vs[ph];
        st.ks[tt] = st.ok[tt] ? ksc : 0.0f;
        st.vs[tt] = st.ok[tt] ? vsc : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// Few columns: 16 columns of one (sequence, head) and one split of its keys
// per workgroup; the 4 waves take the steps of 32 keys in turn and keep their
// own maximum, sum and O^T, merged through LDS at the end.
// ---------------------------------------------------------------------------
template <int D, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void k_kv_few(KvArgs a, AttnArgs t)
{
    constexpr int CPR = D / 8, NB = D / 16, KS = D / 64, LQ = D + 16, LO = D + 4;
    __shared__ __align__(16) char smem[kFewWaves * kKvCols * LO * 4];
    __shared__ float s_f[kKvCols], s_m[kFewWaves][kKvCols], s_l[kFewWaves][kKvCols];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sp = blockIdx.x % t.splits, item = blockIdx.x / t.splits;
    Block b;
    if (!locate(a, t, item, kKvCols, b))
        return;
    const int ts = b.span.base + sp * t.chunk;
    const int te = min(b.span.hi, ts + t.chunk);
    if (ts >= te && t.splits > 1)
        return;                        // (the merging kernel knows how many there are)
    const int qc = tid / CPR, cc = tid % CPR;   // column and chunk of the query and output phases

    if (qc < kKvCols) {
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, f;
        if (qc < b.nc) {
            const int c = b.c0 + qc, i = c / t.group, g = c - i * t.group;
            load_rotated8<BF16>(t.Q.p + (int64_t)(b.q.q0 + i) * t.Q.stride + (int64_t)(b.h * t.group + g) * D,
                                cc, t.rope, max(b.q.begin + i, 0), x);
        }
        uint2 hi, lo;
        split_query<D>(x, hi, lo, f);
        *reinterpret_cast<uint2 *>(smem + qc * LQ + 8 * cc) = hi;
        *reinterpret_cast<uint2 *>(smem + (kKvCols + qc) * LQ + 8 * cc) = lo;
        if (cc == 0)
            s_f[qc] = f * t.scale;
    }
    __syncthreads();
    const int col = lane & 15, g = lane >> 4;
    v4i qh[KS], ql[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
        qh[ks] = *reinterpret_cast<const v4i *>(smem + col * LQ + 64 * ks + 16 * g);
        ql[ks] = *reinterpret_cast<const v4i *>(smem + (kKvCols + col) * LQ + 64 * ks + 16 * g);
    }
    const float f = s_f[col];
    __syncthreads();                   // smem is used again below

    // keys this lane's column sees: [clo, chi)
    const int pos = b.q.begin + (b.c0 + col) / t.group;
    int chi = t.causal ? min(te, pos + 1) : te;
    const int clo = t.window > 0 ? max((int64_t)0, (int64_t)pos + 1 - t.window) : 0;
    if (col >= b.nc)
        chi = 0;
    const int32_t *table = a.table + (int64_t)b.s * a.table_stride;

    v4f acc[NB] = {};
    float m = kNone, l = 0.0f, vref = 0.0f;
    for (int t0 = ts + 32 * wid; t0 < te; t0 += 32 * kFewWaves) {
        Step<D> st;
        load_step<D>(st, a, table, b.h, t0, b.span.lo, te, lane);
        float z[8], zm = -INFINITY;
#pragma unroll
        for (int tt = 0; tt < 2; tt++) {
            v4i sh = {0, 0, 0, 0}, sl = {0, 0, 0, 0};
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                sh = __builtin_amdgcn_mfma_i32_16x16x64_i8(st.k[tt][ks], qh[ks], sh, 0, 0, 0);
                sl = __builtin_amdgcn_mfma_i32_16x16x64_i8(st.k[tt][ks], ql[ks], sl, 0, 0, 0);
            }
            const float fk = f * st.ks[tt];
            const int key = t0 + 16 * tt + 4 * g, hi = st.ok[tt] ? chi : 0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float v = (float)((sh[i] << 7) + sl[i]) * fk;
                z[4 * tt + i] = key + i < hi && key + i >= clo ? v : -INFINITY;
                zm = fmaxf(zm, z[4 * tt + i]);
            }
        }
        // The maximum is moved only when some score is 8 above it (in powers
        // of two): until then the probabilities stay below 2^8, and neither
        // O^T nor the sum has to be scaled.
        if (__any(zm > m + 8.0f)) {
            zm = fmaxf(zm, __shfl_xor(zm, 16, 64));
            zm = fmaxf(zm, __shfl_xor(zm, 32, 64));
            const float mn = fmaxf(m, zm), al = exp2f(m - mn);
#pragma unroll
            for (int n = 0; n < NB; n++)
                acc[n] *= al;
            l *= al;
            m = mn;
        }
        // Value scales relative to the largest so far, so that the operand
        // stays in fp16's range whatever the scales are.
        const float vm = fmaxf(st.vs[0], st.vs[1]);
        if (vm > vref) {
            const float al = vref / vm;
#pragma unroll
            for (int n = 0; n < NB; n++)
                acc[n] *= al;
            vref = vm;
        }
        const float vi = vref > 0.0f ? 1.0f / vref : 0.0f;
        v8h p;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const float pe = exp2f(z[e] - m);
            l += pe;
            p[e] = (_Float16)(pe * (st.vs[e >> 2] * vi));
        }
#pragma unroll
        for (int w = 0; w < KS; w++) {
            uint32_t u[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                u[j] = st.v[j][w] ^ 0x80808080u;
            v4u x0, x1, x2, x3;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x0[j] = codes_f16<0>(u[2 * j], u[2 * j + 1]);
                x1[j] = codes_f16<1>(u[2 * j], u[2 * j + 1]);
                x2[j] = codes_f16<2>(u[2 * j], u[2 * j + 1]);
                x3[j] = codes_f16<3>(u[2 * j], u[2 * j + 1]);
            }
            acc[4 * w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x0), p, acc[4 * w], 0, 0, 0);
            acc[4 * w + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x1), p, acc[4 * w + 1], 0, 0, 0);
            acc[4 * w + 2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x2), p, acc[4 * w + 2], 0, 0, 0);
            acc[4 * w + 3] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x3), p, acc[4 * w + 3], 0, 0, 0);
        }
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // Accumulator n of lane (col, g) holds O^T[(4g + i) NB + n][col], i < 4.
    float *so = reinterpret_cast<float *>(smem) + (wid * kKvCols + col) * LO;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int n = 0; n < NB; n += 4) {
            const v4f o = {acc[n][i] * vref, acc[n + 1][i] * vref, acc[n + 2][i] * vref, acc[n + 3][i] * vref};
            *reinterpret_cast<v4f *>(so + (4 * g + i) * NB + n) = o;
        }
    if (g == 0) {
        s_m[wid][col] = m;
        s_l[wid][col] = l;
    }
    __syncthreads();
    if (qc >= b.nc)
        return;
    float M = kNone, L = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kFewWaves; w++)
        M = fmaxf(M, s_m[w][qc]);
#pragma unroll
    for (int w = 0; w < kFewWaves; w++) {
        const float al = exp2f(s_m[w][qc] - M);
        const float *src = reinterpret_cast<const float *>(smem) + (w * kKvCols + qc) * LO + 8 * cc;
        L += s_l[w][qc] * al;
#pragma unroll
        for (int e = 0; e < 8; e++)
            o[e] += src[e] * al;
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++)
        o[e] *= inv;
    if (t.splits > 1) {
        const int64_t at = ((int64_t)blockIdx.x) * t.used + qc;
        float *po = t.part_o + at * D + 8 * cc;
        *reinterpret_cast<float4 *>(po) = make_float4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<float4 *>(po + 4) = make_float4(o[4], o[5], o[6], o[7]);
        if (cc == 0)
            t.part_m[at] = L > 0.0f ? M + log2f(L) : kNone;
        return;
    }
    const int c = b.c0 + qc, i = c / t.group, gq = c - i * t.group;
    const int64_t row = b.q.q0 + i;
    const int head = b.h * t.group + gq;
    *reinterpret_cast<uint4 *>(t.O + row * t.os + (int64_t)head * D + 8 * cc) = pack8<BF16>(o);
    if (t.lse && cc == 0)
        t.lse[row * (int64_t)(a.heads * t.group) + head] = L > 0.0f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

// ---------------------------------------------------------------------------
// Many columns: 32 columns per wave, kTileWaves waves; the workgroup walks
// its keys in steps of 64 that all waves read from LDS.  K stays int8 there
// (16 MFMAs 32x32x32 i8 per step and wave for the two query parts), V is
// turned into fp16 and transposed on its way in, once for all waves.
// ---------------------------------------------------------------------------
constexpr int kTileWaves = 8;
constexpr int kTileCols = 32 * kTileWaves;
constexpr int kTileKeys = 64;
constexpr float kFar = -12.0f;         // log2: value scales this far below the largest

typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v16f __attribute__((ext_vector_type(16)));

// 16-byte chunks of the LDS tiles are permuted within 128 bytes so that
// neither the fragment reads (32 rows, one chunk each) nor the writes of V
// (rows 4 apart) meet in a bank.
template <int D>
__device__ __forceinline__ int k_place(int row, int chunk)
{
    if constexpr (D == 128)
        return row * 128 + 16 * (chunk ^ (row & 7));
    return row * 64 + 16 * (chunk ^ ((row >> 1) & 3));
}

__device__ __forceinline__ int v_place(int d, int chunk) { return d * 128 + 16 * (chunk ^ ((d ^ (d >> 3)) & 7)); }

template <int D>
struct TileLds {
    static constexpr int K = kTileKeys * D, V = D * kTileKeys * 2;
    static constexpr int stage = K + V;
    static constexpr int q_row = D + 16;
    static constexpr int bytes = 2 * stage > 2 * kTileCols * q_row ? 2 * stage : 2 * kTileCols * q_row;
};

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kTileWaves, 2) void k_kv_tiled(KvArgs a, AttnArgs t, int pairs, int lanes)
{
    constexpr int NT = 64 * kTileWaves, CPR = D / 8, KS = D / 32, DB = D / 32;
    constexpr int NI = kTileKeys * D / 16 / NT > 0 ? kTileKeys * D / 16 / NT : 1;   // staging items of a thread
    constexpr int ITEMS = kTileKeys * D / 16;
    using L = TileLds<D>;
    __shared__ __align__(16) char smem[L::bytes];
    __shared__ float s_f[kTileCols];
    __shared__ __align__(16) float s_sc[2][4][4];   // [buffer][ks, 1/vs, log2 vs, vs][group of 16 keys]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Blocks of one (sequence, head) share its keys: all on 8 / lanes of the
    // XCDs (the hardware deals workgroups to the 8 XCDs in turn), the last
    // block, which sees the most keys, first.
    const int j = blockIdx.x / lanes, per = t.blocks * t.splits;
    const int pair = (j / per) * lanes + blockIdx.x % lanes;
    if (pair >= pairs)
        return;
    const int rest = j % per, sp = rest % t.splits;
    const int item = pair * t.blocks + (t.blocks - 1 - rest / t.splits);
    Block b;
    if (!locate(a, t, item, kTileCols, b))
        return;
    const int ts = b.span.base + sp * t.chunk;
    const int te = min(b.span.hi, ts + t.chunk);
    if (ts >= te && t.splits > 1)
        return;

#pragma unroll
    for (int k = 0; k < CPR / 2; k++) {
        const int it = tid + NT * k, qc = it / CPR, cc = it % CPR;
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, f;
        if (qc < b.nc) {
            const int c = b.c0 + qc, i = c / t.group, g = c - i * t.group;
            load_rotated8<BF16>(t.Q.p + (int64_t)(b.q.q0 + i) * t.Q.stride + (int64_t)(b.h * t.group + g) * D,
                                cc, t.rope, max(b.q.begin + i, 0), x);
        }
        uint2 hi, lo;
        split_query<D>(x, hi, lo, f);
        *reinterpret_cast<uint2 *>(smem + qc * L::q_row + 8 * cc) = hi;
        *reinterpret_cast<uint2 *>(smem + (kTileCols + qc) * L::q_row + 8 * cc) = lo;
        if (cc == 0)
            s_f[qc] = f * t.scale;
    }
    __syncthreads();
    const int col = lane & 31, half = lane >> 5, qcol = 32 * wid + col;
    v4i qh[KS], ql[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
        qh[ks] = *reinterpret_cast<const v4i *>(smem + qcol * L::q_row + 32 * ks + 16 * half);
        ql[ks] = *reinterpret_cast<const v4i *>(smem + (kTileCols + qcol) * L::q_row + 32 * ks + 16 * half);
    }
    const float f = s_f[qcol];
    __syncthreads();

    // keys this lane's column sees, [clo, chi), and what all columns of the
    // wave see, [wlo, whi), or any of them, [ulo, uhi)
    const int pos = b.q.begin + (b.c0 + qcol) / t.group;
    int chi = t.causal ? min(te, pos + 1) : te;
    int clo = t.window > 0 ? max((int64_t)0, (int64_t)pos + 1 - t.window) : 0;
    if (qcol >= b.nc)
        chi = clo = 0;
    const int c_first = 32 * wid, c_last = min(32 * wid + 31, b.nc - 1);
    const int p_first = b.q.begin + (b.c0 + c_first) / t.group, p_last = b.q.begin + (b.c0 + c_last) / t.group;
    const KvSpan seen = kv_span(p_first, p_last, te, t.causal != 0, t.window);
    const bool idle = c_first >= b.nc;
    const int whi = c_last < 32 * wid + 31 ? 0 : t.causal ? min(te, p_first + 1) : te;
    const int wlo = t.window > 0 ? max((int64_t)0, (int64_t)p_last + 1 - t.window) : 0;

    const int32_t *table = a.table + (int64_t)b.s * a.table_stride;
    const int page = 1 << a.page_shift;
    uint4 rk[NI];
    uint32_t rv[NI][4];
    float rks = 0.0f, rvs = 0.0f;
    bool rok = false;
    auto page_of = [&](int key, bool &ok) {
        const int pid = table[min(key >> a.page_shift, a.table_width - 1)];
        ok = (unsigned)pid < (unsigned)a.pages && (key & ~15) < te && (key | 15) >= b.span.lo;
        return (int64_t)(ok ? pid : 0) * a.heads + b.h;
    };
    auto load = [&](int t0) {
#pragma unroll
        for (int k = 0; k < NI; k++) {
            const int it = (tid + NT * k) % ITEMS;
            const int row = it / (D / 16), chunk = it % (D / 16);
            bool ok;
            int64_t ph = page_of(t0 + row, ok);
            rk[k] = *reinterpret_cast<const uint4 *>(a.k + ((ph * D) << a.page_shift) +
                                                     ((t0 + row) & (page - 1)) * D + 16 * chunk);
            const int dg = it % (D / 4), sb = it / (D / 4), key = t0 + 4 * sb;
            ph = page_of(key, ok);
            const int8_t *p = a.v + ((ph * D) << a.page_shift) + (key & (page - 1)) * D + 4 * dg;
#pragma unroll
            for (int e = 0; e < 4; e++)
                rv[k][e] = *reinterpret_cast<const uint32_t *>(p + e * D);
        }
        const int64_t ph = page_of(t0 + 16 * (tid & 3), rok);
        rks = a.ks[ph];
        rvs = a.vs[ph];
    };
    auto store = [&](int buf) {
        char *lk = smem + buf * L::stage, *lv = lk + L::K;
#pragma unroll
        for (int k = 0; k < NI; k++) {
            const int it = tid + NT * k;
            if (ITEMS < NT && it >= ITEMS)
                break;
            const int row = it / (D / 16), chunk = it % (D / 16);
            *reinterpret_cast<uint4 *>(lk + k_place<D>(row, chunk)) = rk[k];
            // 4 keys x 4 dims, keys 4sb .. 4sb+3: quarter q of its group of
            // 16 is part q/2 of the chunk that half q%2 reads
            const int dg = it % (D / 4), sb = it / (D / 4), q = sb & 3;
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; e++)
                u[e] = rv[k][e] ^ 0x80808080u;
            const int chunk_v = 2 * (sb >> 2) + (q & 1), part = 8 * (q >> 1);
            *reinterpret_cast<uint2 *>(lv + v_place(4 * dg, chunk_v) + part) =
                make_uint2(codes_f16<0>(u[0], u[1]), codes_f16<0>(u[2], u[3]));
            *reinterpret_cast<uint2 *>(lv + v_place(4 * dg + 1, chunk_v) + part) =
                make_uint2(codes_f16<1>(u[0], u[1]), codes_f16<1>(u[2], u[3]));
            *reinterpret_cast<uint2 *>(lv + v_place(4 * dg + 2, chunk_v) + part) =
                make_uint2(codes_f16<2>(u[0], u[1]), codes_f16<2>(u[2], u[3]));
            *reinterpret_cast<uint2 *>(lv + v_place(4 * dg + 3, chunk_v) + part) =
                make_uint2(codes_f16<3>(u[0], u[1]), codes_f16<3>(u[2], u[3]));
        }
        if (tid < 4) {
            s_sc[buf][0][tid] = rok ? rks : -1.0f;
            s_sc[buf][1][tid] = rok && rvs > 0.0f ? 1.0f / rvs : 0.0f;
            s_sc[buf][2][tid] = rok ? log2f(rvs) : -INFINITY;
            s_sc[buf][3][tid] = rok ? rvs : 0.0f;
        }
    };

    v16f acc[DB] = {};
    float m = kNone, l = 0.0f, vref = 0.0f, lref = kNone;   // lref: log2 of vref
    const int steps = ts < te ? (te - ts + kTileKeys - 1) / kTileKeys : 0;
    if (steps > 0) {
        load(ts);
        store(0);
        load(ts + kTileKeys);
    }
    __syncthreads();
    for (int i = 0; i < steps; i++) {
        const int t0 = ts + kTileKeys * i;
        const char *lk = smem + (i & 1) * L::stage, *lv = lk + L::K;
        if (i + 1 < steps) {
            store((i + 1) & 1);
            load(t0 + 2 * kTileKeys);
        }
        if (!idle && t0 < seen.hi && t0 + kTileKeys > seen.lo) {
            const v4f ksc = *reinterpret_cast<const v4f *>(s_sc[i & 1][0]);
            const v4f ivs = *reinterpret_cast<const v4f *>(s_sc[i & 1][1]);
            const v4f lvs = *reinterpret_cast<const v4f *>(s_sc[i & 1][2]);
            const v4f vsc = *reinterpret_cast<const v4f *>(s_sc[i & 1][3]);
            float x[2][16], fk[4], zm = -INFINITY;
#pragma unroll
            for (int gi = 0; gi < 4; gi++)
                fk[gi] = fmaxf(f * ksc[gi], 1.0e-30f);   // (not 0: a masked score is -inf times it)
#pragma unroll
            for (int tt = 0; tt < 2; tt++) {
                v16i sh = {}, sl = {};
#pragma unroll
                for (int ks = 0; ks < KS; ks++) {
                    const v4i kf = *reinterpret_cast<const v4i *>(lk + k_place<D>(32 * tt + col, 2 * ks + half));
                    sh = __builtin_amdgcn_mfma_i32_32x32x32_i8(kf, qh[ks], sh, 0, 0, 0);
                    sl = __builtin_amdgcn_mfma_i32_32x32x32_i8(kf, ql[ks], sl, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 16; e++)
                    x[tt][e] = (float)((sh[e] << 7) + sl[e]);
            }
            const float kmin = fminf(fminf(ksc[0], ksc[1]), fminf(ksc[2], ksc[3]));
            const bool whole = t0 >= wlo && t0 + kTileKeys <= whi &&
                               __builtin_amdgcn_readfirstlane(kmin >= 0.0f ? 1 : 0);
            if (!whole) {
#pragma unroll
                for (int tt = 0; tt < 2; tt++)
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        const int key = t0 + 32 * tt + 8 * (e >> 2) + 4 * half + (e & 3);
                        const bool see = key < chi && key >= clo && ksc[2 * tt + (e >> 3)] >= 0.0f;
                        x[tt][e] = see ? x[tt][e] : -INFINITY;
                    }
            }
#pragma unroll
            for (int gi = 0; gi < 4; gi++) {
                const float *xs = x[gi >> 1] + 8 * (gi & 1);
                const float g0 = fmaxf(fmaxf(fmaxf(xs[0], xs[1]), fmaxf(xs[2], xs[3])),
                                       fmaxf(fmaxf(xs[4], xs[5]), fmaxf(xs[6], xs[7])));
                zm = fmaxf(zm, g0 * fk[gi]);
            }
            if (__any(zm > m + 8.0f)) {
                zm = fmaxf(zm, __shfl_xor(zm, 32, 64));
                const float mn = fmaxf(m, zm), al = __builtin_amdgcn_exp2f(m - mn);
#pragma unroll
                for (int n = 0; n < DB; n++)
                    acc[n] *= al;
                l *= al;
                m = mn;
            }
            const float lm = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(
                int, fmaxf(fmaxf(lvs[0], lvs[1]), fmaxf(lvs[2], lvs[3])))));
            if (lm > lref) {
                const float al = __builtin_amdgcn_exp2f(lref - lm);
#pragma unroll
                for (int n = 0; n < DB; n++)
                    acc[n] *= al;
                lref = lm;
                vref = fmaxf(fmaxf(vsc[0], vsc[1]), fmaxf(vsc[2], vsc[3]));
            }
            // The value scale goes into the exponent, 2^(z - m + log2(vs / vref)),
            // and out of the sum again, one factor per group of 16 keys.  A
            // scale too far below the largest would leave fp16's range there:
            // it is multiplied in afterwards.
            const float lmin = fminf(fminf(lvs[0], lvs[1]), fminf(lvs[2], lvs[3]));
            const bool far = __builtin_amdgcn_readfirstlane(lmin - lref < kFar ? 1 : 0);
            v8h p[4];
#pragma unroll
            for (int gi = 0; gi < 4; gi++) {
                const float lv = lvs[gi] - lref;
                const bool fr = lv < kFar;
                const float bias = (fr ? 0.0f : lv) - m;
                float pe[8], lg = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++)
                    pe[e] = __builtin_amdgcn_exp2f(fmaf(x[gi >> 1][8 * (gi & 1) + e], fk[gi], bias));
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    kv_h2 h;
                    h.x = (_Float16)pe[2 * e];
                    h.y = (_Float16)pe[2 * e + 1];
                    lg = __builtin_amdgcn_fdot2(h, (kv_h2){(_Float16)1.0f, (_Float16)1.0f}, lg, false);
                    p[gi][2 * e] = h.x;
                    p[gi][2 * e + 1] = h.y;
                }
                l = fmaf(lg, fr ? 1.0f : vref * ivs[gi], l);
                if (far) {
                    const float ratio = fr ? __builtin_amdgcn_exp2f(lv) : 1.0f;
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        p[gi][e] = (_Float16)(pe[e] * ratio);
                }
            }
#pragma unroll
            for (int n = 0; n < DB; n++)
#pragma unroll
                for (int gi = 0; gi < 4; gi++) {
                    const v8h vf = *reinterpret_cast<const v8h *>(lv + v_place(32 * n + col, 2 * gi + half));
                    acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, p[gi], acc[n], 0, 0, 0);
                }
        }
        __syncthreads();
    }
    if (qcol >= b.nc)
        return;
    l += __shfl_xor(l, 32, 64);
    const float s = l > 0.0f ? vref / l : 0.0f;
    if (t.splits > 1) {
        const int64_t at = ((int64_t)item * t.splits + sp) * t.used + qcol;
#pragma unroll
        for (int n = 0; n < DB; n++)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4 *>(t.part_o + at * D + 32 * n + 2 * e + 4 * half) =
                    make_float4(acc[n][e] * s, acc[n][e + 1] * s, acc[n][e + 2] * s, acc[n][e + 3] * s);
        if (half == 0)
            t.part_m[at] = l > 0.0f ? m + log2f(l) : kNone;
        return;
    }
    const int c = b.c0 + qcol, i = c / t.group, g = c - i * t.group;
    const int64_t row = b.q.q0 + i;
    const int head = b.h * t.group + g;
    uint16_t *o = t.O + row * t.os + (int64_t)head * D + 4 * half;
#pragma unroll
    for (int n = 0; n < DB; n++)
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
            const float x[8] = {acc[n][e] * s, acc[n][e + 1] * s, acc[n][e + 2] * s, acc[n][e + 3] * s,
                                acc[n][e + 4] * s, acc[n][e + 5] * s, acc[n][e + 6] * s, acc[n][e + 7] * s};
            const uint4 w = pack8<BF16>(x);
            *reinterpret_cast<uint2 *>(o + 32 * n + 2 * e) = make_uint2(w.x, w.y);
            *reinterpret_cast<uint2 *>(o + 32 * n + 2 * e + 8) = make_uint2(w.z, w.w);
        }
    if (t.lse && half == 0)
        t.lse[row * (int64_t)(a.heads * t.group) + head] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Merges the splits of one column: O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M),
// m_i the split's log2 of its sum.  256 threads: D/8 chunks x split lanes.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void k_kv_merge(KvArgs a, AttnArgs t)
{
    constexpr int CPR = D / 8, SL = 256 / CPR;
    __shared__ float s_o[SL][D + 4], s_m[SL], s_l[SL];
    const int tid = threadIdx.x, cc = tid % CPR, sl = tid / CPR;
    const int qc = blockIdx.x % t.used, item = blockIdx.x / t.used;
    Block b;
    if (!locate(a, t, item, t.cols, b) || qc >= b.nc)
        return;
    const int na = b.span.hi > b.span.lo ? (b.span.hi - b.span.base + t.chunk - 1) / t.chunk : 0;
    float m = kNone, l = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int i = sl; i < min(na, t.splits); i += SL) {
        const int64_t at = ((int64_t)item * t.splits + i) * t.used + qc;
        const float e = t.part_m[at];
        const float4 x0 = *reinterpret_cast<const float4 *>(t.part_o + at * D + 8 * cc);
        const float4 x1 = *reinterpret_cast<const float4 *>(t.part_o + at * D + 8 * cc + 4);
        const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        const float mn = fmaxf(m, e), al = exp2f(m - mn), be = e > kNone ? exp2f(e - mn) : 0.0f;
        l = l * al + be;
#pragma unroll
        for (int k = 0; k < 8; k++)
            o[k] = o[k] * al + x[k] * be;
        m = mn;
    }
#pragma unroll
    for (int k = 0; k < 8; k++)
        s_o[sl][8 * cc + k] = o[k];
    if (cc == 0) {
        s_m[sl] = m;
        s_l[sl] = l;
    }
    __syncthreads();
    if (sl != 0)
        return;
    float M = kNone, L = 0.0f;
    for (int i = 0; i < SL; i++)
        M = fmaxf(M, s_m[i]);
#pragma unroll
    for (int k = 0; k < 8; k++)
        o[k] = 0.0f;
    for (int i = 0; i < SL; i++) {
        const float al = exp2f(s_m[i] - M);
        L += s_l[i] * al;
#pragma unroll
        for (int k = 0; k < 8; k++)
            o[k] += s_o[i][8 * cc + k] * al;
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++)
        o[k] *= inv;
    const int c = b.c0 + qc, i = c / t.group, g = c - i * t.group;
    const int64_t row = b.q.q0 + i;
    const int head = b.h * t.group + g;
    *reinterpret_cast<uint4 *>(t.O + row * t.os + (int64_t)head * D + 8 * cc) = pack8<BF16>(o);
    if (t.lse && cc == 0)
        t.lse[row * (int64_t)(a.heads * t.group) + head] = L > 0.0f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

constexpr int kFewTarget = 1024;       // workgroups aimed at: 4 for each CU
constexpr int kTileTarget = 512;
constexpr int64_t kTileMinSplit = 1024;
constexpr int kTileFrom = 64;          // columns from which the tiled kernel is taken

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

int64_t plan_items(const li8_kv_batch &b, const li8_kv_cache &c, const KvPlan &p)
{
    return (int64_t)b.seqs * c.heads * p.blocks;
}

template <int D, bool BF16>
hipError_t attention_go(const KvArgs &a, const AttnArgs &t, int64_t items, hipStream_t s)
{
    if (t.cols == kTileCols) {
        const int64_t pairs = items / t.blocks;
        // (sequence, head) pairs dealt over the XCDs: 8 lanes, fewer where
        // that would leave XCDs without work
        const int lanes = pairs >= 64 ? 8 : (int)std::min<int64_t>(8, pairs & -pairs);
        k_kv_tiled<D, BF16><<<(unsigned)(round_up(pairs, lanes) * t.blocks * t.splits), 64 * kTileWaves, 0, s>>>(
            a, t, (int)pairs, lanes);
    } else {
        k_kv_few<D, BF16><<<(unsigned)(items * t.splits), 64 * kFewWaves, 0, s>>>(a, t);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || t.splits == 1)
        return e;
    k_kv_merge<D, BF16><<<(unsigned)(items * t.used), 256, 0, s>>>(a, t);
    return hipGetLastError();
}

} // namespace

KvPlan kv_plan(const li8_kv_batch &b, const li8_kv_cache &c, int q_heads, int window)
{
    KvPlan p = {LI8_KV_EMPTY, kKvCols, 0, 0, 1, 0};
    const int64_t rows = std::min(b.max_q, b.tokens), group = q_heads / c.heads;
    if (rows == 0 || b.seqs == 0)
        return p;
    const int64_t cols = rows * group;
    if (cols >= kTileFrom) {
        p.path = LI8_KV_TILED;
        p.cols = kTileCols;
    } else {
        p.path = LI8_KV_FEW;
    }
    p.blocks = (int)((cols + p.cols - 1) / p.cols);
    p.used = (int)std::min<int64_t>(p.cols, cols);
    const int64_t items = plan_items(b, c, p);
    // keys from a span's base to its end at most: a window's keys, the other
    // rows of the block and the rounding of the base
    int64_t span = b.max_kv;
    if (window > 0)
        span = std::min<int64_t>(span, (int64_t)window + p.cols + 31);
    const int64_t target = p.path == LI8_KV_TILED ? kTileTarget : kFewTarget;
    const int64_t least = p.path == LI8_KV_TILED ? kTileMinSplit : kKvMinSplit;
    const int64_t chunk = std::max(least, round_up((items * span + target - 1) / target, 32 * kFewWaves));
    p.chunk = (int)std::min<int64_t>(chunk, INT32_MAX / 2);
    p.splits = (int)std::max<int64_t>(1, (span + p.chunk - 1) / p.chunk);
    return p;
}

size_t kv_workspace(const li8_kv_batch &b, const li8_kv_cache &c, int q_heads)
{
    const KvPlan p = kv_plan(b, c, q_heads, 0);
    if (p.path == LI8_KV_EMPTY)
        return 0;
    // splits under any window: a part has at least `least` keys, and there are
    // at most target / items parts, rounded up
    const int64_t items = plan_items(b, c, p);
    const int64_t target = p.path == LI8_KV_TILED ? kTileTarget : kFewTarget;
    const int64_t least = p.path == LI8_KV_TILED ? kTileMinSplit : kKvMinSplit;
    const int64_t most = std::min<int64_t>((b.max_kv + least - 1) / least, target / items + 1);
    if (most <= 1)
        return 0;
    const int64_t parts = items * most * p.used;
    return align_up((size_t)parts * 4 * c.head_dim, 256) + align_up((size_t)parts * 4, 256);
}

hipError_t launch_kv_attention(KvTokens Q, bool bf16, int q_heads, float scale, KvRope rope,
                               bool causal, int window, const li8_kv_batch &b,
                               const li8_kv_cache &c, uint16_t *O, int64_t os, float *lse,
                               char *ws, hipStream_t s)
{
    const KvPlan p = kv_plan(b, c, q_heads, window);
    const KvArgs a = kv_args(b, c);
    const int64_t items = plan_items(b, c, p);
    AttnArgs t;
    t.Q = Q; t.rope = rope; t.O = O; t.os = os; t.lse = lse;
    t.part_o = reinterpret_cast<float *>(ws);
    t.part_m = reinterpret_cast<float *>(ws + align_up((size_t)items * p.splits * p.used * 4 * c.head_dim, 256));
    t.scale = scale * kLog2e;
    t.group = q_heads / c.heads; t.causal = causal; t.window = window;
    t.cols = p.cols; t.blocks = p.blocks; t.used = p.used; t.splits = p.splits; t.chunk = p.chunk;
    if (c.head_dim == 128)
        return bf16 ? attention_go<128, true>(a, t, items, s) : attention_go<128, false>(a, t, items, s);
    return bf16 ? attention_go<64, true>(a, t, items, s) : attention_go<64, false>(a, t, items, s);
}

} // namespace li8
