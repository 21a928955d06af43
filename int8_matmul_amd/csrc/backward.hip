// Gradients through the frozen int8 weight, for gfx950.
//
//   dZ[t,n] = dY[t,n] act'(Z[t,n])                      (linear)
//   dZ      = [ dH U act'(G) | dH act(G) ]              (gated pair, N = 2F)
//   dX[t,k] = sum_n dZ[t,n] sW[n] Wq[n,k],   dbias[n] = sum_t dZ[t,n]
//
// 1. k_grad_rows, one workgroup per token row: dZ in fp32 from the fp16 inputs,
//    the row's largest |dZ sW|, and the product's operand
//    A[t,n] = fp16(dZ sW 2^(14 - e)) with e that maximum's exponent: the scale sW
//    sits on the contracted index, so it has to go into one of the operands,
//    and a power of two for each row costs no rounding and keeps gradients of
//    any size inside fp16 (values down to 2^-28 of the row's largest keep all
//    11 bits).  One rounding of each element, 2^-11 at most, is what the matrix
//    instructions' 16-bit operands need; the codes are exact in fp16.
// 2. k_grad_gemm: dX = A . Wq on v_mfma_f32_32x32x16_f16 (fp32 sums), codes
//    converted on the way from LDS to the registers; times 2^(e - 14).
// 3. k_grad_join where the contraction was split between workgroups.
// dbias comes from workgroups of its own in the first launch, and where its rows
// were split its sums are added in the last one.
#include <algorithm>

#include "act_math.h"
#include "li8_internal.h"
#include "quant_math.h"
#include "tile_common.h"

namespace li8 {
namespace {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef v4i v4i_any __attribute__((aligned(2)));   // at any fp16 element
typedef float v4f __attribute__((ext_vector_type(4)));
typedef v4f v4f_any __attribute__((aligned(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// Elementwise part: eight features f .. f+7 of a row.
// ---------------------------------------------------------------------------

// Eight fp16 values in memory order; `n` of them exist, the others are 0.  16-byte
// accesses at whatever alignment p has (the hardware takes any).  WHOLE: all
// or none exist; otherwise a part goes element by element.
template <bool WHOLE>
struct Half8 {
    v4i w;

    __device__ __forceinline__ void load(const uint16_t *p, int n)
    {
        w = v4i{0, 0, 0, 0};
        if constexpr (WHOLE) {
            if (n > 0)
                w = *reinterpret_cast<const v4i_any *>(p);
        } else if (n >= 8) {
            w = *reinterpret_cast<const v4i_any *>(p);
        } else if (n > 0) {
#pragma unroll
            for (int e = 0; e < 7; e++)
                if (e < n)
                    w[e >> 1] |= (int)((uint32_t)p[e] << (16 * (e & 1)));
        }
    }
    __device__ __forceinline__ float value(int e) const
    {
        return h2f(((uint32_t)w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
    }
};

template <bool WHOLE>
__device__ __forceinline__ void store8(uint16_t *p, int n, const float (&v)[8])
{
    const v4i w = {(int)pack_f16x2(v[0], v[1]), (int)pack_f16x2(v[2], v[3]), (int)pack_f16x2(v[4], v[5]),
                   (int)pack_f16x2(v[6], v[7])};
    if constexpr (WHOLE) {
        if (n > 0)
            *reinterpret_cast<v4i_any *>(p) = w;
    } else if (n >= 8) {
        *reinterpret_cast<v4i_any *>(p) = w;
    } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < 7; e++)
            if (e < n)
                p[e] = (uint16_t)((uint32_t)w[e >> 1] >> (16 * (e & 1)));
    }
}

template <bool WHOLE>
__device__ __forceinline__ void load8f(const float *p, int n, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = 0.0f;
    if (WHOLE ? n > 0 : n >= 8) {
        const v4f_any *q = reinterpret_cast<const v4f_any *>(p);
        const v4f lo = q[0], hi = q[1];
#pragma unroll
        for (int e = 0; e < 4; e++)
            v[e] = lo[e], v[4 + e] = hi[e];
    } else if (!WHOLE && n > 0) {
#pragma unroll
        for (int e = 0; e < 7; e++)
            if (e < n)
                v[e] = p[e];
    }
}

// KIND of a linear gradient without an activation: dZ = dY, Z is not read.
constexpr int kNoAct = 3;

struct GradArgs {
    const uint16_t *dY;    // [T, F] (F = N, or N / 2 for a pair)
    const uint16_t *pre;   // [T, N], or null (linear: slope 1)
    const float *sW;
    uint16_t *grad_pre;    // [T, N], or null
    ActParams act;
    int T, N, Np;
};

// Inputs of eight features f .. f+7 of row t.
template <bool GATED, bool WHOLE>
struct RawGrad {
    Half8<WHOLE> d, g, u;

    // `n` of them: 8 or 0 with WHOLE
    __device__ __forceinline__ void load(const GradArgs &a, int64_t t, int f, int n)
    {
        const int F = GATED ? a.N >> 1 : a.N;
        d.load(a.dY + t * F + f, n);
        if (GATED || a.pre)
            g.load(a.pre + t * a.N + f, n);
        if constexpr (GATED)
            u.load(a.pre + t * a.N + F + f, n);
    }

    // dZ: z[0] (linear), or z[0] the gate's and z[1] the up projection's (pair)
    template <int KIND>
    __device__ __forceinline__ void grad(const GradArgs &a, float (&z)[1 + GATED][8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if constexpr (KIND == kNoAct) {
                z[0][e] = d.value(e);
            } else {
                float v, s;
                act_value_slope<KIND>(g.value(e), a.act, v, s);
                if constexpr (GATED) {
                    z[0][e] = d.value(e) * u.value(e) * s;
                    z[1][e] = d.value(e) * v;
                } else {
                    z[0][e] = d.value(e) * s;
                }
            }
        }
    }
};

// From a row's largest magnitude (its bits; NaN above all), of biased exponent e:
// the scale 2^(14 - e) for the product's operand and its inverse for the result.
// (Below 2^-107 the scale stays at 2^121; an all-zero row and one with
// infinities or NaN take 1.)
__device__ __forceinline__ void row_unit(uint32_t m, float &scale, float &inverse)
{
    const uint32_t e = m >> 23, ec = max(e, 20u);
    const bool one = m == 0 || e == 255;
    scale = one ? 1.0f : __builtin_bit_cast(float, (268u - ec) << 23);
    inverse = one ? 1.0f : __builtin_bit_cast(float, (ec - 14u) << 23);
}

// How a row of F features falls into groups of eight: EVEN, F a multiple of 8;
// MOVED, F > 8: the last group is moved back to end with the row, so that it
// is whole and some features are formed twice, alike; SHORT, F < 8: one group.
enum { EVEN, MOVED, SHORT };

inline int row_mode(int F) { return F < 8 ? SHORT : F % 8 ? MOVED : EVEN; }

// First feature of group g, and how many of its eight count.
template <int MODE>
__device__ __forceinline__ int group_start(int g, int F, int &n)
{
    const bool ok = g < (F + 7) / 8;
    n = ok ? (MODE == SHORT ? F : 8) : 0;
    return MODE == MOVED ? min(8 * g, F - 8) : 8 * g;
}

constexpr int kRowThreads = 512;

// ---------------------------------------------------------------------------
// dbias: a workgroup has 16 groups of 8 features and a strip of the rows, shared
// by 32 lanes of threads with four rows in flight each; sums of more than one
// strip go to partial sums [strips][N], added in order by k_grad_join.
// ---------------------------------------------------------------------------
struct ColSums {
    float *out;     // dbias, or the partial sums; null: none asked for
    int blocks;     // of 128 features
    int strips;
};

template <bool GATED, int KIND, int MODE>
__device__ void grad_cols(const GradArgs &a, const ColSums &c, int block)
{
    constexpr int P = 1 + GATED, LANES = kRowThreads / 16, AHEAD = 4;
    constexpr bool WHOLE = MODE != SHORT;
    __shared__ float sum[LANES][P][128];
    const int gl = threadIdx.x & 15, rl = threadIdx.x >> 4, strip = block / c.blocks;
    const int F = GATED ? a.N >> 1 : a.N, g0 = (block - strip * c.blocks) * 16;
    int n;
    const int f = group_start<MODE>(g0 + gl, F, n);
    const int t0 = (int)((int64_t)a.T * strip / c.strips), t1 = (int)((int64_t)a.T * (strip + 1) / c.strips);
    float s[P][8];
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
        for (int e = 0; e < 8; e++)
            s[p][e] = 0.0f;
    for (int t = t0 + rl; t < t1; t += AHEAD * LANES) {
        RawGrad<GATED, WHOLE> raw[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; i++)
            raw[i].load(a, t + i * LANES, f, t + i * LANES < t1 ? n : 0);
#pragma unroll
        for (int i = 0; i < AHEAD; i++) {   // (rows past the end: zeros)
            float z[P][8];
            raw[i].template grad<KIND>(a, z);
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int e = 0; e < 8; e++)
                    s[p][e] += z[p][e];
        }
    }
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
        for (int e = 0; e < 8; e++)
            sum[rl][p][8 * gl + e] = s[p][e];
    __syncthreads();
    if (threadIdx.x < P * 128) {
        const int p = threadIdx.x >> 7, i = threadIdx.x & 127;
        int m;
        const int col = group_start<MODE>(g0 + (i >> 3), F, m) + (i & 7);
        if ((i & 7) < m) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < LANES; w++)
                v += sum[w][p][i];
            c.out[(int64_t)strip * a.N + p * F + col] = v;
        }
    }
}

// TPR threads a row: 64 (a wave, eight rows a workgroup) or all 512.
// NR > 0: the row's NR rounds of 8 TPR features, their inputs requested ahead (all
// of them; of four rounds of a pair one at a time), their results in registers
// between the maximum and the conversion; 0: rows of any length, computed a second
// time.  Two workgroups a CU have 128 registers a thread: four rounds of a pair take
// more even so, and 22 to 24 of them go to scratch memory; no other form spills.
// (512 threads against 1024 with half the rounds: F = 11008, 4096 rows, dZ kept: 133
// and 164 us.)
// The launch's first workgroups form the column sums, where asked for: with 75
// rows a launch of their own costs more than they do.
template <bool GATED, int KIND, int MODE, int TPR, int NR>
__global__ __launch_bounds__(kRowThreads, 4) void k_grad_rows(GradArgs a, ColSums c,
                                                              uint16_t *__restrict__ A, float *__restrict__ fac)
{
    constexpr int P = 1 + GATED, R = NR > 0 ? NR : 1, AHEAD = GATED && NR == 4 ? 1 : R, ROWS = kRowThreads / TPR;
    constexpr bool WHOLE = MODE != SHORT;
    static_assert(TPR == 64 || TPR == kRowThreads, "a wave or the workgroup");
    __shared__ uint32_t wmax[kRowThreads / 64];
    const int cols = c.out ? c.blocks * c.strips : 0;
    if ((int)blockIdx.x < cols) {
        grad_cols<GATED, KIND, MODE>(a, c, blockIdx.x);
        return;
    }
    const int first = blockIdx.x - cols, stride = (gridDim.x - cols) * ROWS;
    const int tid = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int row = TPR == 64 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) : 0;   // (uniform: scalar addresses)
    const int F = GATED ? a.N >> 1 : a.N, groups = (F + 7) / 8;
    // (a wave's row is the same for all its lanes, a workgroup's for all its waves)
    for (int64_t t = (int64_t)first * ROWS + row; t < a.T; t += stride) {
        RawGrad<GATED, WHOLE> raw[AHEAD];
        float keep[R][P][8];
        uint32_t m = 0;   // largest magnitude as bits (NaN above all)
        auto request = [&](int r, int g) {
            int n;
            const int f = group_start<MODE>(g, F, n);
            raw[r].load(a, t, f, n);
        };
        // dZ of a round, written where it is asked for, times sW
        auto compute = [&](int r, int g, bool first) {
            int n;
            const int f = group_start<MODE>(g, F, n);
            raw[r % AHEAD].template grad<KIND>(a, keep[r]);
            if (first && a.grad_pre)
#pragma unroll
                for (int p = 0; p < P; p++)
                    store8<WHOLE>(a.grad_pre + t * a.N + p * F + f, n, keep[r][p]);
#pragma unroll
            for (int p = 0; p < P; p++) {
                float s[8];
                load8f<WHOLE>(a.sW + p * F + f, n, s);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    keep[r][p][e] *= s[e];
                    m = max(m, __builtin_bit_cast(uint32_t, keep[r][p][e]) & 0x7fffffffu);
                }
            }
        };
        if constexpr (NR > 0) {
#pragma unroll
            for (int r0 = 0; r0 < NR; r0 += AHEAD) {
#pragma unroll
                for (int r = 0; r < AHEAD; r++)
                    request(r, tid + (r0 + r) * TPR);
#pragma unroll
                for (int r = r0; r < r0 + AHEAD; r++)
                    compute(r, tid + r * TPR, true);
            }
        } else {
            for (int g = tid; g < groups; g += TPR) {
                request(0, g);
                compute(0, g, true);
            }
        }
        m = wave_max(m);
        if constexpr (TPR > 64) {
            if ((tid & 63) == 0)
                wmax[tid >> 6] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kRowThreads / 64; w++)
                m = max(m, wmax[w]);
        }
        float scale, inverse;
        row_unit(m, scale, inverse);
        if (tid == 0)
            fac[t] = inverse;
        auto put = [&](int r, int g) {
            int n;
            const int f = group_start<MODE>(g, F, n);
#pragma unroll
            for (int p = 0; p < P; p++) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    keep[r][p][e] *= scale;   // (a power of two: exact)
                store8<WHOLE>(A + t * a.Np + p * F + f, n, keep[r][p]);
            }
        };
        if constexpr (NR > 0) {
#pragma unroll
            for (int r = 0; r < NR; r++)
                put(r, tid + r * TPR);
        } else {
            for (int g = tid; g < groups; g += TPR) {
                request(0, g);
                compute(0, g, false);
                put(0, g);
            }
        }
        if (tid < a.Np - a.N)   // (less than 64)
            A[t * a.Np + a.N + tid] = 0;
        if constexpr (TPR > 64)
            __syncthreads();   // (wmax is read)
    }
}

// ---------------------------------------------------------------------------
// The product.  BM x 256 tiles of dX [T,K]; the contraction in stages of 64
// weight rows held in a ring of NS LDS buffers: A rows of 128 bytes, and the
// weight's 64 rows of 256 codes as they lie in memory.  The matrix
// instruction wants eight consecutive n of one column k in a lane, so the codes
// are read with the transposing LDS read (ds_read_b64_tr_b8: 16 lanes read 8 rows
// of 16 bytes and each gets one column): no second, transposed copy of the weight.
// Chunks of 16 codes are permuted in a row by twice the row's index so that
// the 8 rows of a read and its two neighbouring chunks meet all 64 banks once.
// Stages, waits and the tile order are those of k_gemm (gemm.hip).
// Measured: 4096 x 4096 x 22016 in 590-610 us (1.23 PFLOP/s; a library's fp16 product of
// two 16-bit operands takes 621), 4096 x 11008 x 4096 in 310-320 (library: 431).  The
// matrix units are busy for 73 % of the cycles and the clock is at 1.6 GHz, the
// board's power limit.
// ---------------------------------------------------------------------------
constexpr int kGN = 64;    // weight rows per stage
constexpr int kGK = 256;   // columns of dX per tile

// Eight codes as fp16.  0x6400 | u is 1024 + u for a byte u, and with its sign bit
// flipped a code is u - 128, so 1152 less is the code, exactly.
__device__ __forceinline__ v8h codes_to_f16(v2i w)
{
    const v2h off = {(_Float16)1152.0f, (_Float16)1152.0f};
    v4i r;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t u = (uint32_t)w[i] ^ 0x80808080u;
        r[2 * i] = __builtin_bit_cast(
            int, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off);
        r[2 * i + 1] = __builtin_bit_cast(
            int, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off);
    }
    return __builtin_bit_cast(v8h, r);
}

__device__ __forceinline__ v2i read_codes_tr(const int8_t *p)
{
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((LI8_LDS v2i *)const_cast<int8_t *>(p));
}

// A buffer's description as the four scalar words that the instruction takes.
__device__ __forceinline__ v4i rsrc_words(const void *p, int bytes)
{
    const uint64_t a = (uint64_t)(uintptr_t)p;
    return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xffff),
               __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

// 16 bytes per lane from r at voffset + soffset into LDS at dst + 16*lane.  As
// load_to_lds, but written out: behind the builtin the compiler lets every
// transposing LDS read wait for all loads in flight (vmcnt(0)).  It has no
// register to write, and what it writes to LDS is ordered by
// wait_loads_barrier, which counts it.  The LDS address is in M0 by the operand's
// constraint, so the compiler knows that M0 is taken (one wait state before its use).
__device__ __forceinline__ void load_to_lds_raw(v4i r, uint32_t dst, int voffset, int soffset)
{
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "{m0}"(dst), "v"(voffset), "s"(r), "s"(soffset));
}

// Permutation of the 16-byte chunks of A's 128-byte rows: 16 rows' reads of one
// chunk meet all banks, and rows 32 apart have the same one, so that a
// lane's fragments are at constant distances.
__device__ __forceinline__ int swz_a(int row) { return (row ^ ((row >> 3) & 3)) & 7; }

template <int BM, int NS, int WM, int WN, int GM, bool SPLIT>
__global__ __launch_bounds__(WM *WN * 64) void k_grad_gemm(
    const uint16_t *__restrict__ A, const int8_t *__restrict__ Wq, const float *__restrict__ fac,
    int T, int K, int N, int Np, int tiles_m, int tiles_k, int splits, uint16_t *__restrict__ dX,
    float *__restrict__ part)
{
    constexpr int NT = WM * WN * 64, NW = WM * WN;
    constexpr int FM = BM / (WM * 32), FK = kGK / (WN * 32);
    constexpr int KS = kGN / 16;                       // MFMA k-steps per stage
    constexpr int ASZ = BM * kGN * 2, SSZ = ASZ + kGN * kGK;
    constexpr int CA = BM * 8, CB = kGN * 16;          // 16-byte chunks of a stage
    constexpr int LA = (CA + NT - 1) / NT, LB = CB / NT;
    constexpr int CPR = FK * 4;                        // 16-byte chunks per staging row
    constexpr int STG = NW * FM * 32 * CPR * 16;
    constexpr int LDSB = NS * SSZ > STG ? NS * SSZ : STG;
    static_assert(FM * WM * 32 == BM && FK * WN * 32 == kGK, "tile shape");
    static_assert(LB * NT == CB && (LA * NT == CA || (LA == 1 && NT % CA == 0 && CA % 64 == 0)), "loader shape");
    static_assert(LDSB <= 160 * 1024 && NS >= 2, "LDS of one workgroup");
    __shared__ __attribute__((aligned(1024))) int8_t lds[LDSB];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wid / WN, wn = wid % WN;

    // ---- tile and part of the contraction ----
    int bid = blockIdx.x;
    const int tiles = tiles_m * tiles_k;
    {
        const int nblk = tiles * splits;
        const int per = nblk / 8, rem = nblk % 8, xcd = bid % 8, loc = bid / 8;
        bid = (xcd < rem) ? xcd * (per + 1) + loc : rem * (per + 1) + (xcd - rem) * per + loc;
    }
    const int sp = bid / tiles;
    bid -= sp * tiles;
    const int width = GM * tiles_k;
    const int first_m = (bid / width) * GM;
    const int gm = min(tiles_m - first_m, GM);
    const int m0 = (first_m + (bid % width) % gm) * BM, k0 = (bid % width) / gm * kGK;
    const int nst = Np / kGN, stages = nst / splits, more = nst - stages * splits;
    const int st0 = sp * stages + min(sp, more);
    const int ns = stages + (sp < more ? 1 : 0);   // (at least 1: splits <= nst)

    // ---- loaders: load i of this lane fills chunk p = i*NT + tid of A's, or of
    // the weight's, rows (A: row p / 8, weight: row p / 16); with fewer chunks
    // of A than threads the waves fill them twice over, with the same bytes, so
    // that every wave counts the same loads ----
    const int rows = min(BM, T - m0);
    const v4i rA = rsrc_words(A + (int64_t)m0 * Np, 2 * rows * Np), rB = rsrc_words(Wq, N * K);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LI8_LDS int8_t *)lds;
    int voA[LA], voB[LB], rowB[LB];
#pragma unroll
    for (int i = 0; i < LA; i++) {
        const int p = (i * NT + tid) % CA, row = p >> 3, q = (p & 7) ^ swz_a(row);
        voA[i] = min(row, rows - 1) * Np * 2 + q * 16;
    }
#pragma unroll
    for (int i = 0; i < LB; i++) {
        const int p = i * NT + tid, row = p >> 4, k = k0 + 16 * ((p & 15) ^ (2 * (row & 7)));
        voB[i] = row * K + k;
        rowB[i] = k < K ? N - row : 0;   // the row exists while n0 < rowB
    }
    auto issue = [&](int it, int buf) {
        const int n0 = (st0 + it) * kGN;
        const uint32_t dst = lds0 + (uint32_t)buf;
#pragma unroll
        for (int i = 0; i < LA; i++)
            load_to_lds_raw(rA, dst + ((i * NT + wid * 64) % CA) * 16, voA[i], 2 * n0);
#pragma unroll
        for (int i = 0; i < LB; i++)
            load_to_lds_raw(rB, dst + ASZ + (i * NT + wid * 64) * 16, n0 < rowB[i] ? voB[i] : kOutOfRange, n0 * K);
    };

    // ---- fragments ----
    // lane l supplies token row l & 31 of each block and the 16 bytes of chunk
    // 2 kk + (l >> 5) of k-step kk; of the weight it reads half (l & 1) of the
    // chunk of 16 columns (l >> 4) & 1 in row 8 (l >> 5) + (l & 15) / 2 of the
    // k-step, and gets column l & 31.  Everything else is a constant offset.
    const int khalf = lane >> 5;
    int offA[KS], offB[FK];
    {
        const int row = wm * FM * 32 + (lane & 31), r = (lane & 15) >> 1;
#pragma unroll
        for (int kk = 0; kk < KS; kk++)
            offA[kk] = row * 128 + (((kk * 2 + khalf) ^ swz_a(row)) * 16);
#pragma unroll
        for (int b = 0; b < FK; b++) {
            const int c = (wn * FK + b) * 2 + ((lane >> 4) & 1);
            offB[b] = ASZ + (8 * khalf + r) * kGK + ((c ^ (2 * r)) * 16) + 8 * (lane & 1);
        }
    }
    v16f acc[FM][FK];
#pragma unroll
    for (int a = 0; a < FM; a++)
#pragma unroll
        for (int b = 0; b < FK; b++)
            acc[a][b] = v16f{};

    // Fragments of two k-steps: while one is multiplied the next is read, and
    // its codes are converted behind the first products.
    v8h fa[2][FM], fb[2][FK];
    v2i raw[FK];
    auto lread = [&](int set, int st, int kk) {
#pragma unroll
        for (int b = 0; b < FK; b++)
            raw[b] = read_codes_tr(lds + st + offB[b] + kk * 16 * kGK);
#pragma unroll
        for (int a = 0; a < FM; a++)
            fa[set][a] = *reinterpret_cast<const v8h *>(lds + st + offA[kk] + a * 32 * 128);
    };
    auto convert = [&](int set) {
#pragma unroll
        for (int b = 0; b < FK; b++)
            fb[set][b] = codes_to_f16(raw[b]);
    };
    auto mfmas = [&](int set) {
#pragma unroll
        for (int a = 0; a < FM; a++)
#pragma unroll
            for (int b = 0; b < FK; b++)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[set][b], fa[set][a], acc[a][b], 0, 0, 0);
    };
    // One MFMA with up to two LDS reads after it until they are all issued, then
    // with the conversions' share
    constexpr int NMF = FM * FK, NRD = FM + FK, RPM = (NRD + NMF / 2) / (NMF / 2 ? NMF / 2 : 1);
    auto interleave = [&]() {
        int rd = 0;
#pragma unroll
        for (int i = 0; i < NMF; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (rd < NRD) {
                __builtin_amdgcn_sched_group_barrier(0x100, RPM, 0);
                rd += RPM;
            } else {
                __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    int st = 0;   // this stage's ring buffer
    auto stage = [&](int it, auto wait_c, auto issue_c, auto last_c) {
        constexpr int WAIT = decltype(wait_c)::value;
        constexpr bool ISSUE = decltype(issue_c)::value;
        constexpr bool LAST = decltype(last_c)::value;
#pragma unroll
        for (int kk = 0; kk < KS; kk++) {
            const int cur = kk & 1;
            if (kk + 1 < KS) {
                lread(cur ^ 1, st, kk + 1);
                mfmas(cur);
                convert(cur ^ 1);
                interleave();
            } else if constexpr (!LAST) {
                wait_loads_barrier<WAIT>();   // stage it+1 landed; stage it read by all
                if constexpr (ISSUE)
                    issue(it + NS, st);
                st = st + SSZ == NS * SSZ ? 0 : st + SSZ;
                lread(cur ^ 1, st, 0);
                mfmas(cur);
                convert(cur ^ 1);
                interleave();
            } else {
                mfmas(cur);
            }
        }
    };
    using TF = std::false_type;
    using TT = std::true_type;
    using W0 = std::integral_constant<int, 0>;
    using WS = std::integral_constant<int, (LA + LB) * (NS - 2)>;

    // the rows' factors, in registers from here on
    const int ltok = wm * FM * 32 + (lane & 31);
    float fx[FM];
#pragma unroll
    for (int a = 0; a < FM; a++)
        fx[a] = fac[min(m0 + ltok + 32 * a, T - 1)];
#pragma unroll
    for (int s = 0; s < NS; s++)
        if (s < ns)
            issue(s, s * SSZ);
    if (ns >= NS)
        wait_loads_barrier<(NS - 1) * (LA + LB)>();   // stage 0 landed
    else
        wait_loads_barrier<0>();
    lread(0, 0, 0);
    convert(0);
    int it = 0;
    for (; it + NS < ns; it++)      // steady state
        stage(it, WS{}, TT{}, TF{});
    for (; it + 1 < ns; it++)       // drain
        stage(it, W0{}, TF{}, TF{});
    stage(it, W0{}, TF{}, TT{});

    // ---- epilogue ----
    // acc[a][b], register r: token ltok + 32a, column 32b + 8 (r/4) + 4 khalf + r%4
    // of the wave's columns
    const int col0 = k0 + wn * FK * 32;
    wait_loads_barrier<0>();   // the ring is free
    if constexpr (SPLIT) {
        // fp32, in the rows' units: 32 columns at a time through LDS, so that the
        // stores are whole lines; non-temporal, so that the L2 holds nothing to
        // write back when the kernel ends
        float *out = part + (int64_t)sp * T * K;
        int8_t *own = lds + wid * (FM * 32) * 128;
        static_assert(NW * FM * 32 * 128 <= LDSB, "staging rows");
#pragma unroll
        for (int b = 0; b < FK; b++) {
#pragma unroll
            for (int a = 0; a < FM; a++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    const int row = a * 32 + (lane & 31);
                    *reinterpret_cast<v4f *>(own + row * 128 + (((2 * g + khalf) ^ (row & 7)) * 16)) =
                        v4f{acc[a][b][4 * g], acc[a][b][4 * g + 1], acc[a][b][4 * g + 2], acc[a][b][4 * g + 3]};
                }
#pragma unroll
            for (int i = 0; i < FM * 32 * 8 / 64; i++) {
                const int id = i * 64 + lane, row = id >> 3, t = m0 + wm * FM * 32 + row;
                const int k = col0 + 32 * b + 4 * (id & 7);
                const v4f v = *reinterpret_cast<const v4f *>(own + row * 128 + (((id & 7) ^ (row & 7)) * 16));
                if (t < T && k < K)
                    __builtin_nontemporal_store(v, reinterpret_cast<v4f *>(out + (int64_t)t * K + k));
            }
        }
        return;
    }
    int8_t *own = lds + wid * (FM * 32) * CPR * 16;
#pragma unroll
    for (int a = 0; a < FM; a++)
#pragma unroll
        for (int b = 0; b < FK; b++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    p[j] = acc[a][b][4 * g + j] * fx[a];
                    asm("" : "+v"(p[j]));
                }
                *reinterpret_cast<uint2 *>(own + stage_off<CPR>(a * 32 + (lane & 31), b * 4 + g) + 8 * khalf) =
                    make_uint2(pack_f16x2(p[0], p[1]), pack_f16x2(p[2], p[3]));
            }
#pragma unroll
    for (int i = 0; i < FM * 32 * CPR / 64; i++) {
        const int id = i * 64 + lane, row = id / CPR, ch = id % CPR;
        const v4i v = *reinterpret_cast<const v4i *>(own + stage_off<CPR>(row, ch));
        const int t = m0 + wm * FM * 32 + row, k = col0 + 8 * ch;
        if (t < T && k < K)   // (K is a multiple of 16)
            __builtin_nontemporal_store(v, reinterpret_cast<v4i *>(dX + (int64_t)t * K + k));
    }
}

// ---------------------------------------------------------------------------
// Few rows (T <= 64): one kernel from dY to partial sums of dX.  A workgroup has
// 256 columns of dX and a range of weight rows n; it forms its range's dZ for all
// rows itself (the same inputs serve all column tiles from the L2), so nothing
// has to wait for a kernel that knows whole rows: a row's power of two is that of
// its largest value in the range, and the partial sums are stored without it.
// The weight's codes are requested before anything else; a wave's loads complete in
// order, so its inputs, requested after them, come when its codes have.  Every range's
// workgroup of the first column tile sees all rows of its dZ: it writes dbias and
// grad_pre.
// 8 waves of 32 columns, BM rows, at most 256 n: half a wave forms a row, so its
// maximum is a reduction over 32 lanes.  (Longer ranges in a loop, with the next
// inputs and codes on their way, took 30 us at 16, 4096, 22016 and 57 at 64, 4096,
// 22016, where k_grad_rows and k_grad_gemm take 27 and 31.)  37 x 4096 x 4096 with
// gelu and bias: 14.2 us a call with its join, 7.6 us for one row; what is left is the
// chain of loads, dZ (formed 16 times, 3 us of gelu's slopes) and 10 MB of sums.
// (The operand in two fp16 parts, its value and the rest of its rounding, takes dX's error
// from 2.9e-4 to its own rounding's 2.1e-4 and costs 5 to 10 %, 37 x 4096 x 4096 15.2 ->
// 16.4 us, as the waves read twice the A from LDS; one part is what k_grad_gemm has.)
// ---------------------------------------------------------------------------
constexpr int kFewRows = 64;      // most rows
constexpr int kFewStages = 4;     // most stages of 64 n in a range
constexpr int kFewN = kFewStages * kGN;

// Inputs of the eight weight rows n .. n+7 (of a pair: of gate or up rows) in
// row t as they are in memory; 0 past the ends.  Buffer loads at an offset
// past the end where there is nothing to read: no branches.
template <bool GATED, int KIND, bool WHOLE>
struct RawRows {
    static constexpr bool kPre = KIND != kNoAct;
    uint32_t d[4], g[kPre ? 4 : 1], u[GATED ? 4 : 1];

    struct Source {
        __amdgpu_buffer_rsrc_t dY, pre;
    };
    static __device__ __forceinline__ Source source(const GradArgs &a)
    {
        const int F = GATED ? a.N >> 1 : a.N;   // (64 rows of 2^21 features at most: offsets fit)
        return {make_rsrc(a.dY, 2 * a.T * F), make_rsrc(a.pre, kPre ? 2 * a.T * a.N : 0)};
    }

    __device__ __forceinline__ void load(const Source &s, const GradArgs &a, int t, int n)
    {
        const int F = GATED ? a.N >> 1 : a.N;
        const bool row = t < a.T;
        if constexpr (WHOLE) {   // (F is a multiple of 8: all of one part)
            const int f = GATED && n >= F ? n - F : n;
            const bool ok = row && n < a.N;
            vec(s.dY, ok ? 2 * (t * F + f) : kOutOfRange, d);
            if constexpr (kPre)
                vec(s.pre, ok ? 2 * (t * a.N + f) : kOutOfRange, g);
            if constexpr (GATED)
                vec(s.pre, ok ? 2 * (t * a.N + F + f) : kOutOfRange, u);
        } else {
            uint32_t h[3][8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const int f = GATED && n + e >= F ? n + e - F : n + e;
                const bool ok = row && n + e < a.N;
                h[0][e] = __builtin_amdgcn_raw_buffer_load_b16(s.dY, ok ? 2 * (t * F + f) : kOutOfRange, 0, 0);
                if constexpr (kPre)
                    h[1][e] = __builtin_amdgcn_raw_buffer_load_b16(s.pre, ok ? 2 * (t * a.N + f) : kOutOfRange, 0, 0);
                if constexpr (GATED)
                    h[2][e] =
                        __builtin_amdgcn_raw_buffer_load_b16(s.pre, ok ? 2 * (t * a.N + F + f) : kOutOfRange, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                d[i] = h[0][2 * i] | h[0][2 * i + 1] << 16;
                if constexpr (kPre)
                    g[i] = h[1][2 * i] | h[1][2 * i + 1] << 16;
                if constexpr (GATED)
                    u[i] = h[2][2 * i] | h[2][2 * i + 1] << 16;
            }
        }
    }

    // dZ of them
    __device__ __forceinline__ void grad(const GradArgs &a, int n, float (&z)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int sh = 16 * (e & 1);
            const float dv = h2f((d[e >> 1] >> sh) & 0xffffu);
            if constexpr (!kPre) {
                z[e] = dv;
            } else {
                float v, s;
                act_value_slope<KIND>(h2f((g[e >> 1] >> sh) & 0xffffu), a.act, v, s);
                if constexpr (GATED)
                    z[e] = n + e >= a.N >> 1 ? dv * v : dv * h2f((u[e >> 1] >> sh) & 0xffffu) * s;
                else
                    z[e] = dv * s;
            }
        }
    }

private:
    static __device__ __forceinline__ void vec(__amdgpu_buffer_rsrc_t r, int off, uint32_t (&w)[4])
    {
        const v4i x = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = (uint32_t)x[i];
    }
};

// Maximum over the 32 lanes of each half of a wave, in every lane of it.
__device__ __forceinline__ uint32_t half_wave_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // half mirror
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));   // row mirror
    const auto r16 = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max((uint32_t)r16[0], (uint32_t)r16[1]);
}

template <bool GATED, int KIND, bool WHOLE, int BM>
__global__ __launch_bounds__(512) void k_grad_few(GradArgs a, const int8_t *__restrict__ Wq, int K,
                                                  int stages, int more, uint16_t *__restrict__ dX,
                                                  float *__restrict__ part, float *__restrict__ dbias)
{
    constexpr int NT = 512, FM = BM / 32, PASSES = BM / 16, KS = kGN / 16;
    constexpr int BSZ = kGN * kGK, ASZ = BM * 128;    // a stage of codes, of A
    constexpr int LB = BSZ / 16 / NT;
    constexpr int oA = kFewStages * BSZ, oSum = oA + kFewStages * ASZ, oRow = oSum + 16 * kFewN * 4;
    __shared__ __attribute__((aligned(1024))) int8_t lds[oRow + BM * 4];
    float *sums = reinterpret_cast<float *>(lds + oSum);   // [16 half waves][256] column sums
    float *unit = reinterpret_cast<float *>(lds + oRow);   // [BM] the rows' units

    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    // range sp of the weight's rows: `stages` stages, one more in the first `more` ranges
    const int tile = blockIdx.x, sp = blockIdx.y, k0 = tile * kGK;
    const int st0 = sp * stages + min(sp, more), ns = stages + (sp < more ? 1 : 0);

    // ---- the weight's codes (as in k_grad_gemm) ----
    const v4i rB = rsrc_words(Wq, a.N * K);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LI8_LDS int8_t *)lds;
    int voB[LB], rowB[LB];
#pragma unroll
    for (int i = 0; i < LB; i++) {
        const int p = i * NT + tid, row = p >> 4, k = k0 + 16 * ((p & 15) ^ (2 * (row & 7)));
        voB[i] = row * K + k;
        rowB[i] = k < K ? a.N - row : 0;
    }
#pragma unroll
    for (int it = 0; it < kFewStages; it++)
        if (it < ns) {
            const int n0 = (st0 + it) * kGN;
#pragma unroll
            for (int i = 0; i < LB; i++)
                load_to_lds_raw(rB, lds0 + (uint32_t)it * BSZ + (i * NT + wid * 64) * 16,
                                n0 < rowB[i] ? voB[i] : kOutOfRange, n0 * K);
        }

    const int half = tid >> 5, l32 = tid & 31;   // half wave 0..15: rows half, half + 16, ...
    v16f acc[FM];
#pragma unroll
    for (int m = 0; m < FM; m++)
        acc[m] = v16f{};
    const int khalf = lane >> 5, arow = lane & 31;
    int offA[KS], offB;
#pragma unroll
    for (int kk = 0; kk < KS; kk++)
        offA[kk] = oA + arow * 128 + (((kk * 2 + khalf) ^ swz_a(arow)) * 16);
    {
        const int r = (lane & 15) >> 1, c = wid * 2 + ((lane >> 4) & 1);
        offB = (8 * khalf + r) * kGK + ((c ^ (2 * r)) * 16) + 8 * (lane & 1);
    }

    using Raw = RawRows<GATED, KIND, WHOLE>;
    Raw raw[PASSES];
    const typename Raw::Source src = Raw::source(a);
    const __amdgpu_buffer_rsrc_t rS = make_rsrc(a.sW, 4 * a.N);
    float w[8];
    // this lane's eight weight rows (past the range: the next workgroup's, none)
    const int n = st0 * kGN + 8 * l32;
    const bool in = 8 * l32 < ns * kGN;
#pragma unroll
    for (int p = 0; p < PASSES; p++)
        raw[p].load(src, a, in ? half + 16 * p : a.T, n);
    {   // (past the last row of the weight: zeros)
        const v4i lo = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rS, in ? 4 * n : kOutOfRange, 0, 0));
        const v4i hi =
            __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rS, in ? 4 * n + 16 : kOutOfRange, 0, 0));
#pragma unroll
        for (int e = 0; e < 4; e++) {
            w[e] = __builtin_bit_cast(float, (int)lo[e]);
            w[4 + e] = __builtin_bit_cast(float, (int)hi[e]);
        }
    }
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; e++)
        sum[e] = 0.0f;
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
        const int t = half + 16 * p;
        uint4 *dst = reinterpret_cast<uint4 *>(lds + oA + (l32 >> 3) * ASZ + t * 128 + (((l32 & 7) ^ swz_a(t)) * 16));
        if (p > 0 && 16 * p >= a.T) {   // (no such rows)
            *dst = make_uint4(0, 0, 0, 0);
            if (l32 == 0)
                unit[t] = 0.0f;
            continue;
        }
        float z[8];
        raw[p].grad(a, n, z);   // (zeros for rows and lanes without inputs)
        if (tile == 0 && a.grad_pre && in && t < a.T)
            store8<WHOLE>(a.grad_pre + (int64_t)t * a.N + n, a.N - n, z);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            sum[e] += z[e];
            z[e] *= w[e];
            m = max(m, __builtin_bit_cast(uint32_t, z[e]) & 0x7fffffffu);
        }
        // scale and unit as in k_grad_rows
        float scale, inverse;
        row_unit(half_wave_max(m), scale, inverse);
        if (l32 == 0)
            unit[t] = inverse;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            z[e] *= scale;
            asm("" : "+v"(z[e]));
        }
        *dst = make_uint4(pack_f16x2(z[0], z[1]), pack_f16x2(z[2], z[3]), pack_f16x2(z[4], z[5]),
                          pack_f16x2(z[6], z[7]));
    }
    const bool cols = tile == 0 && dbias;
    if (cols)
#pragma unroll
        for (int e = 0; e < 8; e++)
            sums[half * kFewN + 8 * l32 + e] = sum[e];
    wait_loads_barrier<0>();   // the codes landed; A, units and sums are there
    if (cols && tid < ns * kGN && st0 * kGN + tid < a.N) {
        float v = 0.0f;
#pragma unroll
        for (int h = 0; h < 16; h++)
            v += sums[h * kFewN + tid];
        dbias[st0 * kGN + tid] = v;
    }
    for (int ss = 0; ss < ns; ss++) {
        const int8_t *b = lds + ss * BSZ + offB;
        v2i codes[KS];
        v8h fa[KS][FM];
#pragma unroll
        for (int kk = 0; kk < KS; kk++) {
            codes[kk] = read_codes_tr(b + kk * 16 * kGK);
#pragma unroll
            for (int m = 0; m < FM; m++)
                fa[kk][m] = *reinterpret_cast<const v8h *>(lds + ss * ASZ + offA[kk] + m * 32 * 128);
        }
#pragma unroll
        for (int kk = 0; kk < KS; kk++) {
            const v8h fb = codes_to_f16(codes[kk]);
#pragma unroll
            for (int m = 0; m < FM; m++)
                acc[m] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb, fa[kk][m], acc[m], 0, 0, 0);
        }
    }

    // acc[m], register r: token arow + 32m, column 32 wid + 8 (r/4) + 4 khalf + r%4 of
    // the tile.  Through LDS, so that the stores are whole lines of a row's 32
    // columns; those of partial sums are non-temporal (what is dirty in the L2
    // when the kernel ends is written back before the next one starts).
    float u[FM];
#pragma unroll
    for (int m = 0; m < FM; m++)
        u[m] = unit[arow + 32 * m];
    lds_barrier();   // codes, A and units are read by all
    int8_t *own = lds + wid * BM * 128;
    static_assert(8 * BM * 128 <= oSum, "staging rows below the sums");
#pragma unroll
    for (int m = 0; m < FM; m++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const int row = arow + 32 * m;
            *reinterpret_cast<v4f *>(own + row * 128 + (((2 * g + khalf) ^ (row & 7)) * 16)) =
                v4f{acc[m][4 * g], acc[m][4 * g + 1], acc[m][4 * g + 2], acc[m][4 * g + 3]} * u[m];
        }
#pragma unroll
    for (int i = 0; i < BM * 8 / 64; i++) {
        const int id = i * 64 + lane, t = id >> 3, k = k0 + 32 * wid + 4 * (id & 7);
        const v4f v = *reinterpret_cast<const v4f *>(own + t * 128 + (((id & 7) ^ (t & 7)) * 16));
        if (t < a.T && k < K) {
            if (part)
                __builtin_nontemporal_store(v, reinterpret_cast<v4f *>(part + ((int64_t)sp * a.T + t) * K + k));
            else
                *reinterpret_cast<uint2 *>(dX + (int64_t)t * K + k) =
                    make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]));
        }
    }
}

// dX = fp16(fac * sum of the parts, in order); fac null: the parts are in dX's
// units; no part (N = 0): zeros.  The workgroups from `blocks` on add dbias'
// strips (none: zeros).
struct Joins {
    const float *part, *fac;
    uint16_t *dX;
    int64_t n;      // elements of dX
    int splits, K;
    int blocks;
    const float *cols;
    float *dbias;
    int strips, N;
};

template <class V>
__device__ __forceinline__ V sum_parts(const float *p, int64_t stride, int parts)
{
    V v = {};
    int s = 0;
    for (; s + 8 <= parts; s += 8) {   // eight loads in flight
        V x[8];
#pragma unroll
        for (int j = 0; j < 8; j++)
            x[j] = *reinterpret_cast<const V *>(p + (s + j) * stride);
#pragma unroll
        for (int j = 0; j < 8; j++)
            v += x[j];
    }
    for (; s < parts; s++)
        v += *reinterpret_cast<const V *>(p + s * stride);
    return v;
}

__global__ __launch_bounds__(256) void k_grad_join(Joins j)
{
    if ((int)blockIdx.x >= j.blocks) {
        const int n = (int)(blockIdx.x - j.blocks) * 256 + threadIdx.x;
        if (n < j.N)
            j.dbias[n] = sum_parts<float>(j.cols + n, j.N, j.strips);
        return;
    }
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= j.n)
        return;
    v4f v = sum_parts<v4f>(j.part + i, j.n, j.splits);
    const float f = j.fac && j.splits ? j.fac[i / j.K] : 1.0f;   // (K is a multiple of 16: one row)
#pragma unroll
    for (int e = 0; e < 4; e++) {
        v[e] *= f;
        asm("" : "+v"(v[e]));
    }
    *reinterpret_cast<uint2 *>(j.dX + i) = make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]));
}

} // namespace

// Which kernels, the tile's rows, and into how many ranges the weight's rows are
// split.
//  - k_grad_few for T <= 64 where its column tiles times the least number of
//    ranges of 256 rows are at most one workgroup per CU: past that every CU
//    forms dZ several times over.  At T, K, N (silu), against k_grad_rows and
//    k_grad_gemm at their best split: 1, 4096, 4096: 7.6 and 9.8 us; 37, 4096,
//    4096: 14.4 and 14.8; 64, 4096, 4096: 17.5 and 18.1; 8, 1024, 1024: 6.2 and
//    8.3; but 8, 11008, 4096: 20.3 and 17.7; 64, 11008, 4096: 40 and 23.
//    At least 8 ranges: 8, 1024, 1024 takes 7.7 us with 4, 6.2 with 8, 6.6 with
//    16; 37, 1024, 2048: 9.8, 10.0 and 11.7 with 8, 16 and 32.
//  - else the tile's rows and the ranges of least modelled time: rounds of
//    workgroups over the 256 CUs, each 4 us and its stages at 1.55, 1.05, 0.65
//    or 0.5 us (tiles of 256, 128, 64, 32 rows: fewer rows use a stage's codes
//    less), and the join of the ranges' sums at 5 TB/s.  At T, K, N, tile / ranges
//    of the model's choice against others: 256, 4096, 4096: 64/4 25.7 us, 128/6
//    26.9, 256/16 39; 1024, 4096, 4096: 64/1 46.9, 128/2 53.4, 256/4 61; 2048,
//    4096, 4096: 128/1 78, 64/1 87, 256/1 90; 3000, 4096, 4096: 256/1 107, 128/1 and
//    64/1 131; 512, 5120, 27648: 256/6 154, 128/3 179.
//  - ranges beyond 32 only while their partial sums are at most 16 MB.
BackwardPlan backward_plan(int64_t T, int64_t K, int64_t N)
{
    const int64_t nst = std::max<int64_t>(1, (N + kGN - 1) / kGN), tk = std::max<int64_t>(1, (K + kGK - 1) / kGK);
    const int64_t most = std::max<int64_t>(kGradSplits, ((int64_t)4 << 20) / std::max<int64_t>(T * K, 1));
    if (T <= kFewRows) {
        const int64_t least = (nst + kFewStages - 1) / kFewStages;
        if (tk * least <= 256 && least <= most)
            return {T <= 32 ? 32 : 64, (int)std::min(std::max<int64_t>(least, 8), nst), true};
    }
    static const struct {
        int bm;
        double stage;
    } kTiles[] = {{256, 1.55}, {128, 1.05}, {64, 0.65}, {32, 0.5}};
    BackwardPlan best{256, 1, false};
    double least = 1e300;
    for (const auto &c : kTiles) {
        // (rows that a tile of half the size holds would leave it half empty; 32 only for few rows)
        if ((c.bm > 64 && T <= c.bm / 2) || (c.bm == 64 && T <= 32) || (c.bm == 32 && T > 32))
            continue;
        const int64_t tiles = (T + c.bm - 1) / c.bm * tk;
        for (int64_t s = 1; s <= std::min<int64_t>({std::max<int64_t>(1, nst / 2), most, 64}); s++) {
            if (s > 1 && tiles * s > 256 + tiles)   // (past one round, more ranges only add sums)
                break;
            const double join = s > 1 ? 3.0 + (double)(s * T * K) * 8.0 / 5.0e6 : 0.0;
            const double cost =
                (double)((tiles * s + 255) / 256) * (4.0 + c.stage * (double)((nst + s - 1) / s)) + join;
            if (cost < least) {
                least = cost;
                best = BackwardPlan{c.bm, (int)s, false};
            }
        }
    }
    return best;
}

// A wave for short rows (a workgroup left most of its threads without work:
// 3621 x 176 x 2 * 135 took 31.8 us a call, 13.3 with waves and the product's
// smaller tile), else a workgroup.  Uneven rows take more registers for their addresses, so
// only up to two rounds of them stay in registers.
RowPlan row_plan(int64_t F)
{
    const int64_t g = (F + 7) / 8, rounds = (g + kRowThreads - 1) / kRowThreads;
    if (g <= 2 * 64)
        return {64, (int)((g + 63) / 64)};
    return {kRowThreads, rounds <= (row_mode((int)F) == MOVED ? 2 : 4) ? (int)rounds : 0};
}

// 512 rows a strip, while that leaves enough workgroups for the chip
int col_strips(int64_t T, int64_t F)
{
    return (int)std::max<int64_t>(1, std::min<int64_t>({kMaxColStrips, (T + 255) / 512, 2048 / ((F + 127) / 128)}));
}

BackwardLayout backward_layout(int64_t T, int64_t K, int64_t N)
{
    const size_t A = 256;
    const BackwardPlan p = backward_plan(T, K, N);
    BackwardLayout L;
    L.Np = (int)((N + kGN - 1) / kGN * kGN);
    size_t off = 0;
    const bool rows = !p.few || K == 0;   // (K = 0: no product, and few rows go the general way)
    const int strips = rows ? col_strips(T, (N + 1) / 2) : 1;   // (a pair's; a single weight has no more)
    L.A = off;     off = align_up(off + (rows ? 2 * (size_t)T * (size_t)L.Np : 0), A);
    L.fac = off;   off = align_up(off + (rows ? 4 * (size_t)T : 0), A);
    L.cols = off;  off = align_up(off + (strips > 1 ? 4 * (size_t)strips * (size_t)N : 0), A);
    L.part = off;  off = align_up(off + (p.splits > 1 ? 4 * (size_t)p.splits * (size_t)T * (size_t)K : 0), A);
    L.total = off;
    return L;
}

namespace {

template <bool GATED, int KIND, int MODE, int TPR, int NR>
void launch_rows_as(const GradArgs &a, const ColSums &c, uint16_t *A, float *fac, hipStream_t s)
{
    const int per = kRowThreads / TPR, rows = std::min((a.T + per - 1) / per, 1 << 20);
    hipLaunchKernelGGL((k_grad_rows<GATED, KIND, MODE, TPR, NR>), dim3((unsigned)(rows + (c.out ? c.blocks * c.strips : 0))),
                       dim3(kRowThreads), 0, s, a, c, A, fac);
}

template <bool GATED, int KIND, int MODE>
void launch_rows_mode(const GradArgs &a, const ColSums &c, const RowPlan &p, uint16_t *A, float *fac, hipStream_t s)
{
    if (p.threads == 64)
        return p.rounds == 1 ? launch_rows_as<GATED, KIND, MODE, 64, 1>(a, c, A, fac, s)
                             : launch_rows_as<GATED, KIND, MODE, 64, 2>(a, c, A, fac, s);
    switch (p.rounds) {
    case 1: return launch_rows_as<GATED, KIND, MODE, kRowThreads, 1>(a, c, A, fac, s);
    case 2: return launch_rows_as<GATED, KIND, MODE, kRowThreads, 2>(a, c, A, fac, s);
    case 0: return launch_rows_as<GATED, KIND, MODE, kRowThreads, 0>(a, c, A, fac, s);
    }
    if constexpr (MODE == EVEN) {
        if (p.rounds == 3)
            launch_rows_as<GATED, KIND, MODE, kRowThreads, 3>(a, c, A, fac, s);
        else
            launch_rows_as<GATED, KIND, MODE, kRowThreads, 4>(a, c, A, fac, s);
    }
}

template <bool GATED, int KIND>
void launch_rows(const GradArgs &a, const ColSums &c, uint16_t *A, float *fac, hipStream_t s)
{
    const int F = GATED ? a.N / 2 : a.N, mode = row_mode(F);
    const RowPlan p = row_plan(F);
    if (mode == SHORT)
        launch_rows_as<GATED, KIND, SHORT, 64, 1>(a, c, A, fac, s);
    else if (mode == MOVED)
        launch_rows_mode<GATED, KIND, MOVED>(a, c, p, A, fac, s);
    else
        launch_rows_mode<GATED, KIND, EVEN>(a, c, p, A, fac, s);
}

// f(integral_constant<int, KIND>) for the call's activation.
template <bool GATED, class F>
void by_kind(const GradArgs &a, F &&f)
{
    if (!GATED && !a.pre)
        f(std::integral_constant<int, GATED ? 0 : kNoAct>{});
    else if (a.act.kind == 0)
        f(std::integral_constant<int, 0>{});
    else if (a.act.kind == 1)
        f(std::integral_constant<int, 1>{});
    else
        f(std::integral_constant<int, 2>{});
}

template <bool GATED, int KIND, bool WHOLE, int BM>
void launch_few_kernel(const GradArgs &a, const int8_t *Wq, int K, const BackwardPlan &p, uint16_t *dX, float *part,
                   float *dbias, hipStream_t s)
{
    const int nst = (a.N + kGN - 1) / kGN, stages = nst / p.splits, more = nst % p.splits;
    const dim3 grid((unsigned)((K + kGK - 1) / kGK), (unsigned)p.splits), block(512);
    part = p.splits > 1 ? part : nullptr;
    hipLaunchKernelGGL((k_grad_few<GATED, KIND, WHOLE, BM>), grid, block, 0, s, a, Wq, K, stages, more, dX, part, dbias);
}

template <bool GATED, int KIND, bool WHOLE>
void launch_few_bm(const GradArgs &a, const int8_t *Wq, int K, const BackwardPlan &p, uint16_t *dX, float *part,
                   float *dbias, hipStream_t s)
{
    if (p.bm == 32)
        launch_few_kernel<GATED, KIND, WHOLE, 32>(a, Wq, K, p, dX, part, dbias, s);
    else
        launch_few_kernel<GATED, KIND, WHOLE, 64>(a, Wq, K, p, dX, part, dbias, s);
}

template <int BM, int NS, int WM, int WN, int GM>
void launch_tiles(const uint16_t *A, const int8_t *Wq, const float *fac, int T, int K, int N, int Np, int splits,
                  uint16_t *dX, float *part, hipStream_t s)
{
    const int tm = (T + BM - 1) / BM, tk = (K + kGK - 1) / kGK;
    const dim3 grid((unsigned)(tm * tk * splits)), block(WM * WN * 64);
    if (splits > 1)
        hipLaunchKernelGGL((k_grad_gemm<BM, NS, WM, WN, GM, true>), grid, block, 0, s, A, Wq, fac, T, K, N, Np, tm, tk,
                           splits, dX, part);
    else
        hipLaunchKernelGGL((k_grad_gemm<BM, NS, WM, WN, GM, false>), grid, block, 0, s, A, Wq, fac, T, K, N, Np, tm, tk,
                           splits, dX, part);
}

void launch_join(Joins j, hipStream_t s)
{
    j.blocks = j.dX ? (int)((j.n / 4 + 255) / 256) : 0;
    const int more = j.dbias ? (j.N + 255) / 256 : 0;
    if (j.blocks + more > 0)
        hipLaunchKernelGGL(k_grad_join, dim3((unsigned)(j.blocks + more)), dim3(256), 0, s, j);
}

} // namespace

hipError_t launch_backward(const uint16_t *dY, const uint16_t *pre, const ActParams &act, bool gated, const int8_t *Wq,
                           const float *sW, int64_t T, int64_t K, int64_t N, uint16_t *dX, uint16_t *grad_pre,
                           float *dbias, char *ws, hipStream_t s)
{
    Joins join{};
    join.n = T * K;
    join.K = (int)K;
    join.N = (int)N;
    if (T == 0 || N == 0) {   // sums of nothing
        join.dX = dX;
        join.dbias = dbias;
        launch_join(join, s);
        return hipGetLastError();
    }
    const BackwardLayout L = backward_layout(T, K, N);
    const BackwardPlan p = backward_plan(T, K, N);
    uint16_t *A = reinterpret_cast<uint16_t *>(ws + L.A);
    float *fac = reinterpret_cast<float *>(ws + L.fac), *part = reinterpret_cast<float *>(ws + L.part);
    const GradArgs a{dY, pre, sW, grad_pre, act, (int)T, (int)N, L.Np};
    const bool few = p.few && K > 0;
    const int features = (int)(gated ? N / 2 : N);
    ColSums c{};
    if (dbias && !few) {
        c.blocks = (features + 127) / 128;
        c.strips = col_strips(T, features);
        c.out = c.strips > 1 ? reinterpret_cast<float *>(ws + L.cols) : dbias;
        if (c.strips > 1) {
            join.cols = c.out;
            join.strips = c.strips;
            join.dbias = dbias;
        }
    }
    const auto pair = [&](auto gated_c) {
        constexpr bool G = decltype(gated_c)::value;
        by_kind<G>(a, [&](auto kind_c) {
            constexpr int KIND = decltype(kind_c)::value;
            if (!few)
                launch_rows<G, KIND>(a, c, A, fac, s);
            else if (features % 8 == 0)
                launch_few_bm<G, KIND, true>(a, Wq, (int)K, p, dX, part, dbias, s);
            else
                launch_few_bm<G, KIND, false>(a, Wq, (int)K, p, dX, part, dbias, s);
        });
    };
    if (gated)
        pair(std::true_type{});
    else
        pair(std::false_type{});
    if (!few && K > 0) {
        const int t = (int)T, k = (int)K, n = (int)N;
        if (p.bm == 256)
            launch_tiles<256, 3, 2, 4, 4>(A, Wq, fac, t, k, n, L.Np, p.splits, dX, part, s);
        else if (p.bm == 128)
            launch_tiles<128, 4, 2, 4, 4>(A, Wq, fac, t, k, n, L.Np, p.splits, dX, part, s);
        else if (p.bm == 64)
            launch_tiles<64, 6, 1, 8, 4>(A, Wq, fac, t, k, n, L.Np, p.splits, dX, part, s);
        else
            launch_tiles<32, 7, 1, 8, 4>(A, Wq, fac, t, k, n, L.Np, p.splits, dX, part, s);
    }
    if (p.splits > 1 && K > 0) {
        join.part = part;
        join.fac = few ? nullptr : fac;
        join.splits = p.splits;
        join.dX = dX;
    }
    launch_join(join, s);
    return hipGetLastError();
}

} // namespace li8
