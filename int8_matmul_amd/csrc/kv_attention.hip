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
//                            probabilities are rounded to it (11 bits; in
//                            two parts 22 bits, or 2^-25 of the largest
//                            where that is more)
// The transposed form leaves a column in the lanes that hold it as the next
// product's operand: with the keys of a step of 32 numbered so that lane
// group g has keys 4g..4g+3 and 16+4g..16+4g+3, the scores' accumulator
// registers are the probabilities' operand registers, and neither goes
// through LDS.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "kv_device.h"
#include "quant_math.h"

namespace li8 {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr float kNone = -1.0e30f;      // a running maximum over nothing yet
constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;
constexpr float kQMax = 16256.0f;      // 127 * 128: the largest 15-bit query integer
// Fewest steps of a workgroup that shares: a part costs its prologue and its
// merge.  With 4, 8 and 16 (us): 8 heads of a group of 8, one token over 1500 keys
// 14.5, 16.1, 18.4, 4000 keys 15.4, 17.3, 19.2, 16000 keys 20.5, 20.6, 19.9; one
// head of 16 over 20000 keys 14.0, 13.7, 14.7; with more steps than 8 for each
// workgroup no difference.
constexpr int kLeastSteps = 8;

struct AttnArgs {
    KvTokens Q;
    KvRope rope;
    uint16_t *O;
    int64_t os;
    float *lse;
    // partial results: [2 part + k][used][D] and [2 part + k][used], k = 0 for
    // the run's first block
    float *part_o, *part_m;
    float scale, inv_group;            // scale * log2(e), 1 / group
    int group, causal, window;
    int cols, blocks, used;
    int seqs, parts;                   // parts: workgroups that share the steps, 0: one per block
};

// Where a workgroup's columns lie.  Column c of a (sequence, head) is row
// c / group, head c % group of the group.
struct Block {
    KvSeq q;
    KvSpan span;
    int s, h, c0, nc;                  // sequence, head, first column, columns
    int i0, g0;                        // row and head of the first column
    // Row of column c0 + k, k < 256, and its head in g.  In fp32 the quotient
    // (g0 + k + 1/2) / group is at most 1 + 255 / group and off by less than
    // 2^-21 of itself, and 1 / (2 group) away from a whole number: its integer
    // part is right for every group below 2^20.
    __device__ __forceinline__ int row_of(int k, const AttnArgs &t, int &g) const
    {
        const int i = (int)(((float)(g0 + k) + 0.5f) * t.inv_group);
        g = g0 + k - i * t.group;
        return i0 + i;
    }
};

// Block cb of sequence s and head h; false where it has no column.
__device__ __forceinline__ bool place(const AttnArgs &t, const KvSeq &q, int s, int h, int cb, int cols, Block &b)
{
    b.s = s;
    b.h = h;
    b.q = q;
    const int64_t ncol = (int64_t)q.n * t.group;
    if ((int64_t)cb * cols >= ncol)
        return false;
    b.c0 = cb * cols;
    b.nc = (int)min((int64_t)cols, ncol - b.c0);
    b.i0 = b.c0 / t.group;
    b.g0 = b.c0 - b.i0 * t.group;
    int g;
    b.span = kv_span(q.begin + b.i0, q.begin + b.row_of(b.nc - 1, t, g), q.len, t.causal != 0, t.window);
    return true;
}

__device__ __forceinline__ bool locate(const KvArgs &a, const AttnArgs &t, int item, int cols, Block &b)
{
    const int cb = item % t.blocks, sh = item / t.blocks, s = sh / a.heads;
    return place(t, kv_sequence_of(a, s), s, sh % a.heads, cb, cols, b);
}

// The work in steps of 2^SHIFT keys, one sequence after another, and within it
// head after head and block after block, each with the sequence's largest
// number of steps (at least one, so that an empty row is written).  `parts` workgroups take equal runs of steps, whatever the
// lengths are: a grid over sequences alone leaves most of the chip to the
// longest one.  Every workgroup, of the merging kernel too, counts the steps
// itself, a lane for each of 64 sequences at a time.  (All counts are below
// 2^30: the host shares no more than that.)
template <int SHIFT>
struct Steps {
    KvSeq q;                           // this lane's sequence
    int steps, blocks;                 // steps of each of its blocks
    int all, upto;                     // its steps, and those of the lanes up to it
    int chunk, base;                   // 64 sequences from 64 chunk on, steps before them

    __device__ __forceinline__ void look(const KvArgs &a, const AttnArgs &t, int c, int lane)
    {
        chunk = c;
        const int s = min(64 * c + lane, t.seqs - 1);
        q = kv_sequence_of(a, s);
        blocks = (int)(((int64_t)q.n * t.group + t.cols - 1) / t.cols);
        int span = q.len;
        if (t.window > 0)
            span = (int)min((int64_t)span, (int64_t)t.window + (t.causal ? t.cols : (int64_t)q.len - q.begin) + 31);
        steps = max(1, (span + (1 << SHIFT) - 1) >> SHIFT);
        all = 64 * c + lane < t.seqs ? a.heads * blocks * steps : 0;
        upto = all;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int y = __shfl_up(upto, d, 64);
            upto += lane >= d ? y : 0;
        }
    }

    // Steps of a workgroup, and of all; chunk 0 is looked at afterwards.
    __device__ __forceinline__ int share(const KvArgs &a, const AttnArgs &t, int lane, int &total)
    {
        total = 0;
        for (int c = (t.seqs - 1) >> 6; c >= 0; c--) {
            look(a, t, c, lane);
            total += __builtin_amdgcn_readlane(upto, 63);
        }
        base = 0;
        return max(kLeastSteps, (total + t.parts - 1) / t.parts);
    }

    // The lane whose sequence has step `at` (at < total, not before `base`).
    __device__ __forceinline__ int find(const KvArgs &a, const AttnArgs &t, int at, int lane)
    {
        while (true) {
            const uint64_t over = __ballot(base + upto > at);
            if (over)
                return __ffsll((unsigned long long)over) - 1;
            base += __builtin_amdgcn_readlane(upto, 63);
            look(a, t, chunk + 1, lane);
        }
    }

    __device__ __forceinline__ KvSeq seq_of(int k) const
    {
        KvSeq r;
        r.q0 = __builtin_amdgcn_readlane(q.q0, k);
        r.n = __builtin_amdgcn_readlane(q.n, k);
        r.len = __builtin_amdgcn_readlane(q.len, k);
        r.begin = __builtin_amdgcn_readlane(q.begin, k);
        return r;
    }
};

// The blocks of one workgroup's run of steps, one after another: block b,
// steps first .. first + count - 1 of it, and the slot of its partial result.
// A run's first block goes to the run's slot 0, a later one that it does not
// finish to slot 1, and one that is all its own to O (-1).
// Without KEEP the sequences are looked at anew for each block, and the lanes
// hold nothing of them in between.
template <int SHIFT, bool KEEP>
struct Run {
    Steps<SHIFT> w;
    int part, begin, at, end, chunk, base;

    __device__ __forceinline__ bool start(const KvArgs &a, const AttnArgs &t, int run, int lane)
    {
        int total;
        part = run;
        const int per = __builtin_amdgcn_readfirstlane(w.share(a, t, lane, total));
        const int64_t b = (int64_t)run * per;
        if (b >= total)
            return false;
        begin = at = (int)b;
        end = (int)min(b + per, (int64_t)total);
        chunk = base = 0;
        return true;
    }

    // false: the block has no column (its steps are passed over)
    __device__ __forceinline__ bool next(const KvArgs &a, const AttnArgs &t, int cols, int lane, Block &b, int &first,
                                         int &count, int64_t &slot)
    {
        if constexpr (!KEEP) {
            w.look(a, t, chunk, lane);
            w.base = base;
        }
        const int k = __builtin_amdgcn_readfirstlane(w.find(a, t, at, lane));
        chunk = __builtin_amdgcn_readfirstlane(w.chunk);
        base = __builtin_amdgcn_readfirstlane(w.base);
        const int steps = __builtin_amdgcn_readlane(w.steps, k), blocks = __builtin_amdgcn_readlane(w.blocks, k);
        const int r = at - base - __builtin_amdgcn_readlane(w.upto - w.all, k);
        const int unit = r / steps, h = unit / blocks, cb = unit - h * blocks;
        first = r - unit * steps;
        count = min(steps - first, end - at);
        slot = count == steps ? -1 : 2 * (int64_t)part + (at == begin ? 0 : 1);
        at += count;
        return place(t, w.seq_of(k), 64 * chunk + k, h, cb, cols, b);
    }
};

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), cd = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    return ab | cd;
}

// Two chunks of 8 values of a row and what their rotation takes.  Rotated by
// halves a lane has both values of its pairs, so that the tables' numbers and
// the partners are loaded once; else the chunks are neighbours.
struct RowPair {
    uint4 x[2];
    float4 c[2], s[2];
};

// The chunks of lane l.
template <int ROT>
__device__ __forceinline__ void pair_chunks(int l, const KvRope &r, int (&c)[2])
{
    const int hc = r.half >> 3;
    const bool turned = ROT == ROT_HALVES && l < hc;
    c[0] = turned ? l : 2 * l;
    c[1] = turned ? l + hc : 2 * l + 1;
}

template <int ROT>
__device__ __forceinline__ void fetch_pair(RowPair &w, const uint16_t *row, int l, const int (&c)[2], const KvRope &r,
                                           int pos)
{
    w.x[0] = load_u4(row + 8 * c[0]);
    w.x[1] = load_u4(row + 8 * c[1]);
    if constexpr (ROT != ROT_NONE) {   // (a chunk past the rotated values: the row's first numbers)
        const int64_t t = (int64_t)pos * r.half + (8 * l < r.half ? 8 * l : 0);
        const float4 *pc = reinterpret_cast<const float4 *>(r.cos + t);
        const float4 *ps = reinterpret_cast<const float4 *>(r.sin + t);
        w.c[0] = pc[0]; w.c[1] = pc[1];
        w.s[0] = ps[0]; w.s[1] = ps[1];
    }
}

// The rotated values; each product and sum is rounded by itself, as the keys' are.
template <bool BF16, int ROT>
__device__ __forceinline__ void rotate_pair(const RowPair &w, int l, const KvRope &r, float (&x)[16])
{
    unpack8<BF16>(w.x[0], x);
    unpack8<BF16>(w.x[1], x + 8);
    if constexpr (ROT != ROT_NONE) {
        const bool turned = 8 * l < r.half;
        const float cv[8] = {w.c[0].x, w.c[0].y, w.c[0].z, w.c[0].w, w.c[1].x, w.c[1].y, w.c[1].z, w.c[1].w};
        const float sv[8] = {w.s[0].x, w.s[0].y, w.s[0].z, w.s[0].w, w.s[1].x, w.s[1].y, w.s[1].z, w.s[1].w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float &a = x[ROT == ROT_HALVES ? i : 2 * i], &b = x[ROT == ROT_HALVES ? 8 + i : 2 * i + 1];
            const float za = a * cv[i] - b * sv[i], zb = b * cv[i] + a * sv[i];
            a = turned ? za : a;
            b = turned ? zb : b;
        }
    }
}

// N query values of a row as two int8 parts; f is the factor of the row's
// integers, without the softmax scale.  LANES neighbours have a row.
template <int LANES, int N>
__device__ __forceinline__ void split_query(const float (&x)[N], uint2 (&hi)[N / 8], uint2 (&lo)[N / 8], float &f)
{
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < N; e++)
        m = fmaxf(m, fabsf(x[e]));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1)
        m = fmaxf(m, __shfl_xor(m, o, 64));
    // x inv in [-16256, 16256] plus 1.5 2^23 is rounded half to even to an
    // integer n in the low bits: n = 128 qh + ql, qh = n >> 7 in -127 .. 127,
    // ql = n & 127.  (For the least subnormal rows inv is cut to what fp32
    // holds, which only makes n smaller.)
    const float inv = m > 0.0f ? fminf(kQMax * __builtin_amdgcn_rcpf(m), FLT_MAX) : 0.0f;
    f = inv > 0.0f ? 1.0f / inv : 0.0f;
#pragma unroll
    for (int k = 0; k < N / 8; k++) {
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; e++)
            b[e] = __builtin_bit_cast(uint32_t, fmaf(x[8 * k + e], inv, 12582912.0f));
        lo[k] = make_uint2(low_bytes(b[0], b[1], b[2], b[3]) & 0x7f7f7f7fu,
                           low_bytes(b[4], b[5], b[6], b[7]) & 0x7f7f7f7fu);
#pragma unroll
        for (int e = 0; e < 8; e++)
            b[e] >>= 7;
        hi[k] = make_uint2(low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7]));
    }
}

// The block's query columns into LDS, COLS rows of LQ bytes with the first
// parts and as many with the second, and their factors.  between() runs once
// the rows have been requested.  PAIR: two chunks per lane, which take half
// the loads of a rotation (256 columns: 8.7 us with one chunk, a 4096-token
// prompt 168 -> 163 us); with few columns one, as half the lanes would idle
// (64 sequences' one token each 126 against 128 us).
template <int D, bool BF16, int COLS, int NT, int LQ, bool PAIR, class Between>
__device__ __forceinline__ void split_queries(const KvArgs &a, const AttnArgs &t, const Block &b, char *lds,
                                              float *factor, int tid, Between between)
{
    constexpr int N = PAIR ? 16 : 8, LPR = D / N;   // values of a lane, lanes of a row
    constexpr int PASSES = COLS * LPR / NT > 0 ? COLS * LPR / NT : 1;
    static_assert(PASSES <= 4, "rows in flight");
    const int l = tid % LPR;
    with_rotation(t.rope, [&](auto rot) {
        constexpr int ROT = decltype(rot)::value;
        int c[2] = {l, l};
        if constexpr (PAIR)
            pair_chunks<ROT>(l, t.rope, c);
        std::conditional_t<PAIR, RowPair, RowChunk> w[PASSES];
#pragma unroll
        for (int k = 0; k < PASSES; k++) {
            int g;   // (columns past the last: the last one again)
            const int qc = min(tid / LPR + k * (NT / LPR), b.nc - 1);
            const int i = b.row_of(qc, t, g), pos = max(b.q.begin + i, 0);
            const uint16_t *row =
                t.Q.p + (int64_t)(b.q.q0 + i) * t.Q.stride + (int64_t)(b.h * t.group + g) * D;
            if constexpr (PAIR)
                fetch_pair<ROT>(w[k], row, l, c, t.rope, pos);
            else
                fetch_row<ROT>(w[k], row, l, t.rope, pos);
        }
        between();
#pragma unroll
        for (int k = 0; k < PASSES; k++) {
            const int qc = tid / LPR + k * (NT / LPR);
            float x[N], f;
            uint2 hi[N / 8], lo[N / 8];
            if constexpr (PAIR)
                rotate_pair<BF16, ROT>(w[k], l, t.rope, x);
            else
                rotate_row<BF16, ROT>(w[k], l, t.rope, x);
            split_query<LPR, N>(x, hi, lo, f);
            if (COLS * LPR < NT && qc >= COLS)
                continue;
#pragma unroll
            for (int j = 0; j < N / 8; j++) {
                *reinterpret_cast<uint2 *>(lds + qc * LQ + 8 * c[j]) = hi[j];
                *reinterpret_cast<uint2 *>(lds + (COLS + qc) * LQ + 8 * c[j]) = lo[j];
            }
            if (l == 0)
                factor[qc] = f * t.scale;
        }
    });
}

// Codes of one byte of two keys' words as fp16.  0x6400 | u is 1024 + u for a
// byte u; with the code's sign bit flipped u is code + 128, so 1152 less is the
// code, exactly.
template <int BYTE>
__device__ __forceinline__ uint32_t codes_f16(uint32_t a, uint32_t b)
{
    const uint32_t w = __builtin_amdgcn_perm(b, a, 0x0c000c00u | BYTE | ((4 + BYTE) << 16)) ^ 0x64806480u;
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

// Read-only data at addresses that are the same for a whole wave: scalar loads.
typedef const int32_t __attribute__((address_space(4))) *kv_const_i32;
typedef const float __attribute__((address_space(4))) *kv_const_f32;

template <class T, bool NT>
__device__ __forceinline__ T load_as(const int8_t *p)
{
    if constexpr (NT)
        return __builtin_nontemporal_load(reinterpret_cast<const T *>(p));
    return *reinterpret_cast<const T *>(p);
}

template <int D, bool NT>
__device__ __forceinline__ void load_step(Step<D> &st, const KvArgs &a, const int (&pid)[2], int h, int t0,
                                          int lo, int te, uint32_t koff, uint32_t voff)
{
    const int page = 1 << a.page_shift;
#pragma unroll
    for (int tt = 0; tt < 2; tt++) {
        const int t = t0 + 16 * tt;
        // a tile past the end, before the first key seen or in no page is
        // masked; page 0 is read in its place
        st.ok[tt] = (unsigned)pid[tt] < (unsigned)a.pages && t < te && t + 16 > lo;
        const int64_t ph = (int64_t)(st.ok[tt] ? pid[tt] : 0) * a.heads + h;
        const int64_t base = ((ph * D) << a.page_shift) + (t & (page - 1)) * D;
        const int8_t *kp = a.k + base + koff;
        const int8_t *vp = a.v + base + voff;
#pragma unroll
        for (int ks = 0; ks < D / 64; ks++)
            st.k[tt][ks] = load_as<v4i, NT>(kp + 64 * ks);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if constexpr (D == 128) {
                const v2u w = load_as<v2u, NT>(vp + j * D);
                st.v[4 * tt + j][0] = w.x;
                st.v[4 * tt + j][D / 64 - 1] = w.y;
            } else {
                st.v[4 * tt + j][0] = load_as<uint32_t, NT>(vp + j * D);
            }
        }
        const float ksc = ((kv_const_f32)(uintptr_t)a.ks)[ph], vsc = ((kv_const_f32)(uintptr_t)a.vs)[ph];
        st.ks[tt] = st.ok[tt] ? ksc : 0.0f;
        st.vs[tt] = st.ok[tt] ? vsc : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// Few columns: 16 NC columns of one (sequence, head) and a run of its keys per
// workgroup; the NW waves take the steps of 32 keys in turn and keep their own
// maximum, sum and O^T, merged through LDS at the end.  K and V go from memory
// into the MFMA operands' registers, V through a byte transpose (4 keys x 4
// dims by v_perm), and a step is requested while the one before is computed
// (two and three steps ahead were slower: registers, and no fewer waits).
// Bound by reading the cache once: 64 sequences of up to 8192 tokens, 8 heads
// of a group of 8, one token each, 701 MB: 127 us with the merge, 5.5 TB/s (a
// copy of 2 GiB moves 5.0, read and written); one sequence of 131071 tokens,
// 268 MB: 51 us.  (Several such caches in turn, so that none of it is in the
// Infinity Cache: 1 % more.  fp16 and bf16 take the same.)
// Short calls are bound by the chain of loads (lengths, page number, step) and
// the launch: one token of 32 heads over 777 keys 11.9 us.
// ---------------------------------------------------------------------------
template <int D, bool BF16, int NC, int NW, bool NT>
__device__ __forceinline__ void few_block(const KvArgs &a, const AttnArgs &t, const Block &b, int ts, int te,
                                          int64_t slot, char *smem, float *s_f, float *s_m, float *s_l)
{
    constexpr int CPR = D / 8, NB = D / 16, KS = D / 64, LQ = D + 16, LO = D + 4, COLS = kKvCols * NC;
    constexpr int kStride = 32 * NW;
    // fp16 outputs: the probabilities in two parts, so that only the output's
    // own rounding shows (error 2.2e-4 of the output's norm against 2.9e-4,
    // 2.1e-4 of it from that rounding).  22 bits for probabilities of 2^-3 of
    // the maximum and more; the second part of smaller ones is subnormal and
    // off by 2^-25 of it, which leaves 14 bits of a probability of 2^-10.  One token of 40 heads x 16
    // sequences takes 89.3 us either way, as reading the cache hides the
    // second product; one token of 32 heads over 1000 keys 11.9 against 11.3.
    // With 32 columns a workgroup is bound by its instructions (a prompt of
    // 1024 tokens 47 us against 41), and bf16 outputs are rounded 8 times as
    // coarsely: one part.
    constexpr bool TWO = !BF16 && NC == 1;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const kv_const_i32 table = (kv_const_i32)(uintptr_t)(a.table + (int64_t)b.s * a.table_stride);
    const int col = lane & 15, g = lane >> 4;
    const uint32_t koff = col * D + 16 * g, voff = 4 * g * D + col * (D / 16);
    auto pages = [&](int (&pid)[2], int t0) {
        pid[0] = table[min(t0 >> a.page_shift, a.table_width - 1)];
        pid[1] = table[min((t0 + 16) >> a.page_shift, a.table_width - 1)];
    };
    int t0 = ts + 32 * wid, pid[2];
    Step<D> st[2];
    const bool any = t0 < te;
    // the queries and the first step's data are requested together
    if (any)
        pages(pid, t0);
    split_queries<D, BF16, COLS, 64 * NW, LQ, false>(a, t, b, smem, s_f, tid, [&]() {
        if (any) {
            load_step<D, NT>(st[0], a, pid, b.h, t0, b.span.lo, te, koff, voff);
            pages(pid, t0 + kStride);
        }
    });
    __syncthreads();
    v4i qh[NC][KS], ql[NC][KS];
    float f[NC];
    int chi[NC], clo[NC];              // keys this lane's columns see: [clo, chi)
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int qc = kKvCols * c + col;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
            qh[c][ks] = *reinterpret_cast<const v4i *>(smem + qc * LQ + 64 * ks + 16 * g);
            ql[c][ks] = *reinterpret_cast<const v4i *>(smem + (COLS + qc) * LQ + 64 * ks + 16 * g);
        }
        f[c] = s_f[qc];
        int gcol;
        const int pos = b.q.begin + b.row_of(qc, t, gcol);
        chi[c] = qc >= b.nc ? 0 : t.causal ? min(te, pos + 1) : te;
        clo[c] = t.window > 0 ? max((int64_t)0, (int64_t)pos + 1 - t.window) : 0;
    }
    __syncthreads();                   // smem is used again below

    v4f acc[NC][NB] = {};
    float m[NC], l[NC], vref = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        m[c] = kNone;
        l[c] = 0.0f;
    }
    auto compute = [&](const Step<D> &w, int t0) {
        // value scales relative to the largest so far, so that the operand
        // stays in fp16's range whatever the scales are
        const float vm = fmaxf(w.vs[0], w.vs[1]);
        if (vm > vref) {
            const float al = vref / vm;
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int n = 0; n < NB; n++)
                    acc[c][n] *= al;
            vref = vm;
        }
        // (below the normal range the reciprocal is infinite: such scales count as 0)
        const float vi = vref >= FLT_MIN ? __builtin_amdgcn_rcpf(vref) : 0.0f;
        const float r[2] = {w.vs[0] * vi, w.vs[1] * vi};
        v8h p[NC], rest[TWO ? NC : 1];
#pragma unroll
        for (int c = 0; c < NC; c++) {
            float z[8], zm = -INFINITY;
#pragma unroll
            for (int tt = 0; tt < 2; tt++) {
                v4i sh = {0, 0, 0, 0}, sl = {0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < KS; ks++) {
                    sh = __builtin_amdgcn_mfma_i32_16x16x64_i8(w.k[tt][ks], qh[c][ks], sh, 0, 0, 0);
                    sl = __builtin_amdgcn_mfma_i32_16x16x64_i8(w.k[tt][ks], ql[c][ks], sl, 0, 0, 0);
                }
                const float fk = f[c] * w.ks[tt];
                const int key = t0 + 16 * tt + 4 * g, hi = w.ok[tt] ? chi[c] : 0;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float v = (float)((sh[i] << 7) + sl[i]) * fk;
                    z[4 * tt + i] = key + i < hi && key + i >= clo[c] ? v : -INFINITY;
                    zm = fmaxf(zm, z[4 * tt + i]);
                }
            }
            // The maximum is moved only when some score is 8 above it (in
            // powers of two): until then the probabilities stay below 2^8,
            // and neither O^T nor the sum has to be scaled.
            if (__any(zm > m[c] + 8.0f)) {
                zm = fmaxf(zm, __shfl_xor(zm, 16, 64));
                zm = fmaxf(zm, __shfl_xor(zm, 32, 64));
                const float mn = fmaxf(m[c], zm), al = __builtin_amdgcn_exp2f(m[c] - mn);
#pragma unroll
                for (int n = 0; n < NB; n++)
                    acc[c][n] *= al;
                l[c] *= al;
                m[c] = mn;
            }
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float pe = __builtin_amdgcn_exp2f(z[e] - m[c]);
                l[c] += pe;
                const float w = pe * r[e >> 2];
                p[c][e] = (_Float16)w;
                if constexpr (TWO)
                    rest[c][e] = (_Float16)(w - (float)p[c][e]);
            }
        }
        // Lane (col, g) has the bytes col NB .. col NB + NB - 1 of its 8 keys:
        // operand n is dim col NB + n of all of them.
#pragma unroll
        for (int d = 0; d < KS; d++) {
            v4u x0, x1, x2, x3;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x0[j] = codes_f16<0>(w.v[2 * j][d], w.v[2 * j + 1][d]);
                x1[j] = codes_f16<1>(w.v[2 * j][d], w.v[2 * j + 1][d]);
                x2[j] = codes_f16<2>(w.v[2 * j][d], w.v[2 * j + 1][d]);
                x3[j] = codes_f16<3>(w.v[2 * j][d], w.v[2 * j + 1][d]);
            }
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const v8h x[4] = {__builtin_bit_cast(v8h, x0), __builtin_bit_cast(v8h, x1),
                                  __builtin_bit_cast(v8h, x2), __builtin_bit_cast(v8h, x3)};
#pragma unroll
                for (int n = 0; n < 4; n++)
                    acc[c][4 * d + n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[n], p[c], acc[c][4 * d + n], 0, 0, 0);
                if constexpr (TWO) {
#pragma unroll
                    for (int n = 0; n < 4; n++)
                        acc[c][4 * d + n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[n], rest[c], acc[c][4 * d + n], 0, 0, 0);
                }
            }
        }
    };
    // (a step past the end is requested all the same, masked, from page 0)
    if (any) {
        while (true) {
            load_step<D, NT>(st[1], a, pid, b.h, t0 + kStride, b.span.lo, te, koff, voff);
            pages(pid, t0 + 2 * kStride);
            __builtin_amdgcn_sched_barrier(0);
            compute(st[0], t0);
            t0 += kStride;
            if (t0 >= te)
                break;
            load_step<D, NT>(st[0], a, pid, b.h, t0 + kStride, b.span.lo, te, koff, voff);
            pages(pid, t0 + 2 * kStride);
            __builtin_amdgcn_sched_barrier(0);
            compute(st[1], t0);
            t0 += kStride;
            if (t0 >= te)
                break;
        }
    }

    // Accumulator n of lane (col, g) holds O^T[(4g + i) NB + n][col], i < 4.
#pragma unroll
    for (int c = 0; c < NC; c++) {
        l[c] += __shfl_xor(l[c], 16, 64);
        l[c] += __shfl_xor(l[c], 32, 64);
        float *so = reinterpret_cast<float *>(smem) + (wid * COLS + kKvCols * c + col) * LO;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int n = 0; n < NB; n += 4) {
                const v4f o = {acc[c][n][i] * vref, acc[c][n + 1][i] * vref, acc[c][n + 2][i] * vref,
                               acc[c][n + 3][i] * vref};
                *reinterpret_cast<v4f *>(so + (4 * g + i) * NB + n) = o;
            }
        if (g == 0) {
            s_m[wid * COLS + kKvCols * c + col] = m[c];
            s_l[wid * COLS + kKvCols * c + col] = l[c];
        }
    }
    __syncthreads();
    for (int qc = tid / CPR; qc < b.nc; qc += 64 * NW / CPR) {
        const int cc = tid % CPR;
        float M = kNone, L = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; w++)
            M = fmaxf(M, s_m[w * COLS + qc]);
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const float al = __builtin_amdgcn_exp2f(s_m[w * COLS + qc] - M);
            const float *src = reinterpret_cast<const float *>(smem) + (w * COLS + qc) * LO + 8 * cc;
            L += s_l[w * COLS + qc] * al;
#pragma unroll
            for (int e = 0; e < 8; e++)
                o[e] += src[e] * al;
        }
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e++)
            o[e] *= inv;
        if (slot >= 0) {
            const int64_t at = slot * t.used + qc;
            float *po = t.part_o + at * D + 8 * cc;
            *reinterpret_cast<float4 *>(po) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4 *>(po + 4) = make_float4(o[4], o[5], o[6], o[7]);
            if (cc == 0)
                t.part_m[at] = L > 0.0f ? M + log2f(L) : kNone;
            continue;
        }
        int gq;
        const int i = b.row_of(qc, t, gq);
        const int64_t row = b.q.q0 + i;
        const int head = b.h * t.group + gq;
        *reinterpret_cast<uint4 *>(t.O + row * t.os + (int64_t)head * D + 8 * cc) = pack8<BF16>(o);
        if (t.lse && cc == 0)
            t.lse[row * (int64_t)(a.heads * t.group) + head] = L > 0.0f ? (M + log2f(L)) * kLn2 : -INFINITY;
    }
}

template <int D, bool BF16, int NC, int NW, bool NT>
__global__ __launch_bounds__(64 * NW, 2) void k_kv_few(KvArgs a, AttnArgs t)
{
    constexpr int COLS = kKvCols * NC;
    __shared__ __align__(16) char smem[NW * COLS * (D + 4) * 4];
    __shared__ float s_f[COLS], s_m[NW * COLS], s_l[NW * COLS];
    Block b;
    if (t.parts == 0) {
        // (a prompt's last blocks, which see the most keys, first)
        const int cb = blockIdx.x % t.blocks;
        if (locate(a, t, blockIdx.x - cb + (t.blocks - 1 - cb), COLS, b))
            few_block<D, BF16, NC, NW, NT>(a, t, b, b.span.base, b.span.hi, -1, smem, s_f, s_m, s_l);
        return;
    }
    const int lane = threadIdx.x & 63;
    Run<5, true> run;
    if (!run.start(a, t, blockIdx.x, lane))
        return;
    while (run.at < run.end) {
        int first, count;
        int64_t slot;
        if (run.next(a, t, COLS, lane, b, first, count, slot)) {
            const int ts = b.span.base + 32 * first;
            few_block<D, BF16, NC, NW, NT>(a, t, b, ts, min(b.span.hi, ts + 32 * count), slot, smem, s_f, s_m, s_l);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Many columns: 32 columns per wave, kTileWaves waves; the workgroup walks
// its keys in steps of 64 that all waves read from LDS.  K stays int8 there
// (16 MFMAs 32x32x32 i8 per step and wave for the two query parts), V is
// turned into fp16 and transposed on its way in, once for all waves.
// A prompt of 4096 tokens, 32 heads, D = 128: 166 us, 830 TFLOP/s by the
// formula's products (158 to 168 on four boards); a chunk of 512 tokens in each
// of 4 sequences of 8192, 8 heads of a group of 8: 548 us, 1000 TFLOP/s.  (In
// bursts of 8 calls, while the clock ramps up, 185 and 670 us.)  The matrix
// units are busy for a third of the time and the vector ALUs for half of it;
// with the exponentials left out, or the staging, or the reads of LDS, or the
// second product, the time falls by 11, 10, 5 and 10 % at the prompt (by 14, 16,
// 11 and 15 % at the chunks), so no one of them alone is the bound.
// ---------------------------------------------------------------------------
constexpr int kTileWaves = 8;
constexpr int kTileCols = 32 * kTileWaves;
constexpr int kTileKeys = 64;
// log2 of the smallest relative value scale.  Smaller ones, 0 among them, are
// taken as it: 2^-60 of the others' values, nothing that fp16 holds.  Their
// weights come back into the sum from 2^(z - m - 60), so that what the
// exponential drops below 2^-126 is below 2^-66 of the maximum (from -100 on
// weights below 2^-26 were lost, 1.4e-3 of a sum over 131071 keys).
constexpr float kLeast = -60.0f;
constexpr float kMost = 8192.0f;       // largest sum of 8 probabilities taken as it is

typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));

// 16-byte chunks of the LDS tiles are permuted within 128 bytes so that
// neither the fragment reads (one chunk of 16 rows at a time) nor the writes
// of V (rows 4 apart) meet in a bank: a ninth of the LDS's busy cycles are
// conflicts (a quarter with row & 7 for K: 0.6 % more time).
template <int D>
__device__ __forceinline__ int k_place(int row, int chunk)
{
    if constexpr (D == 128)
        return row * 128 + 16 * (chunk ^ ((row ^ ((row >> 3) & 1)) & 7));
    return row * 64 + 16 * (chunk ^ (((row >> 1) ^ (row >> 3)) & 3));
}

__device__ __forceinline__ int v_place(int d, int chunk) { return d * 128 + 16 * (chunk ^ ((d ^ (d >> 3)) & 7)); }

template <int D>
struct TileLds {
    static constexpr int K = kTileKeys * D, V = D * kTileKeys * 2;
    static constexpr int stage = K + V;
    static constexpr int q_row = D + 16;
    static constexpr int bytes = 3 * stage > 2 * kTileCols * q_row ? 3 * stage : 2 * kTileCols * q_row;
};

template <int D, bool BF16>
__device__ __forceinline__ void tile_block(const KvArgs &a, const AttnArgs &t, const Block &b, int ts, int te,
                                           int64_t slot, char *smem, float *s_f, float (*s_sc)[4][4])
{
    constexpr int NT = 64 * kTileWaves, KS = D / 32, DB = D / 32;
    constexpr int ITEMS = kTileKeys * D / 16;   // pieces to stage, at most one for each thread
    static_assert(ITEMS <= NT && ITEMS % 256 == 0, "staging");
    using L = TileLds<D>;
    // (read anew for each block: what follows from it would be kept in
    // registers from block to block, which there are none for)
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    split_queries<D, BF16, kTileCols, NT, L::q_row, true>(a, t, b, smem, s_f, tid, []() {});
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
    // wave see, [wlo, whi), or any of them (seen)
    int gcol, gdrop;
    const int pos = b.q.begin + b.row_of(qcol, t, gcol);
    int chi = t.causal ? min(te, pos + 1) : te;
    int clo = t.window > 0 ? max((int64_t)0, (int64_t)pos + 1 - t.window) : 0;
    if (qcol >= b.nc)
        chi = clo = 0;
    const int c_first = 32 * wid, c_last = min(32 * wid + 31, b.nc - 1);
    const int p_first = b.q.begin + b.row_of(c_first, t, gdrop);
    const int p_last = b.q.begin + b.row_of(max(c_last, 0), t, gdrop);
    const KvSpan seen = kv_span(p_first, p_last, te, t.causal != 0, t.window);
    const bool idle = c_first >= b.nc;
    const int whi = c_last < 32 * wid + 31 ? 0 : t.causal ? min(te, p_first + 1) : te;
    const int wlo = t.window > 0 ? max((int64_t)0, (int64_t)p_last + 1 - t.window) : 0;

    // Staging: a wave's 16-byte pieces of K and its 4 x 4 blocks of V lie in
    // one group of 16 keys, so in one page: the page's address is the wave's,
    // in scalar registers.  Page numbers are requested two steps ahead of the
    // data that they address, the data one step ahead of the step that uses
    // it.  (Page numbers and scales are asked for with a lane's offset of 0,
    // as vector loads: a scalar load in flight makes every read of LDS wait
    // for it, since the two count together and end in any order.)
    int zero;
    asm("v_mov_b32 %0, 0" : "=v"(zero));
    const int32_t *table = a.table + (int64_t)b.s * a.table_stride;
    const int it = tid % ITEMS, group = wid * 64 % ITEMS / (ITEMS / 4);
    const int krow = it / (D / 16), kchunk = it % (D / 16), dg = it % (D / 4), sb = it / (D / 4);
    const uint32_t koff = (krow & 15) * D + 16 * kchunk, voff = 4 * (sb & 3) * D + 4 * dg;
    const int kput = k_place<D>(krow, kchunk);
    // 4 keys x 4 dims: quarter q = sb % 4 of a group of 16 keys is part q / 2
    // of the chunk that half q % 2 reads
    int vput = L::K + v_place(4 * dg, 2 * (sb >> 2) + (sb & 1)) + 8 * ((sb >> 1) & 1);
    uint4 rk;
    uint32_t rv[4];
    float rks = 0.0f, rvs = 0.0f;
    bool rok = false;
    int vpid = 0;
    auto pages = [&](int t0) { vpid = table[min((t0 + 16 * group) >> a.page_shift, a.table_width - 1) + zero]; };
    auto load = [&](int t0) {
        const int pid = __builtin_amdgcn_readfirstlane(vpid), key = t0 + 16 * group;
        rok = (unsigned)pid < (unsigned)a.pages && key < te && key + 16 > b.span.lo;
        const int64_t ph = (int64_t)(rok ? pid : 0) * a.heads + b.h;
        const int64_t at = ((ph * D) << a.page_shift) + (key & ((1 << a.page_shift) - 1)) * D;
        rk = *reinterpret_cast<const uint4 *>(a.k + at + koff);
#pragma unroll
        for (int e = 0; e < 4; e++)
            rv[e] = *reinterpret_cast<const uint32_t *>(a.v + at + e * D + voff);
        rks = a.ks[ph + zero];
        rvs = a.vs[ph + zero];
    };
    auto store = [&](int buf) {
        if (ITEMS < NT && tid >= ITEMS)
            return;
        const int at = buf * L::stage;
        asm("" : "+v"(vput));
        *reinterpret_cast<uint4 *>(smem + at + kput) = rk;
        *reinterpret_cast<uint2 *>(smem + (at + vput)) =
            make_uint2(codes_f16<0>(rv[0], rv[1]), codes_f16<0>(rv[2], rv[3]));
        *reinterpret_cast<uint2 *>(smem + ((at + vput) ^ 16) + 128) =
            make_uint2(codes_f16<1>(rv[0], rv[1]), codes_f16<1>(rv[2], rv[3]));
        *reinterpret_cast<uint2 *>(smem + ((at + vput) ^ 32) + 256) =
            make_uint2(codes_f16<2>(rv[0], rv[1]), codes_f16<2>(rv[2], rv[3]));
        *reinterpret_cast<uint2 *>(smem + ((at + vput) ^ 48) + 384) =
            make_uint2(codes_f16<3>(rv[0], rv[1]), codes_f16<3>(rv[2], rv[3]));
        if (lane == 0) {   // (the waves of a group write the same)
            // no such page: a factor of 0, and -inf added to every score
            *reinterpret_cast<v4f *>(s_sc[buf][group]) =
                rok ? v4f{rks, __builtin_amdgcn_logf(rvs), 0.0f, 0.0f} : v4f{0.0f, -INFINITY, -INFINITY, 0.0f};
        }
    };

    // The wave's part of the steps: those that any of its columns sees.
    const int steps = ts < te ? (te - ts + kTileKeys - 1) / kTileKeys : 0;
    const bool some = !idle && seen.hi > seen.lo && seen.hi > ts;
    const int first = some ? max(seen.lo - ts, 0) / kTileKeys : steps;
    const int last = some ? min((seen.hi - ts + kTileKeys - 1) / kTileKeys, steps) : steps;

    // A subtile is 32 keys.  MFMA and VALU work of neighbouring subtiles is
    // independent and put side by side, instruction by instruction:
    //   X(j)  O^T += V^T P^T of subtile j - 1  |  the scores of j as floats
    //   Y(j)  S^T of subtile j + 1             |  the probabilities of j
    // The kernel is bound by the instructions that its two waves per SIMD
    // issue, VALU above all, so the running maximum is not computed: the
    // probabilities are taken against the last one, and only when their sum
    // shows one that fp16 may not hold (Y's last line) is the maximum moved
    // and the subtile's probabilities taken again, which is rare after the
    // first (171 us against 178 for a 4096-token prompt with 32 heads).
    v16f acc[DB] = {};
    v16i si;
    float x[16];
    v8h p[2], vf[DB];
    v4i kf[KS];
    v4f sc[2];
    float m = kNone, l = 0.0f, lref = kNone;   // lref: log2 of the largest value scale so far

    // LDS places: the permutation of the chunks is an exclusive or, so all of
    // a lane's places follow from one (kept out of the compiler's sight, which
    // would hold each of them in a register of its own).
    int kplace = k_place<D>(col, half), vplace = L::K + v_place(col, half);
    auto read_k = [&](int buf, int tt) {
        asm("" : "+v"(kplace));
        const int at = kplace + buf * L::stage;
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
            kf[ks] = *reinterpret_cast<const v4i *>(smem + (at ^ (32 * ks)) + 32 * D * tt);
    };
    auto read_v1 = [&](int buf, int tt, int gi, int n) {
        vf[n] = *reinterpret_cast<const v8h *>(smem + ((vplace + buf * L::stage) ^ (64 * (tt ^ (n & 1)) + 32 * gi)) +
                                               4096 * n);
    };
    auto read_v = [&](int buf, int tt, int gi) {
        asm("" : "+v"(vplace));
#pragma unroll
        for (int n = 0; n < DB; n++)
            read_v1(buf, tt, gi, n);
    };
#define LI8_FENCE __builtin_amdgcn_sched_barrier(0)
    auto mfma_k = [&](int ks, const v4i (&q)[KS]) {
        si = __builtin_amdgcn_mfma_i32_32x32x32_i8(kf[ks], q[ks], si, 0, 0, 0);
        LI8_FENCE;
    };
    auto mfma_v = [&](int n, int gi) {
        acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[n], p[gi], acc[n], 0, 0, 0);
        LI8_FENCE;
    };
    auto to_float = [&](int e0) {
#pragma unroll
        for (int e = e0; e < e0 + 4; e++)
            x[e] = (float)si[e];
        LI8_FENCE;
    };
    // Four probabilities.  The value scale goes into the exponent,
    // 2^(z - m + log2(vs / vref)), and out of the sum again.
    float y[16], bias[2], lv[2], lg[2];
    auto biases = [&]() {
#pragma unroll
        for (int gi = 0; gi < 2; gi++) {
            lv[gi] = fmaxf(sc[gi].y - lref, kLeast);
            bias[gi] = lv[gi] - m + sc[gi].z;
        }
    };
    auto exps = [&](int e0) {
#pragma unroll
        for (int e = e0; e < e0 + 4; e++)
            y[e] = __builtin_amdgcn_exp2f(fmaf(x[e], sc[e >> 3].x, bias[e >> 3]));
        LI8_FENCE;
    };
    auto to_half = [&](int gi) {
        const float *v = y + 8 * gi;
        lg[gi] = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
#pragma unroll
        for (int e = 0; e < 8; e++)
            p[gi][e] = (_Float16)v[e];
        LI8_FENCE;
    };
    // X: PV of the subtile before (its first fragments are in vf, each
    // replaced by its second as soon as it is used), this one's scores as
    // floats; kf is read on the way.
    auto part_x = [&](int vbuf, int vtt, int buf, int tt, int kbuf, int ktt) {
        sc[0] = *reinterpret_cast<const v4f *>(s_sc[buf][2 * tt]);
        sc[1] = *reinterpret_cast<const v4f *>(s_sc[buf][2 * tt + 1]);
        asm("" : "+v"(vplace));
        read_k(kbuf, ktt);
        LI8_FENCE;
#pragma unroll
        for (int n = 0; n < DB; n++) {
            mfma_v(n, 0);
            read_v1(vbuf, vtt, 1, n);
            LI8_FENCE;
        }
#pragma unroll
        for (int n = 0; n < DB; n++) {
            to_float(16 / DB * n);
            if (DB == 2)
                to_float(8 * n + 4);
            mfma_v(n, 1);
        }
    };
    // Y: the next subtile's products with the queries (kf), this one's
    // probabilities; vf is read on the way.
    auto part_y = [&](int buf, int tt) {
        read_v(buf, tt, 0);
        si = v16i{};
        // the factor of the integers (not 0: a masked score is -inf times it)
        sc[0].x = fmaxf(f * sc[0].x, 1.0e-30f);
        sc[1].x = fmaxf(f * sc[1].x, 1.0e-30f);
        biases();
        LI8_FENCE;
        if constexpr (KS == 4) {
            mfma_k(0, qh); exps(0);
            mfma_k(1, qh); exps(4);
            mfma_k(2, qh); to_half(0);
            mfma_k(3, qh); exps(8);
        } else {
            mfma_k(0, qh); exps(0); exps(4);
            mfma_k(1, qh); to_half(0); exps(8);
        }
        si <<= 7;
        LI8_FENCE;
        if constexpr (KS == 4) {
            mfma_k(0, ql); exps(12);
            mfma_k(1, ql); to_half(1);
            mfma_k(2, ql);
            mfma_k(3, ql);
        } else {
            mfma_k(0, ql); exps(12);
            mfma_k(1, ql); to_half(1);
        }
        if (__any(fmaxf(lg[0], lg[1]) > kMost)) {
            float zm = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; e++)
                zm = fmaxf(zm, fmaf(x[e], sc[e >> 3].x, sc[e >> 3].z));
            zm = fmaxf(zm, __shfl_xor(zm, 32, 64));
            const float mn = fmaxf(m, zm), ln = fmaxf(lref, fmaxf(sc[0].y, sc[1].y));
            const float am = __builtin_amdgcn_exp2f(m - mn);
            const float al = am * __builtin_amdgcn_exp2f(lref - ln);
#pragma unroll
            for (int n = 0; n < DB; n++)
                acc[n] *= al;
            l *= am;
            m = mn;
            lref = ln;
            biases();
#pragma unroll
            for (int e0 = 0; e0 < 16; e0 += 4)
                exps(e0);
            to_half(0);
            to_half(1);
        }
        l = fmaf(lg[0], __builtin_amdgcn_exp2f(-lv[0]), l);
        l = fmaf(lg[1], __builtin_amdgcn_exp2f(-lv[1]), l);
    };
    auto mask = [&](int t0) {
        if (t0 < wlo || t0 + 32 > whi) {
#pragma unroll
            for (int e = 0; e < 16; e++) {
                const int key = t0 + 8 * (e >> 2) + 4 * half + (e & 3);
                x[e] = key < chi && key >= clo ? x[e] : -INFINITY;
            }
        }
    };

    if (steps > 0) {
        pages(ts);
        load(ts);
        pages(ts + kTileKeys);
        store(0);
        load(ts + kTileKeys);
        pages(ts + 2 * kTileKeys);
    }
    __syncthreads();
    int buf = 0, pbuf = 0, i = 0;
    // Three buffers: tile i + 1 goes where tile i - 2 was, which every wave
    // has left behind before the last barrier.
    auto next = [&]() { return buf == 2 ? 0 : buf + 1; };
    auto stage = [&]() {
        if (i + 1 < steps) {
            store(next());
            load(ts + kTileKeys * (i + 2));
            pages(ts + kTileKeys * (i + 3));
        }
    };
    auto leave = [&]() {
        pbuf = buf;
        buf = next();
    };
    // (three loops, so that the middle one has no other way through it: the
    // compiler would keep the accumulators twice)
    for (; i < first; i++) {
        stage();
        lds_barrier();
        leave();
    }
    if (first < last) {
        read_k(buf, 0);
        si = v16i{};
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
            si = __builtin_amdgcn_mfma_i32_32x32x32_i8(kf[ks], qh[ks], si, 0, 0, 0);
        si <<= 7;
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
            si = __builtin_amdgcn_mfma_i32_32x32x32_i8(kf[ks], ql[ks], si, 0, 0, 0);
        p[0] = p[1] = v8h{};   // (nothing to add yet)
#pragma unroll
        for (int n = 0; n < DB; n++)
            vf[n] = v8h{};
        pbuf = buf;
        for (; i < last; i++) {
            const int t0 = ts + kTileKeys * i;
            stage();
            part_x(pbuf, 1, buf, 0, buf, 1);
            mask(t0);
            part_y(buf, 0);
            lds_barrier();
            part_x(buf, 0, buf, 1, next(), 0);   // (past the last step: keys of no use, and not used)
            mask(t0 + 32);
            part_y(buf, 1);
            leave();
        }
#pragma unroll
        for (int n = 0; n < DB; n++)
            mfma_v(n, 0);
        read_v(pbuf, 1, 1);
#pragma unroll
        for (int n = 0; n < DB; n++)
            mfma_v(n, 1);
    }
    for (; i < steps; i++) {
        stage();
        lds_barrier();
        leave();
    }
#undef LI8_FENCE
    if (qcol >= b.nc)
        return;
    l += __shfl_xor(l, 32, 64);
    const float s = l > 0.0f ? __builtin_amdgcn_exp2f(lref) / l : 0.0f;
    if (slot >= 0) {
        const int64_t at = slot * t.used + qcol;
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
    const int64_t row = b.q.q0 + (pos - b.q.begin);
    const int head = b.h * t.group + gcol;
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

template <int D, bool BF16>
__global__ __launch_bounds__(64 * kTileWaves, 2) void k_kv_tiled(KvArgs a, AttnArgs t, int pairs, int lanes, int deep)
{
    __shared__ __align__(16) char smem[TileLds<D>::bytes];
    __shared__ float s_f[kTileCols];
    __shared__ __align__(16) float s_sc[3][4][4];   // [buffer][group of 16 keys][k scale, log2 v scale, 0 or -inf]
    const int lane = threadIdx.x & 63;
    Run<6, false> run;
    Block b;
    int first = 0, count = 0;
    int64_t slot = -1;
    bool there;
    if (t.parts == 0) {
        // Blocks of one (sequence, head) share its keys: they stay on
        // 8 / lanes of the XCDs (the hardware deals workgroups to the 8 XCDs
        // in turn).  Where a chunk is most of its sequence (deep == 0) its
        // last blocks see the most keys and go first, those of all pairs of
        // the lane before any block that sees fewer: a long block that starts
        // late would run alone at the end.  Chunks over much longer sequences
        // have blocks alike, and one pair goes after the other, so that its
        // keys stay in the L2.  Measured, pair by pair : longest first (us):
        //   longest first up to half of the sequence: prompts of 4096 with 32
        //   heads 228 : 167, 4096 of 8000 486 : 428, 8 x 1024 of 1500 193 : 160;
        //   but 4 x 2048 of 4000, 8 heads of a group of 8, 718 : 823
        //   pair by pair past it, groups of 8: 4 x 512 of 8192 411 : 477, 1024
        //   of 4096 387 : 467, 2048 of 4300 783 : 898; but 32 heads of one:
        //   4096 of 8300 509 : 451, 8 x 512 of 2048 149 : 139
        const int j = blockIdx.x / lanes, ppl = (pairs + lanes - 1) / lanes;
        const int pair = (deep ? j / t.blocks : j % ppl) * lanes + blockIdx.x % lanes;
        if (pair >= pairs)
            return;
        there = locate(a, t, pair * t.blocks + (t.blocks - 1 - (deep ? j % t.blocks : j / ppl)), kTileCols, b);
        run.at = run.end = 0;
    } else {
        // neighbouring runs on one XCD
        const int per = t.parts >> 3;
        if (!run.start(a, t, t.parts & 7 ? blockIdx.x : (blockIdx.x & 7) * per + (blockIdx.x >> 3), lane))
            return;
        there = run.next(a, t, kTileCols, lane, b, first, count, slot);
    }
    while (true) {
        if (there) {
            const int ts = min(b.span.base + kTileKeys * first, b.span.hi);
            const int te = count ? min(b.span.hi, ts + kTileKeys * count) : b.span.hi;
            tile_block<D, BF16>(a, t, b, ts, te, slot, smem, s_f, s_sc);
        }
        if (run.at >= run.end)
            return;
        __syncthreads();
        there = run.next(a, t, kTileCols, lane, b, first, count, slot);
    }
}

template <int D, bool BF16, int SL>
__device__ __forceinline__ void merge_column(const KvArgs &a, const AttnArgs &t, const Block &b, int qc, int na,
                                             int64_t slot0, int p0, int sl, int cc)
{
    constexpr int CPR = D / 8, WIDTH = SL * CPR;
    float m = kNone, l = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int i = sl; i < na; i += 4 * SL) {
        float e[4], x[4][8];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int j = min(i + k * SL, na - 1);
            const int64_t at = (j == 0 ? slot0 : 2 * (int64_t)(p0 + j)) * t.used + qc;
            e[k] = t.part_m[at];
            *reinterpret_cast<float4 *>(x[k]) = *reinterpret_cast<const float4 *>(t.part_o + at * D + 8 * cc);
            *reinterpret_cast<float4 *>(x[k] + 4) = *reinterpret_cast<const float4 *>(t.part_o + at * D + 8 * cc + 4);
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float ek = i + k * SL < na ? e[k] : kNone;
            const float mn = fmaxf(m, ek), al = __builtin_amdgcn_exp2f(m - mn);
            const float be = ek > kNone ? __builtin_amdgcn_exp2f(ek - mn) : 0.0f;
            l = l * al + be;
#pragma unroll
            for (int j = 0; j < 8; j++)
                o[j] = o[j] * al + x[k][j] * be;
            m = mn;
        }
    }
    auto join = [&](float m2, float l2, const float (&o2)[8]) {
        const float mn = fmaxf(m, m2), al = __builtin_amdgcn_exp2f(m - mn), be = __builtin_amdgcn_exp2f(m2 - mn);
        l = l * al + l2 * be;
#pragma unroll
        for (int k = 0; k < 8; k++)
            o[k] = o[k] * al + o2[k] * be;
        m = mn;
    };
#pragma unroll
    for (int d = CPR; d < (WIDTH < 64 ? WIDTH : 64); d *= 2) {
        float o2[8];
#pragma unroll
        for (int k = 0; k < 8; k++)
            o2[k] = __shfl_xor(o[k], d, 64);
        join(__shfl_xor(m, d, 64), __shfl_xor(l, d, 64), o2);
    }
    if constexpr (WIDTH > 64) {
        constexpr int W = WIDTH / 64;
        __shared__ float s_o[W][D], s_m[W], s_l[W];
        const int w = threadIdx.x / 64;
        __syncthreads();                         // (the column before)
        if (threadIdx.x % 64 < CPR) {
#pragma unroll
            for (int k = 0; k < 8; k++)
                s_o[w][8 * cc + k] = o[k];
            s_m[w] = m;
            s_l[w] = l;
        }
        __syncthreads();
        if (w == 0) {
            for (int i = 1; i < W; i++) {
                float o2[8];
#pragma unroll
                for (int k = 0; k < 8; k++)
                    o2[k] = s_o[i][8 * cc + k];
                join(s_m[i], s_l[i], o2);
            }
        }
    }
    if (sl != 0 || threadIdx.x >= (WIDTH == 256 ? 64 : 256))
        return;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++)
        o[k] *= inv;
    int g;
    const int i = b.row_of(qc, t, g);
    const int64_t row = b.q.q0 + i;
    const int head = b.h * t.group + g;
    *reinterpret_cast<uint4 *>(t.O + row * t.os + (int64_t)head * D + 8 * cc) = pack8<BF16>(o);
    if (t.lse && cc == 0)
        t.lse[row * (int64_t)(a.heads * t.group) + head] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Merges the partial results of a block's columns: O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M),
// m_i the part's log2 of its sum.  SL lanes of parts x D/8 chunks work on a
// column: with many parts the workgroup, else a wave, or (SL = 1, where blocks
// are wide and in few parts) D/8 lanes of it.  A wave has `each` columns of
// one block; four parts are in flight per lane.  The workgroup from 15 parts for
// each block on: with 64 the call takes 53.7 us against 55.5 with a wave, with 1
// (512 blocks) 155 against 146, between 4 and 16 no difference.  64 sequences' one token each
// (512 blocks of 8 columns, up to 4 parts) takes 7.8 us, 8 blocks of 64 parts
// 4.9: the launch and two chains of loads, lengths and then parts.
template <int D, bool BF16, int SL, int SHIFT>
__global__ __launch_bounds__(256) void k_kv_merge(KvArgs a, AttnArgs t, int items, int each)
{
    constexpr int CPR = D / 8, WIDTH = SL * CPR;
    constexpr int TASK = WIDTH > 64 ? WIDTH : 64;   // threads of a task
    const int cc = threadIdx.x % CPR, sl = threadIdx.x % WIDTH / CPR, lane = threadIdx.x & 63;
    const int task = blockIdx.x * (256 / TASK) + threadIdx.x / TASK, tasks = (t.used + each - 1) / each;
    const int item = min(task / tasks, items - 1);
    Block b;
    const bool there = locate(a, t, item, t.cols, b) && task / tasks < items;
    // steps before the block
    const int cb = item % t.blocks, sh = item / t.blocks, s = sh / a.heads, h = sh % a.heads;
    Steps<SHIFT> w;
    int total, before = 0;
    const int per = w.share(a, t, lane, total);
    for (int c = 0; c < (s >> 6); c++) {
        before += __shfl(w.upto, 63, 64);
        w.look(a, t, c + 1, lane);
    }
    const int k = s & 63, steps = __shfl(w.steps, k, 64), blocks = __shfl(w.blocks, k, 64);
    const int u0 = before + __shfl(w.upto - w.all, k, 64) + (h * blocks + cb) * steps, u1 = u0 + steps - 1;
    const int p0 = u0 / per, p1 = u1 / per;
    if (!there || p1 == p0)                      // (its workgroup has written it)
        return;
    // Its first part is the last block of its run (slot 1) unless the run
    // begins with it; the others begin theirs (slot 0).
    const int na = p1 - p0 + 1;
    const int64_t slot0 = u0 == p0 * per ? 2 * (int64_t)p0 : 2 * (int64_t)p0 + 1;
    const int first = task % tasks * each, stop = min(first + each, b.nc);
    for (int qc = first + threadIdx.x % TASK / WIDTH; qc < stop; qc += TASK / WIDTH)
        merge_column<D, BF16, SL>(a, t, b, qc, na, slot0, p0, sl, cc);
}

// Which kernel, and whether blocks are shared, measured (us):
//   tiled from 128 columns and 4096 steps (blocks x steps of 64 keys) on: two
//   chunks' worth of work per CU.  Few columns against tiled at 128 heads x
//   blocks of a 1024-token prompt with 32 heads (2048 steps) 41 : 42, at 2048
//   tokens (8192 steps) 164 : 72, 64 tokens x 64 heads over 8192 keys (2048
//   steps) 45 : 50, 256 tokens x 64 heads over 8192 keys (8192 steps)
//   127 : 97; 8 tokens x 8 heads of a group, 64 columns, in 16 sequences of
//   up to 4096 keys 52 : 69, twice as many 83 : 72.
//   few columns are shared past 40 steps of 32 keys: at 25 steps one launch
//   took 11.3 against 18.3, at 41 to 4096 sharing is up to 4 times as fast.
//   From 4096 blocks on (8 for each workgroup that would share) they are not:
//   one token each, whole : shared, 128 sequences x 32 heads of 300 to 4000 keys
//   394 : 461, 512 x 8 heads of a group of 8 406 : 584, of 2000 keys each 390 :
//   415 (32 heads 370 : 353).  One sequence of 131071 keys among 127 of 1000
//   then runs alone at the end, 928 : 377; the host does not see the lengths.
//   tiled blocks are shared where there are fewer than CUs: 64 blocks of 128
//   steps 97 against 242 unshared, 256 blocks of a 2048-token prompt 77
//   against 72 (their keys differ, which the count of steps does not know).
//   Chunks over long sequences shared from 256 blocks on, 380 and 500 blocks
//   of up to 128 steps: 415 against 409, 491 against 571; the host does not
//   see which.
constexpr int kTileColumns = 128;
constexpr int kTileSteps = 4096;
constexpr int kFewWhole = 40;
constexpr int kFewSlots = 512;         // workgroups that share steps: 2 for each CU
constexpr int kTileSlots = 256;        // tiled: 1 for each CU

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

int64_t plan_items(const li8_kv_batch &b, const li8_kv_cache &c, const KvPlan &p)
{
    return (int64_t)b.seqs * c.heads * p.blocks;
}

// (sequence, head) pairs of the tiled kernel dealt over the XCDs: 8 lanes,
// fewer where that would leave XCDs without work.
int tiled_lanes(int64_t pairs) { return pairs >= 64 ? 8 : (int)std::min<int64_t>(8, pairs & -pairs); }

// Work-items of an unshared few-column workgroup: 8 waves where blocks are few,
// measured 8 : 4 (us): 5 tokens of 4 heads of a group, D = 64, 1200 keys, in 128
// blocks 12.7 : 14.6, in 256 14.2 : 15.7; one token of 32 heads over 777 keys
// 11.5 : 11.5; 768 blocks of 1200 keys 48 : 39.  At 512 blocks 4 are ahead already
// (34 : 29; a 512-token prompt 22 : 17).
int few_items(int64_t items) { return items <= 512 ? 512 : 256; }

template <int D, bool BF16>
hipError_t attention_go(const KvArgs &a, const AttnArgs &t, int64_t items, hipStream_t s)
{
    if (t.cols == kTileCols) {
        const int64_t pairs = items / t.blocks;
        const int lanes = tiled_lanes(pairs);
        const unsigned grid = t.parts > 0 ? (unsigned)t.parts : (unsigned)(round_up(pairs, lanes) * t.blocks);
        k_kv_tiled<D, BF16><<<grid, 64 * kTileWaves, 0, s>>>(a, t, (int)pairs, lanes,
                                                                !t.causal || a.max_q < a.max_kv / 2);
    } else {
        const bool wide = t.cols != kKvCols, once = t.blocks == 1;
        if (t.parts > 0) {
            const unsigned grid = (unsigned)t.parts;
            if (wide && once)
                k_kv_few<D, BF16, 2, 4, true><<<grid, 256, 0, s>>>(a, t);
            else if (wide)
                k_kv_few<D, BF16, 2, 4, false><<<grid, 256, 0, s>>>(a, t);
            else
                k_kv_few<D, BF16, 1, 4, true><<<grid, 256, 0, s>>>(a, t);
        } else if (few_items(items) == 512) {
            if (wide)
                k_kv_few<D, BF16, 2, 8, false><<<(unsigned)items, 512, 0, s>>>(a, t);
            else
                k_kv_few<D, BF16, 1, 8, false><<<(unsigned)items, 512, 0, s>>>(a, t);
        } else {
            if (wide)
                k_kv_few<D, BF16, 2, 4, false><<<(unsigned)items, 256, 0, s>>>(a, t);
            else
                k_kv_few<D, BF16, 1, 4, false><<<(unsigned)items, 256, 0, s>>>(a, t);
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || t.parts == 0)
        return e;
    // about as many lanes as a column can have parts
    const int each = t.cols == kTileCols ? 16 : 1;
    const int64_t tasks = items * ((t.used + each - 1) / each);
    if (t.cols == kTileCols)
        k_kv_merge<D, BF16, 1, 6><<<(unsigned)((tasks + 3) / 4), 256, 0, s>>>(a, t, (int)items, each);
    else if (t.parts / items + 2 <= 16)
        k_kv_merge<D, BF16, 64 * 8 / D, 5><<<(unsigned)((tasks + 3) / 4), 256, 0, s>>>(a, t, (int)items, each);
    else
        k_kv_merge<D, BF16, 256 * 8 / D, 5><<<(unsigned)tasks, 256, 0, s>>>(a, t, (int)items, each);
    return hipGetLastError();
}

} // namespace

KvPlan kv_plan(const li8_kv_batch &b, const li8_kv_cache &c, int q_heads, bool causal, int window)
{
    KvPlan p = {LI8_KV_EMPTY, kKvCols, 0, 0, 1, 0};
    const int64_t rows = std::min(b.max_q, b.tokens), group = q_heads / c.heads;
    if (rows == 0 || b.seqs == 0)
        return p;
    const int64_t cols = rows * group;
    // keys from a span's base to its end at most: a window's keys, the other
    // rows of the block (without `causal` the end is the sequence's, so all
    // rows that follow) and the rounding of the base
    auto steps_of = [&](int64_t key_step) {
        int64_t span = b.max_kv;
        if (window > 0)
            span = std::min<int64_t>(span, (int64_t)window + (causal ? p.cols : rows) + 31);
        return (span + key_step - 1) / key_step;
    };
    auto items_of = [&]() { return (int64_t)b.seqs * c.heads * ((cols + p.cols - 1) / p.cols); };
    p.cols = kTileCols;
    int64_t steps = steps_of(kTileKeys), items = items_of(), slots = kTileSlots;
    bool whole = items >= slots;
    if (cols >= kTileColumns && items * steps >= kTileSteps) {
        p.path = LI8_KV_TILED;
    } else {
        p.path = LI8_KV_FEW;
        p.cols = cols > kKvCols ? 2 * kKvCols : kKvCols;
        steps = steps_of(32);
        items = items_of();
        slots = kFewSlots;
        whole = steps <= kFewWhole || items >= 8 * slots;
    }
    p.blocks = (int)((cols + p.cols - 1) / p.cols);
    p.used = (int)std::min<int64_t>(p.cols, cols);
    // (counted as without a window, so that what is shared, and with it the
    // workspace, does not depend on it)
    if (!whole && items * (((int64_t)b.max_kv + 31) / 32) < ((int64_t)1 << 30)) {
        p.parts = (int)std::min(slots, (items * steps + kLeastSteps - 1) / kLeastSteps);
        p.splits = (int)std::min<int64_t>(p.parts, steps);
    }
    return p;
}

size_t kv_workspace(const li8_kv_batch &b, const li8_kv_cache &c, int q_heads)
{
    // The kernel, and with it the columns of a slot, can change with the
    // window; so the most that either takes: two slots for each workgroup
    // that shares.
    const KvPlan p = kv_plan(b, c, q_heads, true, 0);
    if (p.path == LI8_KV_EMPTY)
        return 0;
    const int64_t cols = std::min<int64_t>(kTileCols, (int64_t)std::min(b.max_q, b.tokens) * (q_heads / c.heads));
    int64_t rows = 2 * (int64_t)p.parts * p.used;
    if (p.path == LI8_KV_TILED)   // (few columns under a window: at most 32 in each of 512)
        rows = std::max<int64_t>(p.parts ? 2 * (int64_t)kTileSlots * cols : 0, 2 * (int64_t)kFewSlots * 2 * kKvCols);
    if (rows == 0)
        return 0;
    return align_up((size_t)rows * 4 * c.head_dim, 256) + align_up((size_t)rows * 4, 256);
}

double kv_attention_items(const li8_kv_batch &b, const li8_kv_cache &c, const KvPlan &p)
{
    if (p.path == LI8_KV_EMPTY || p.parts > 0)   // (shared: fewer than 8 kFewSlots blocks, merging them included)
        return 0;
    const int64_t pairs = (int64_t)b.seqs * c.heads;
    if (p.path == LI8_KV_TILED)
        return (double)round_up(pairs, tiled_lanes(pairs)) * p.blocks * (64 * kTileWaves);
    return (double)pairs * p.blocks * few_items(plan_items(b, c, p));
}

hipError_t launch_kv_attention(KvTokens Q, bool bf16, int q_heads, float scale, KvRope rope,
                               bool causal, int window, const li8_kv_batch &b,
                               const li8_kv_cache &c, uint16_t *O, int64_t os, float *lse,
                               char *ws, hipStream_t s)
{
    const KvPlan p = kv_plan(b, c, q_heads, causal, window);
    const KvArgs a = kv_args(b, c);
    const int64_t items = plan_items(b, c, p);
    const int64_t slots = 2 * (int64_t)p.parts;
    AttnArgs t;
    t.Q = Q; t.rope = rope; t.O = O; t.os = os; t.lse = lse;
    t.part_o = reinterpret_cast<float *>(ws);
    t.part_m = reinterpret_cast<float *>(ws + align_up((size_t)(slots * p.used) * 4 * c.head_dim, 256));
    t.scale = scale * kLog2e;
    t.group = q_heads / c.heads; t.inv_group = 1.0f / (float)t.group; t.causal = causal; t.window = window;
    t.cols = p.cols; t.blocks = p.blocks; t.used = p.used;
    t.seqs = b.seqs; t.parts = p.parts;
    if (c.head_dim == 128)
        return bf16 ? attention_go<128, true>(a, t, items, s) : attention_go<128, false>(a, t, items, s);
    return bf16 ? attention_go<64, true>(a, t, items, s) : attention_go<64, false>(a, t, items, s);
}

} // namespace li8
