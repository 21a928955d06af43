// Appending to the int8 key/value cache and reading it back, for gfx950.
//
// Append: for every (page touched, head, keys or values), with x the new rows
// (keys rotated) and s0 the page's scale if it holds older rows, else 0:
//   s = max(fl32(max|x| / 127), s0)       r = min(fl32(1/s), FLT_MAX)
//   code = clamp(rne(fl32(x r)))          older rows coded again where s > s0
// (lowentro.cn "model quantization" notes, Q2 and Q11: symmetric absmax codes.)
// The scale needs every new row of the page before the first code, so one
// workgroup owns one (page, head): it keeps its rows in registers between the
// maximum and the codes, and every value is read once (the rotation's partner
// half comes from the cache line that another lane of the row has fetched).
// What bounds it: 2 bytes read and 1 written per value, so memory for a prompt
// (chunks of 5622 tokens, 40 heads, D = 128, 173 MB: 39 us, 4.5 TB/s, where a copy
// has 5.0; 30 us over again on the same tokens, which are in the Infinity Cache
// then); for one token per sequence the launch and one chain of dependent loads
// (lengths, page number, scale and row): 3.4 us for 8 sequences, 4.4 for 256.
//
// Read: one thread per 8 codes, K and V in one launch, 1 byte read and 2
// written per value, with non-temporal stores: lines left dirty in the L2 are
// written back when the kernel ends, and the next one waits for that (four
// sequences of up to 8191 tokens, 176 MB moved: 41.9 -> 26.9 us over again on the
// same pages, whose 59 MB the Infinity Cache holds; on other pages each time
// 39.6 us, 4.4 TB/s).
#include <float.h>

#include <algorithm>

#include "kv_device.h"

namespace li8 {
namespace {

__device__ __forceinline__ uint32_t code_word(const float x[4], float r)
{
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float q = fminf(fmaxf(rintf(x[i] * r), -127.0f), 127.0f);
        w |= ((uint32_t)(int)q & 0xffu) << (8 * i);
    }
    return w;
}

__device__ __forceinline__ float byte_value(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// RPT: rows per thread, at least ceil(rows of a page and chunk / rows at once).
template <int D, int THREADS, int RPT, bool BF16>
__global__ __launch_bounds__(THREADS) void k_kv_append(KvArgs a, KvTokens K, KvTokens V, KvRope rope,
                                                       int touched)
{
    constexpr int CPR = D / 8, RA = THREADS / CPR;   // chunks of a row, rows at once
    const int tid = threadIdx.x, s = blockIdx.x / touched, b = blockIdx.x % touched;
    const int h = blockIdx.y, page = 1 << a.page_shift;
    const bool value = blockIdx.z != 0;
    const KvSeq q = kv_sequence_of(a, s);
    const int begin = max(q.begin, 0), end = q.begin + q.n;   // positions to store
    const int pi = (begin >> a.page_shift) + b;
    const int lo = max(begin, pi << a.page_shift), hi = min(end, (pi + 1) << a.page_shift);
    if (lo >= hi)
        return;
    const int pid = a.table[(int64_t)s * a.table_stride + pi];
    if ((unsigned)pid >= (unsigned)a.pages)
        return;
    const int64_t ph = (int64_t)pid * a.heads + h;
    int8_t *codes = (value ? a.v : a.k) + ((ph * D) << a.page_shift);
    float *scale = (value ? a.vs : a.ks) + ph;
    const int off = lo & (page - 1);                 // older rows of the page
    const float s_old = off ? *scale : 0.0f;
    const KvTokens src = value ? V : K;
    KvRope rr = rope;
    if (value)
        rr.cos = nullptr;
    const int c = tid % CPR, ra = tid / CPR;
    float x[RPT][8], m = 0.0f;
    with_rotation(rr, [&](auto rot) {
        constexpr int ROT = decltype(rot)::value, BATCH = RPT < 4 ? RPT : 4;   // rows in flight
#pragma unroll
        for (int k0 = 0; k0 < RPT; k0 += BATCH) {
            RowChunk w[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; k++) {   // (rows past the end: the last one again)
                const int pos = min(lo + ra + RA * (k0 + k), hi - 1);
                fetch_row<ROT>(w[k], src.p + (q.q0 + pos - q.begin) * src.stride + h * D, c, rr, pos);
            }
#pragma unroll
            for (int k = 0; k < BATCH; k++) {
                rotate_row<BF16, ROT>(w[k], c, rr, x[k0 + k]);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    m = fmaxf(m, fabsf(x[k0 + k][e]));
            }
        }
    });
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
        m = fmaxf(m, __shfl_xor(m, o, 64));
    if constexpr (THREADS > 64) {
        __shared__ float part[THREADS / 64];
        if ((tid & 63) == 0)
            part[tid >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 64; w++)
            m = fmaxf(m, part[w]);
    }
    const float sn = fmaxf(m / 127.0f, s_old);
    const float r = sn > 0.0f ? fminf(1.0f / sn, FLT_MAX) : 0.0f;
    if (tid == 0)
        *scale = sn;
#pragma unroll
    for (int k = 0; k < RPT; k++) {
        const int row = off + ra + RA * k;
        if (row < off + (hi - lo))
            *reinterpret_cast<uint2 *>(codes + row * D + 8 * c) =
                make_uint2(code_word(x[k], r), code_word(x[k] + 4, r));
    }
    if (off == 0 || !(sn > s_old))
        return;
    // The page's older rows under the larger scale, 16 codes per load and
    // four loads in flight.
    uint4 *old = reinterpret_cast<uint4 *>(codes);
    const int units = off * (D / 16);
    for (int u0 = tid; u0 < units; u0 += 4 * THREADS) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            v[j] = old[min(u0 + j * THREADS, units - 1)];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    y[i] = byte_value(w[e], i) * s_old;
                w[e] = code_word(y, r);
            }
            if (u0 + j * THREADS < units)
                old[u0 + j * THREADS] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

typedef uint32_t kv_u4 __attribute__((ext_vector_type(4)));

constexpr int kReadTokens = 64;   // tokens of a read workgroup

template <int D, bool BF16>
__global__ __launch_bounds__(256) void k_kv_read(KvArgs a, uint16_t *K, int64_t ks, uint16_t *V,
                                                 int64_t vs, int blocks)
{
    constexpr int CPR = D / 8, RA = 256 / CPR, RPT = kReadTokens / RA;
    const int tid = threadIdx.x, s = blockIdx.x / blocks, b = blockIdx.x % blocks;
    const int h = blockIdx.y;
    const bool value = blockIdx.z != 0;
    const KvSeq q = kv_sequence_of(a, s);
    const int c = tid % CPR, i0 = b * kReadTokens + tid / CPR;
    if (b * kReadTokens >= q.n)
        return;
    const int8_t *codes = value ? a.v : a.k;
    const float *scales = value ? a.vs : a.ks;
    uint16_t *out = (value ? V : K) + h * D + 8 * c;
    const int64_t stride = value ? vs : ks;
    uint2 w[RPT];
    float f[RPT];
#pragma unroll
    for (int k = 0; k < RPT; k++) {
        const int i = i0 + RA * k, pos = q.begin + i;
        w[k] = make_uint2(0, 0);
        f[k] = 0.0f;
        if (i < q.n && pos >= 0) {
            const int pid = a.table[(int64_t)s * a.table_stride + (pos >> a.page_shift)];
            if ((unsigned)pid < (unsigned)a.pages) {
                const int64_t ph = (int64_t)pid * a.heads + h;
                const int row = pos & ((1 << a.page_shift) - 1);
                w[k] = *reinterpret_cast<const uint2 *>(codes + ((ph * D) << a.page_shift) + row * D + 8 * c);
                f[k] = scales[ph];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < RPT; k++) {
        const int i = i0 + RA * k;
        if (i >= q.n)
            continue;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e++)
            x[e] = byte_value(e < 4 ? w[k].x : w[k].y, e & 3) * f[k];
        const uint4 r = pack8<BF16>(x);
        __builtin_nontemporal_store(kv_u4{r.x, r.y, r.z, r.w}, reinterpret_cast<kv_u4 *>(out + (q.q0 + i) * stride));
    }
}

template <int D, int THREADS, int RPT, bool BF16>
hipError_t append_go(const KvArgs &a, KvTokens K, KvTokens V, KvRope rope, int seqs, int touched,
                     hipStream_t s)
{
    k_kv_append<D, THREADS, RPT, BF16>
        <<<dim3((unsigned)(seqs * touched), (unsigned)a.heads, 2), THREADS, 0, s>>>(a, K, V, rope, touched);
    return hipGetLastError();
}

// Pages that a chunk of the longest length can touch, and its new rows in one.
int touched_pages(int q, int page) { return (int)(((int64_t)q + page - 2) / page + 1); }
int page_rows(int q, int page) { return std::min(page, q); }

// One wave per page and head while its rows fit one pass of the wave: a step
// of one token per sequence has 4 rows at D = 128 of which one is there, and a
// larger workgroup would idle.
bool one_wave(int rows, int dim) { return rows <= 64 / (dim / 8); }

template <int D, bool BF16>
hipError_t append_d(const KvArgs &a, KvTokens K, KvTokens V, KvRope rope, int seqs, hipStream_t s)
{
    const int page = 1 << a.page_shift, q = std::min(a.max_q, a.tokens);
    const int touched = touched_pages(q, page), rows = page_rows(q, page);
    if (one_wave(rows, D))
        return append_go<D, 64, 1, BF16>(a, K, V, rope, seqs, touched, s);
    const int rpt = (rows + 256 / (D / 8) - 1) / (256 / (D / 8));
    if (rpt <= 1)
        return append_go<D, 256, 1, BF16>(a, K, V, rope, seqs, touched, s);
    if (rpt <= 2)
        return append_go<D, 256, 2, BF16>(a, K, V, rope, seqs, touched, s);
    if (rpt <= 4)
        return append_go<D, 256, 4, BF16>(a, K, V, rope, seqs, touched, s);
    return append_go<D, 256, 8, BF16>(a, K, V, rope, seqs, touched, s);
}

int64_t read_blocks(const li8_kv_batch &b)
{
    return ((int64_t)std::min(b.max_q, b.tokens) + kReadTokens - 1) / kReadTokens;
}

} // namespace

double kv_append_items(const li8_kv_batch &b, const li8_kv_cache &c)
{
    const int q = std::min(b.max_q, b.tokens);
    return (double)b.seqs * touched_pages(q, c.page_size) *
           (one_wave(page_rows(q, c.page_size), c.head_dim) ? 64 : 256);
}

double kv_read_items(const li8_kv_batch &b) { return (double)b.seqs * read_blocks(b) * 256; }

hipError_t launch_kv_append(KvTokens K, KvTokens V, bool bf16, KvRope rope, const li8_kv_batch &b,
                            const li8_kv_cache &c, hipStream_t s)
{
    const KvArgs a = kv_args(b, c);
    if (c.head_dim == 128)
        return bf16 ? append_d<128, true>(a, K, V, rope, b.seqs, s)
                    : append_d<128, false>(a, K, V, rope, b.seqs, s);
    return bf16 ? append_d<64, true>(a, K, V, rope, b.seqs, s)
                : append_d<64, false>(a, K, V, rope, b.seqs, s);
}

hipError_t launch_kv_read(const li8_kv_cache &c, const li8_kv_batch &b, bool bf16, uint16_t *K,
                          int64_t ks, uint16_t *V, int64_t vs, hipStream_t s)
{
    const KvArgs a = kv_args(b, c);
    const int blocks = (int)read_blocks(b);
    const dim3 grid((unsigned)(b.seqs * blocks), (unsigned)c.heads, 2);
    if (c.head_dim == 128) {
        if (bf16)
            k_kv_read<128, true><<<grid, 256, 0, s>>>(a, K, ks, V, vs, blocks);
        else
            k_kv_read<128, false><<<grid, 256, 0, s>>>(a, K, ks, V, vs, blocks);
    } else {
        if (bf16)
            k_kv_read<64, true><<<grid, 256, 0, s>>>(a, K, ks, V, vs, blocks);
        else
            k_kv_read<64, false><<<grid, 256, 0, s>>>(a, K, ks, V, vs, blocks);
    }
    return hipGetLastError();
}

} // namespace li8
