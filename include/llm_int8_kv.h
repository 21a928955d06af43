/*
 * llm_int8_kv.h - C ABI of the int8 key/value cache of libllm_int8.so: what
 * stands between the int8 projections of a decoder layer (llm_int8.h).
 *
 * The cache holds keys and values as int8 codes in pages of tokens, with one
 * symmetric absmax scale for each page and head (the scheme of llm_int8.h,
 * scale = absmax/127, round half to even, clip at +-127, applied to a block
 * of tokens; lowentro.cn "model quantization" notes, Q11: the key/value
 * cache as a runtime tensor that is quantized on the way):
 *   k, v              int8 [pages][heads][page_size][head_dim]
 *   k_scale, v_scale  fp32 [pages][heads]        value = code * scale
 * Three operators work on it:
 *   int8_kv_append     stores new tokens' keys and values, rotating the keys
 *                      by their positions on the way;
 *   int8_kv_read       gives stored tokens back in 16 bits;
 *   int8_kv_attention  attends over it, rotating the queries on the way.
 *
 * Conventions are those of llm_int8.h: asynchronous and ordered on `stream`
 * (of the current device, where all memory lives), validated on the host
 * before anything is launched, nothing allocated, synchronized or read back,
 * no mutable state in the library.  In addition:
 *   - 16-bit tensors are fp16 or bf16 (li8_dtype); rows of tokens may be
 *     strided (a slice of a fused projection), each row is [heads][head_dim]
 *     without gaps.  Row strides are in elements, a multiple of 8.
 *   - Pointers to 16-bit tensors, codes, rotation tables and workspaces are
 *     16-byte aligned; the int32 and the scale and lse arrays 4-byte.
 *   - Lengths and page numbers are device data that the host does not see.
 *     A sequence longer than max_kv or than its table row is cut to it, a
 *     chunk longer than max_q has the tokens past it left out, and a page
 *     number outside [0, pages) is never followed: nothing is stored there,
 *     reading gives zeros, and attention treats its tokens as masked.
 *   - A batch is refused (LI8_ERR_SHAPE) where a grid would have 2^32
 *     work-items or more.  With q = min(max_q, tokens): append from seqs x
 *     pages of q tokens of 2^24 on, read from seqs x ceil(q / 64) of 2^24 on,
 *     attention from seqs x heads x blocks of columns of 2^23 on (at the
 *     earliest; smaller workgroups go further).
 *   - Inputs must be finite where they are read (keys and queries after their
 *     rotation too); the scales of pages with stored tokens >= 0 and below 2^126
 *     (append writes none above 2^121).  Codes and scales of tokens that no
 *     query sees, and rows outside [q_start[0], q_start[seqs]), may hold
 *     anything.
 *   - Lengths, starts and page numbers must not change while a call runs (work
 *     on other streams that changes them has to wait for it).
 */
#ifndef LLM_INT8_KV_H
#define LLM_INT8_KV_H

#include "llm_int8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum li8_dtype { LI8_F16 = 0, LI8_BF16 = 1 } li8_dtype;

/* The cache: device memory owned by the caller (plain description, copied
 * at the call). */
typedef struct li8_kv_cache {
    int8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t pages;     /* 0 <= pages < 2^31                                */
    int32_t heads;     /* key/value heads, 1 .. 65535                      */
    int32_t page_size; /* 16, 32, 64 or 128 tokens                         */
    int32_t head_dim;  /* 64 or 128                                        */
} li8_kv_cache;

/*
 * A batch of sequences.  Sequence s has kv_len[s] tokens, of which the last
 * n = q_start[s+1] - q_start[s] are the rows q_start[s] .. q_start[s+1]-1 of
 * the packed token tensors; row q_start[s] + i is at position
 * kv_len[s] - n + i.  Tokens p of sequence s are held by page
 * table[s * table_stride + p / page_size].
 */
typedef struct li8_kv_batch {
    const int32_t *q_start; /* [seqs + 1], ascending                       */
    const int32_t *kv_len;  /* [seqs], the chunk's own tokens included     */
    const int32_t *table;   /* [seqs] rows of table_width page numbers     */
    int64_t table_stride;   /* elements between rows, >= table_width       */
    int32_t table_width;
    int32_t seqs;
    int32_t tokens;         /* rows of the packed tensors                  */
    int32_t max_q;          /* >= the longest chunk                        */
    int32_t max_kv;         /* >= the longest sequence,
                               <= table_width * page_size and 2^30         */
} li8_kv_batch;

/*
 * Rotation of the first `dims` values of every head by position: with
 * c = cos[p][i], s = sin[p][i] for the token at position p,
 *   (a, b) -> (fl32(fl32(a*c) - fl32(b*s)), fl32(fl32(b*c) + fl32(a*s)))
 * for the pairs a = x[i], b = x[i + dims/2] or, interleaved, a = x[2i],
 * b = x[2i + 1].  Values past `dims` stay as they are.
 */
typedef struct li8_rope {
    const float *cos, *sin; /* fp32 [rows][dims / 2]                       */
    int32_t rows;           /* >= max_kv                                   */
    int32_t dims;           /* a multiple of 16, at most head_dim          */
    int32_t interleaved;    /* 0 or 1                                      */
} li8_rope;

/*
 * Stores the batch's new tokens.  For every page that they touch and every
 * head, with x the new rows (keys rotated in fp32), a = max |x| over them,
 * and "old rows" the tokens before the chunk in the page:
 *   s = max(fl32(a / 127), old scale)   (no old rows: fl32(a / 127))
 *   r = min(fl32(1 / s), FLT_MAX), 0 for s = 0
 *   code = clamp(rne(fl32(x * r)), -127, 127)
 * and where s is larger than the old scale the old rows are coded again,
 * code = clamp(rne(fl32(fl32(code * old scale) * r)), -127, 127).  A page
 * whose first token is new forgets what it held.  Coding again is off by at
 * most half a new step each time; a scale never shrinks while its page has
 * old rows.  (The product with the reciprocal differs from a division only
 * for values within about 2^-17 of a step of a rounding border.)
 *   K, V    [tokens][heads][head_dim], rows k_stride, v_stride apart
 *   rope    NULL: keys are stored as they are
 * Tokens at negative positions (kv_len[s] < n) are left out.  A page must
 * not be written twice in a batch, for two sequences or for two places in the
 * table row of one.  Codes of a page behind
 * the sequence's last token, and pages that hold no new token, keep their
 * contents.  Appending the same tokens twice gives the same cache.
 */
li8_status int8_kv_append(const void *K, int64_t k_stride, const void *V, int64_t v_stride,
                          li8_dtype dtype, const li8_rope *rope, const li8_kv_batch *batch,
                          const li8_kv_cache *cache, hipStream_t stream);

/*
 * Reads tokens back: the values of the last n tokens of every sequence into
 * rows q_start[s] ..  of K and V, each fl32(code * scale) rounded to dtype.
 * The inverse of int8_kv_append on the same batch (n may be as large as
 * kv_len[s]).  Tokens at negative positions and in pages that do not exist
 * read as zeros; rows outside every chunk are not written.
 */
li8_status int8_kv_read(const li8_kv_cache *cache, const li8_kv_batch *batch, li8_dtype dtype,
                        void *K, int64_t k_stride, void *V, int64_t v_stride, hipStream_t stream);

/*
 * Attention of the batch's rows over the cache, after their own keys and
 * values were appended.  Query head j reads key/value head j / (q_heads /
 * heads).  With p the row's position, a key at position t is seen if
 *   t < kv_len, t <= p (causal != 0), t > p - window (window > 0);
 *   z[t] = scale * (rotated q) . (k code * k scale)
 *   O    = sum_t softmax(z)[t] * (v code * v scale)     over the seen keys
 *   lse  = log sum_t exp(z[t])                          (natural logarithm)
 * A row that sees nothing gets O = 0 and lse = -inf; rows of no sequence, and
 * those of a chunk past max_q, are not written.  The products run on
 * the matrix units: q as 15-bit integers of its row's largest magnitude
 * (two int8 parts) times the key codes, exact in int32; the softmax in fp32;
 * the probabilities rounded to fp16 (in some kernels in two parts) times the
 * value codes, summed in fp32.
 *   scale   >= 0 and below 10^29 (else refused), and such that scale sum |q| |k|
 *           stays below it for any row and key, |k| as large as its page's
 *           scale allows (127 of it)
 *   Q, O    [tokens][q_heads][head_dim], rows q_stride, o_stride apart;
 *           O must not alias Q (O == Q is refused)
 *   rope    as for the keys; a negative position (only without `causal`
 *           does it see anything) is rotated as position 0
 *   lse     [tokens][q_heads] or NULL
 *   workspace  int8_kv_attention_workspace_bytes(...) bytes; NULL is
 *           accepted where that is 0; its contents do not matter.  Calls that
 *           may run at once (two streams, two graphs) need one each.
 * The same call repeats bit for bit.  A long sequence's keys are divided over
 * workgroups by the lengths of the whole batch, max_q and max_kv, so a row's
 * last bits can differ between batches.  Value scales of a sequence and head
 * more than 2^10 apart cost the pages with the small ones precision: their
 * probabilities are held in fp16 relative to the largest scale so far.
 * Value scales below 2^-126 count as 0.
 * One kernel runs for the whole batch, chosen by its longest chunk: single
 * tokens over long sequences are better put into a call of their own than
 * beside a prompt's chunk (one of 131071 keys beside a chunk of 512 over 2048:
 * 3264 us, apart 56 and 65).
 */
size_t int8_kv_attention_workspace_bytes(const li8_kv_batch *batch, const li8_kv_cache *cache,
                                         int32_t q_heads);
li8_status int8_kv_attention(const void *Q, int64_t q_stride, li8_dtype dtype, int32_t q_heads,
                             float scale, const li8_rope *rope, int32_t causal, int32_t window,
                             const li8_kv_batch *batch, const li8_kv_cache *cache, void *O,
                             int64_t o_stride, float *lse, void *workspace,
                             size_t workspace_bytes, hipStream_t stream);

/*
 * How int8_kv_attention runs a batch of this shape (introspection; nothing
 * is enqueued, no pointer is looked at):
 *   *path    LI8_KV_EMPTY   no rows, nothing is launched
 *            LI8_KV_FEW     16 or 32 query columns (tokens x heads of a
 *                           group) per workgroup
 *            LI8_KV_TILED   256 query columns per workgroup
 *   *splits  the most parts that a row's keys are split into (1: one launch,
 *            else a second one merges the parts)
 */
enum { LI8_KV_EMPTY = 0, LI8_KV_FEW = 1, LI8_KV_TILED = 2 };
li8_status int8_kv_attention_plan(const li8_kv_batch *batch, const li8_kv_cache *cache,
                                  int32_t q_heads, int32_t causal, int32_t window, int32_t *path,
                                  int32_t *splits);

#ifdef __cplusplus
}
#endif

#endif /* LLM_INT8_KV_H */
