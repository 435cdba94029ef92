/*
 * kv8.h -- C ABI of the 8-bit key/value cache of libq8_0.so (AMD MI355X,
 * gfx950): writing new tokens into a paged cache, reading tokens back, and
 * causal attention over it, for single tokens and for prompts.  It stands
 * between the projections of q8_0.h that make queries, keys and values and the
 * output projection.
 *
 * The cache is a pool of pages.  A page holds page_size tokens of every
 * key/value head: their int8 codes and one fp32 scale for each block of `block`
 * tokens and head, keys and values apart.  A value is code * scale.
 *   k_codes  : int8 [n_pages][n_kv][page_size / 16][head_dim / 16][16 tokens][16 dims]
 *   v_codes  : int8 [n_pages][n_kv][page_size / 4][head_dim][4 tokens]
 *   k_scales, v_scales : fp32 [n_pages][n_kv][page_size / block]
 * (Tokens lie in the order in which the matrix core takes them: 16 tokens of 64
 * dims are 1024 adjacent bytes, one load of a wave.)
 * A block's scale covers its tokens written so far.  Tokens that are written
 * later may raise it; the block's older codes are then rounded to the new scale
 * (each raise moves an older value by at most half of the new scale).
 * A block whose scale is NaN holds NaN values (it was given a NaN or an
 * infinity) until its first token is written anew.
 *
 * Conventions are those of q8_0.h: device pointers owned by the caller, no
 * allocation, work only enqueued on `stream`, argument errors found on the host
 * before anything is enqueued and returned as Q8_0_E* codes (q8_0_strerror),
 * deterministic results.  The current device must be the one that owns `stream`
 * and the buffers.  Page tables and lengths are read by the kernels, so a
 * captured graph may be replayed with other contents; values out of range never
 * lead out of the buffers (below, at each call).
 */
#ifndef KV8_H
#define KV8_H

#include "q8_0.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of unquantized inputs and outputs. */
enum { KV8_F32 = 0, KV8_BF16 = 1, KV8_F16 = 2 };

/* A pool of pages.  Codes must be 16-byte aligned, scales 4-byte aligned. */
typedef struct kv8_cache {
    void *k_codes, *v_codes;
    float *k_scales, *v_scales; /* not negative, as kv8_write makes them             */
    int64_t n_pages;    /* 1 .. 2^31 - 1                                            */
    int32_t n_kv;       /* key/value heads, 1 .. 4096                               */
    int32_t head_dim;   /* 64, 128, 192, 256 or 512                                 */
    int32_t page_size;  /* tokens of a page: a power of two, 16 .. 1024             */
    int32_t block;      /* tokens under one scale: a power of two, 16 .. min(128, page_size) */
} kv8_cache;

/* A ragged batch of sequences and their newest tokens.
 * Sequence s has lens[s] tokens; rows starts[s] .. starts[s + 1] - 1 of the
 * call's token arrays are its last ones, in order: row i is at position
 * lens[s] - starts[s + 1] + i.  The token at position p is in page
 * page_table[s][p / page_size].
 * Entries of the table beyond a sequence's length are not looked at.  lens[s]
 * is held within 0 .. table_width * page_size, starts within 0 .. n_tok. */
typedef struct kv8_batch {
    const int32_t *page_table;  /* int32 [n_seq][table_width]                        */
    const int32_t *lens;        /* int32 [n_seq]                                     */
    const int32_t *starts;      /* int32 [n_seq + 1], ascending from 0; NULL: one row each */
    int64_t n_seq;              /* 0 .. 2^20, and n_seq * n_kv <= 2^22               */
    int64_t n_tok;              /* rows of the token arrays, 0 .. 2^24; n_seq where starts is NULL */
    int64_t table_width;        /* pages of a table row; table_width * page_size <= 2^30 */
    int64_t max_new;            /* no sequence may have more rows than this (1 where starts is NULL) */
    int64_t max_len;            /* no lens[s] is above this: work is spread by it; 0: unknown */
} kv8_batch;

/* Write the batch's rows into the cache.
 *   k, v : [n_tok][n_kv][head_dim] of `type`; token t's head h starts at element
 *          t * token_stride + h * head_stride (any strides >= 0, head_dim
 *          adjacent values; any alignment the type has, 16-byte aligned rows are
 *          the fast ones).
 * Per block and head, N being its new rows and O its tokens before the first of
 * them:
 *   s1 = max(|N|) / 127 in fp32, or the old scale where O is not empty and that is larger
 *   new codes = N / s1 rounded to nearest even (the exact quotient, held within -127 .. 127,
 *   which subnormal scales alone exceed; 0 where s1 is 0),
 *   O's codes = code * s0 / s1 rounded to nearest even, where the scale grew from s0.
 * A NaN or an infinity in N, or a NaN scale of O, gives s1 = NaN and new codes 0.
 * Codes are bit-exact for every input.  Tokens of the block behind the new ones
 * keep their bytes.  Two sequences of a batch must not write into one block.
 * Rows at negative positions (starts beyond lens) and rows whose page id is
 * outside 0 .. n_pages - 1 are skipped.
 * Errors: sizes out of the ranges above, unknown type, negative strides, null
 * pointers -> Q8_0_EINVAL; misaligned pointers -> Q8_0_EALIGN. */
int kv8_write(const kv8_cache *cache, const kv8_batch *batch, const void *k, int64_t k_token_stride,
              int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
              int32_t type, hipStream_t stream);

/* Read the batch's rows back (all of a sequence where it has lens[s] rows).
 *   k, v : [n_tok][n_kv][head_dim] of `type`, written: code * scale in fp32, rounded
 *          once to the type; 16-byte aligned.  Either may be NULL.
 * Rows at negative positions are zeros, rows of a page id out of range NaN; rows
 * behind the last sequence are left as they were.
 * Errors as kv8_write. */
int kv8_read(const kv8_cache *cache, const kv8_batch *batch, void *k, void *v, int32_t type,
             hipStream_t stream);

/* Arguments of kv8_attention beside the cache and the batch. */
typedef struct kv8_attention_args {
    void *out;             /* [n_tok][n_q][head_dim] of out_type, written, 16-byte aligned  */
    const void *q;         /* [n_tok][n_q][head_dim] of q_type                               */
    int64_t q_token_stride, q_head_stride; /* in elements, as k's of kv8_write               */
    int32_t out_type, q_type;
    int32_t n_q;           /* query heads, a multiple of n_kv, up to 2^14, and n_tok * n_q <= 2^27; head h reads key/value head h / (n_q / n_kv) */
    int32_t window;        /* keys a row sees, its own among them; 0: all before it          */
    float scale;           /* on the scores, e.g. 1 / sqrt(head_dim)                         */
    const float *sinks;    /* optional fp32 [n_q]: a score without a value, per head         */
    float *lse;            /* optional fp32 [n_tok][n_q], written                            */
} kv8_attention_args;

/* Workspace bytes of kv8_attention's fastest plan without a window (partial outputs of a
 * split over the keys); 0 when it needs none or the arguments are invalid. */
size_t kv8_attention_workspace_bytes(const kv8_cache *cache, const kv8_batch *batch, int32_t n_q);

/* Causal attention of the batch's rows over their sequences' cached tokens (the
 * rows' own keys and values must have been written before).  For row i at
 * position p and query head h:
 *   z_j = scale * q . (k code_j * k scale_j),  max(0, p - window + 1) <= j <= p
 *   out = sum_j exp(z_j) (v code_j * v scale_j) / (exp(sink_h) + sum_j exp(z_j))
 *   lse = log(exp(sink_h) + sum_j exp(z_j))     (without sinks the term is left out)
 * A row without keys (a position below 0, a sequence of length 0) gives zeros and
 * lse = sink or -infinity.  Keys that a row does not see have no part in it,
 * whatever their scales hold.  Rows behind the last sequence are left as they were.
 * A NaN scale makes the rows that see its tokens NaN (one of V not their lse, which has
 * no V in it), and so does a page id out of 0 .. n_pages - 1.  A NaN or an infinity in a
 * query makes that row NaN.
 * Numbers: codes enter the matrix core exactly as fp16, queries as fp16 under a
 * power of two per row (16-bit queries exactly, but for values below 2^-28 of the
 * row's largest), fp32 queries as two such halves; exp, sums and outputs are fp32.
 * A key's weight and V scale become one factor under the largest V scale that the row
 * sees.  It is rounded to fp16 (11 bits) for 16-bit outputs and queries, and kept in
 * two halves (22 bits) where out_type or q_type is KV8_F32, either way no finer than
 * 2^-31 of the largest weight under that scale (so values of V lose some of the 11 bits from
 * 2^21 below others that the row sees on, some of the 22 from 2^10 below).
 *   workspace / workspace_bytes : optional scratch, 16-byte aligned device memory, its
 *     contents on entry do not matter.  With less than
 *     kv8_attention_workspace_bytes() a plan with fewer splits that fits is taken;
 *     NULL / 0 is always valid.  Calls that share a workspace must not overlap in time.
 * Equal calls give equal bits; the order of a row's sums depends on the batch's sizes.
 * Errors: sizes out of the ranges above, n_q not a multiple of n_kv, negative
 * window, a scale that is not finite, unknown types, null pointers ->
 * Q8_0_EINVAL; misaligned pointers -> Q8_0_EALIGN. */
int kv8_attention(const kv8_cache *cache, const kv8_batch *batch, const kv8_attention_args *args,
                  void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Kernel variants (for kv8_attention_debug; 0 lets the library choose). */
enum {
    KV8_KERNEL_AUTO = 0,
    KV8_KERNEL_STREAM = 1, /* 16 query rows a workgroup, codes straight from memory        */
    KV8_KERNEL_TILED = 2   /* 64 to 256 query rows a workgroup, codes through LDS as fp16;
                              not for heads of 512 where out_type or q_type is KV8_F32     */
};

/* Test hook: kv8_attention by the given kernel with `splits` splits over the keys (0 or 1:
 * none, up to 256; their workspace is splits * n_tok * n_q * (head_dim + 1) * 4 bytes).  With
 * KV8_KERNEL_AUTO splits must be 0.
 * Errors as kv8_attention; a kernel, or splits of more than 2^20 rows (n_tok * n_q), that
 * do not exist -> Q8_0_EINVAL; workspace too small -> Q8_0_EWORKSPACE. */
int kv8_attention_debug(const kv8_cache *cache, const kv8_batch *batch, const kv8_attention_args *args,
                        void *workspace, size_t workspace_bytes, int32_t kernel, int32_t splits,
                        hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KV8_H */
