/*
 * mxfp4.h -- C ABI of the MXFP4 operators and the MoE router of libq8_0.so
 * (AMD MI355X, gfx950): the routed experts of the engine whose 8-bit
 * projections are in q8_0.h, held in 4 bits.
 *
 * MXFP4 block (OCP Microscaling Formats, v1.0): 32 values that share one
 * scale.  A value is a 4-bit e2m1 code -- bit 3 the sign, the magnitudes of
 * codes 0..7 being 0, 0.5, 1, 1.5, 2, 3, 4, 6 -- times 2^(s - 127), s being the
 * block's e8m0 scale byte; s = 255 makes every value of the block NaN.
 * A matrix [rows][k] (k a multiple of 32) is two arrays:
 *   codes  : rows * k/2 bytes, row-major; byte j of a row holds value 2j in its
 *            low half and value 2j + 1 in its high half.
 *   scales : rows * k/32 bytes, row-major.
 * The two arrays are separate so that a block's 16 code bytes are one aligned
 * matrix-core operand and rows can be sliced without a copy.
 *
 * Conventions are those of q8_0.h: device pointers owned by the caller, no
 * allocation, work only enqueued on `stream`, argument errors found on the host
 * before anything is enqueued and returned as Q8_0_E* codes (q8_0_strerror),
 * deterministic results.  `codes` arrays must be 16-byte aligned (every row then
 * is: rows are k/2 bytes), `scales` arrays may have any alignment.  The current
 * device must be the one that owns `stream` and the buffers.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "q8_0.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MXFP4_BLOCK_ELEMS 32

/* Element types of unquantized inputs and outputs. */
enum { MXFP4_F32 = 0, MXFP4_BF16 = 1, MXFP4_F16 = 2 };

/* Quantize rows to MXFP4.
 *   codes, scales : [n_rows][in_dim], written.
 *   x        : [n_rows][in_dim] of x_type, row r starting at element r * x_stride
 *              (x_stride >= in_dim; any alignment the type has).
 * Per block: amax = max|x_i|, E = max(floor(log2 amax) - 2, -127), scale byte
 * E + 127 (0 when amax == 0); code i = x_i * 2^-E rounded to the nearest e2m1
 * value, ties to the even code, magnitudes above 6 held at 6 (the sign is kept,
 * also of values that round to zero).  The arithmetic is exact, so the result
 * is bit-exact for every input.  A block holding a NaN or an infinity is stored
 * with scale byte 255 (NaN) and zero codes.
 * Errors: in_dim % 32 != 0, negative sizes, x_stride < in_dim, unknown type,
 * null pointers -> Q8_0_EINVAL; codes not 16-byte aligned or x not aligned to
 * its type -> Q8_0_EALIGN. */
int mxfp4_quantize(void *codes, void *scales, const void *x, int32_t x_type, int64_t x_stride,
                   int64_t n_rows, int64_t in_dim, hipStream_t stream);

/* The values an MXFP4 matrix stands for.
 *   out : [n_rows][in_dim] of out_type, row-major, written.  Exact in fp32 and bf16
 *         for every block (subnormals included); fp16 rounds to nearest even and
 *         overflows to infinity.  Blocks of scale byte 255 give NaN.
 * Errors as mxfp4_quantize (out needs 16-byte alignment). */
int mxfp4_dequantize(void *out, int32_t out_type, const void *codes, const void *scales,
                     int64_t n_rows, int64_t in_dim, hipStream_t stream);

/* Scores of moe_topk, from a token's logits z. */
enum {
    MOE_SOFTMAX = 0,      /* exp(z) / sum exp(z); ordered by z itself */
    MOE_SIGMOID = 1,      /* 1 / (1 + exp(-z))                       */
    MOE_SQRT_SOFTPLUS = 2 /* sqrt(log(1 + exp(z)))                   */
};

#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_USED 32

/* The router: each token's n_used experts of largest score + bias, largest
 * first, ties to the lowest id, with their weights.  Its outputs are the
 * `selected` and `weights` of q8_0_moe_ffn and q8_0_moe_grouped.
 *   selected : int32 [n_tok][n_used], written.
 *   weights  : fp32 [n_tok][n_used], written: the scores (without bias) of the
 *              chosen experts, divided by their sum if renormalize is set (for
 *              MOE_SOFTMAX without it, by the sum over all experts), times `scale`
 *              (a sum of exactly zero divides nothing: those weights are 0).
 *   logits   : fp32 [n_tok][n_expert] (a router projection's output).
 *   bias     : fp32 [n_expert] added to the score for the choice only (to the
 *              logit for MOE_SOFTMAX), or NULL.
 * An expert whose logit or biased score is -infinity is never chosen: a token
 * with fewer than n_used others gets id -1 and weight 0 in its last slots (all
 * of them for a token whose logits are all -infinity, e.g. padding).  NaN keys
 * come before all others, and a NaN or +infinite score among those summed
 * makes the weights that its sum divides NaN.
 * MOE_SOFTMAX compares z + bias in fp32; the other scores are formed and
 * compared in 64 bits.
 * Errors: n_expert outside [1, MOE_MAX_EXPERTS], n_used outside [1,
 * min(n_expert, MOE_MAX_USED)], n_tok * n_used above 2^31 - 1, unknown scoring,
 * null pointers -> Q8_0_EINVAL; pointers not 4-byte aligned -> Q8_0_EALIGN. */
int moe_topk(int32_t *selected, float *weights, const float *logits, const float *bias,
             int64_t n_tok, int32_t n_expert, int32_t n_used, int32_t scoring,
             int32_t renormalize, float scale, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
