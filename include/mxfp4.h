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
 *         (subnormals included) but for values of 2^128 and above, which scale bytes
 *         253 and 254 can stand for and mxfp4_quantize does not make (252 is its
 *         largest): those are infinite.  fp16 rounds to nearest even and overflows to
 *         infinity.  Blocks of scale byte 255 give NaN.
 * Errors as mxfp4_quantize (out needs 16-byte alignment). */
int mxfp4_dequantize(void *out, int32_t out_type, const void *codes, const void *scales,
                     int64_t n_rows, int64_t in_dim, hipStream_t stream);

/* Workspace bytes of mxfp4_matmul's fastest plan for this shape (partial sums
 * of a split over in_dim); 0 when it needs none or the shape is invalid. */
size_t mxfp4_matmul_workspace_bytes(int64_t in_dim, int64_t out_dim, int64_t n_tok);

/* MXFP4 product, the 4-bit counterpart of q8_0_matmul:
 *   out[t][o] = sum_b 2^(sw[o][b] + sx[t][b] - 254) * sum_{i<32} w[o][b][i] * x[t][b][i]
 *   out    : [n_tok][out_dim] of out_type, written (fp32 sums, rounded once).
 *   w_*    : MXFP4 [out_dim][in_dim]; x_* : MXFP4 [n_tok][in_dim] (e.g. from
 *            mxfp4_quantize).
 *   workspace / workspace_bytes : optional scratch (16-byte aligned device
 *            memory; its contents on entry do not matter).  With less than
 *            mxfp4_matmul_workspace_bytes() the library picks a plan that fits;
 *            NULL / 0 is always valid.  Calls that share a workspace must not
 *            overlap in time.
 * Products are exact and summed in fp32: |out - exact| <= (in_dim / 32 + 8) *
 * 2^-23 * sum |w x| + in_dim * 2^-125 before the rounding to out_type (the second
 * part is what terms and sums below fp32's normal numbers may lose).  Where a term
 * or a partial sum exceeds fp32's largest number, as it can where sum |w x| reaches
 * 2^127, that output is infinite or NaN; no other output is touched.  A NaN block
 * makes every output that uses it NaN.
 * n_tok == 0 or out_dim == 0 is a successful no-op.
 * Errors: in_dim % 32 != 0, in_dim == 0 with work to do, in_dim above 2^24,
 * out_dim or n_tok above 2^28, out_dim * n_tok above 2^35, negative sizes,
 * unknown type, null pointers -> Q8_0_EINVAL; codes or workspace not 16-byte
 * aligned, out not aligned to its type -> Q8_0_EALIGN. */
int mxfp4_matmul(void *out, int32_t out_type, const void *w_codes, const void *w_scales,
                 int64_t in_dim, int64_t out_dim, const void *x_codes, const void *x_scales,
                 int64_t n_tok, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Scores of moe_topk, from a token's logits z. */
enum {
    MOE_SOFTMAX = 0,      /* exp(z) / sum exp(z); ordered by z + bias */
    MOE_SIGMOID = 1,      /* 1 / (1 + exp(-z))                       */
    MOE_SQRT_SOFTPLUS = 2 /* sqrt(log(1 + exp(z)))                   */
};

#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_USED 32

/* The router: each token's n_used experts of largest key, largest first, ties to
 * the lowest id, with their weights.  Its outputs are the `selected` and `weights`
 * of q8_0_moe_ffn and q8_0_moe_grouped.
 *   key      : score + bias for MOE_SIGMOID and MOE_SQRT_SOFTPLUS; the logit + bias
 *              for MOE_SOFTMAX.  Without a bias that is the order of the
 *              probabilities, with one the order of probability * exp(bias).  A
 *              bias that a model adds to the softmax probabilities themselves gives
 *              another order and is not what this call computes.
 *   selected : int32 [n_tok][n_used], written.
 *   weights  : fp32 [n_tok][n_used], written: the scores (without bias) of the
 *              chosen experts, divided by their sum if renormalize is set (for
 *              MOE_SOFTMAX without it, by the sum over all experts), times `scale`.
 *              The sum may lie far below fp32's range; where it is zero in 64 bits
 *              (logits below -745) it divides nothing and those weights are 0.
 *   logits   : fp32 [n_tok][n_expert] (a router projection's output).
 *   bias     : fp32 [n_expert], part of the key only, or NULL.
 * An expert whose logit or key is -infinity is never chosen: a token with fewer
 * than n_used others gets id -1 and weight 0 in its last slots (all of them for a
 * token whose logits are all -infinity, e.g. padding).  NaN keys come before all
 * others.  A NaN score among those summed makes the weights that its sum divides
 * NaN, and so does a +infinite logit for MOE_SOFTMAX; a +infinite MOE_SQRT_SOFTPLUS
 * score that is divided by its sum is NaN itself, beside others of 0.
 * MOE_SOFTMAX compares z + bias in fp32; the other scores are formed and
 * compared in 64 bits.
 * Errors: n_expert outside [1, MOE_MAX_EXPERTS], n_used outside [1,
 * min(n_expert, MOE_MAX_USED)], n_tok above 2^25, unknown scoring,
 * null pointers -> Q8_0_EINVAL; pointers not 4-byte aligned -> Q8_0_EALIGN. */
int moe_topk(int32_t *selected, float *weights, const float *logits, const float *bias,
             int64_t n_tok, int32_t n_expert, int32_t n_used, int32_t scoring,
             int32_t renormalize, float scale, hipStream_t stream);

#define MXFP4_MOE_MAX_TOKENS 64
#define MXFP4_MOE_MAX_EXPERTS 512

/* Arguments of mxfp4_moe_layer. */
typedef struct mxfp4_moe_layer_args {
    void *out;               /* [n_tok][d_model] of out_type, written                */
    const void *x;           /* [n_tok][d_model] of x_type: the layer's input        */
    int32_t out_type, x_type;
    const float *logits;     /* fp32 [n_tok][n_expert]: router logits                */
    const float *bias;       /* fp32 [n_expert], or NULL (as moe_topk)               */
    int32_t n_expert;        /* 1 .. MXFP4_MOE_MAX_EXPERTS                           */
    int32_t n_used;          /* experts per token, as moe_topk                       */
    int32_t scoring;         /* MOE_SOFTMAX, ...                                     */
    int32_t renormalize;
    float scale;
    float clamp;             /* SwiGLU limit; <= 0 or NaN: no clamp                  */
    int64_t d_model;         /* expert input and output width, a multiple of 32      */
    int64_t d_ff;            /* expert hidden width, a multiple of 32                */
    int64_t n_tok;           /* 0 .. MXFP4_MOE_MAX_TOKENS                            */
    const void *gate_codes, *gate_scales; /* MXFP4 [n_expert][d_ff][d_model]         */
    const void *up_codes, *up_scales;     /* MXFP4 [n_expert][d_ff][d_model]         */
    const void *down_codes, *down_scales; /* MXFP4 [n_expert][d_model][d_ff]         */
    int32_t *selected;       /* optional int32 [n_tok][n_used]: moe_topk's ids       */
    float *weights;          /* optional fp32 [n_tok][n_used]: moe_topk's weights    */
} mxfp4_moe_layer_args;

/* Workspace bytes mxfp4_moe_layer needs (routing tables, the quantized x and the
 * quantized mid of every pair); 0 for sizes it refuses. */
size_t mxfp4_moe_layer_workspace_bytes(int64_t n_tok, int32_t n_used, int32_t n_expert,
                                       int64_t d_model, int64_t d_ff);

/* The whole MoE layer for a few tokens, from router logits to the weighted sum
 * of the experts, in two kernels up to eight tokens (and 256 experts, and
 * n_tok * d_model about 2^16) and three above (q8_0_moe_ffn is its 8-bit
 * counterpart from given ids on).  For token t, with (e_j, w_j) = moe_topk of its logits:
 *   x4    = mxfp4_quantize(x_t)
 *   gate  = W_gate[e_j] x4, up = W_up[e_j] x4          (products as mxfp4_matmul)
 *   mid   = silu(gate) * up, silu(g) = g / (1 + exp(-g)), after the optional
 *           limits (gate from above, up to +-clamp)    (fp32)
 *   out_t = sum_j w_j W_down[e_j] mxfp4_quantize(mid)  (fp32 sums, rounded once)
 * Equal calls give equal bits.  The order in which a token's experts are summed
 * depends on the sizes and on the experts that the call's tokens choose, so the
 * last bits of a token alone and of the same token among others may differ.
 * Each touched expert's matrices are loaded once for every 16 of its tokens, and
 * the activation is the plain SwiGLU above, without biases.  Slots without an
 * eligible expert add nothing: a token whose logits are all -infinity (padding)
 * gives zeros.
 *   workspace : device memory, 256-byte aligned, contents on entry do not
 *     matter; calls that share one must not overlap in time.
 * Errors: bad sizes (as above and moe_topk's; d_model and d_ff up to 2^20;
 * n_expert * d_model * d_ff up to 2^46), unknown types or scoring, null
 * pointers -> Q8_0_EINVAL; codes, x, out or workspace not 16-byte (workspace:
 * 256-byte) aligned, other pointers not 4-byte aligned (scales: any) ->
 * Q8_0_EALIGN; workspace smaller than mxfp4_moe_layer_workspace_bytes() ->
 * Q8_0_EWORKSPACE. */
int mxfp4_moe_layer(const mxfp4_moe_layer_args *args, void *workspace, size_t workspace_bytes,
                    hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
