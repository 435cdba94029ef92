// mxfp4_api.hip -- the C ABI of include/mxfp4.h: host-side argument checks and
// launches on the caller's stream.  Nothing here allocates device memory.
#include <stdint.h>

#include "launch.h"
#include "moe_topk.h"
#include "mxfp4.h"
#include "mxfp4_launch.h"

static_assert(MXFP4_F32 == mx::kF32 && MXFP4_BF16 == mx::kBF16 && MXFP4_F16 == mx::kF16,
              "header and library agree on the element types");
static_assert(MOE_SOFTMAX == mx::kSoftmax && MOE_SIGMOID == mx::kSigmoid &&
                  MOE_SQRT_SOFTPLUS == mx::kSqrtSoftplus &&
                  MOE_MAX_EXPERTS == mx::kMaxRouteExperts && MOE_MAX_USED == mx::kMaxUsed,
              "header and library agree on the router");
static_assert(MXFP4_MOE_MAX_TOKENS == mx::kMaxLayerTokens &&
                  MXFP4_MOE_MAX_EXPERTS == mx::kMaxLayerExperts,
              "header and library agree on the layer");

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int32_t t) { return t == MXFP4_F32 || t == MXFP4_BF16 || t == MXFP4_F16; }
int type_size(int32_t t) { return t == MXFP4_F32 ? 4 : 2; }
int status_of(hipError_t e) { return e == hipSuccess ? Q8_0_OK : Q8_0_ELAUNCH; }

// The largest matrix of the elementwise kernels: 2^20 by 2^12 workgroups of 2048 values.
constexpr int64_t kMaxElems = int64_t{1} << 43;

// Sizes of a matrix that a call reads or writes: Q8_0_OK, or EINVAL.
int check_matrix(int64_t rows, int64_t k) {
  if (rows < 0 || k < 0 || k % MXFP4_BLOCK_ELEMS != 0) return Q8_0_EINVAL;
  if (k > 0 && rows > kMaxElems / k) return Q8_0_EINVAL;
  return Q8_0_OK;
}

// Sizes of a product: the kernels count blocks, rows, tokens and tiles in 32 bits, and a
// launch has fewer than 2^32 threads: one for 16 outputs, and less than twice that where
// the last row or token tile is cut.
constexpr int64_t kMaxInDim = 1 << 24, kMaxRows = 1 << 28, kMaxOut = int64_t{1} << 35;
int check_product(int64_t in_dim, int64_t out_dim, int64_t n_tok) {
  if (in_dim < 0 || out_dim < 0 || n_tok < 0 || in_dim % MXFP4_BLOCK_ELEMS != 0) return Q8_0_EINVAL;
  if (in_dim > kMaxInDim || out_dim > kMaxRows || n_tok > kMaxRows || out_dim * n_tok > kMaxOut)
    return Q8_0_EINVAL;
  return Q8_0_OK;
}

// The tiled kernel above 32 tokens; from 17 on where its stages are few or its rows
// many; and never for rows of less than 512 values, whose scales it cannot fetch.
// Measured (us, streaming / tiled): 4096 -> 2048 at 16 tokens 5.0 / 7.7, at 32 6.3 /
// 8.0, at 64 8.6 / 6.8; 1024 -> 4096 at 32 6.2 / 4.2; 1024 -> 32768 at 32 10.3 / 7.5;
// 32768 -> 1024 at 32 12.9 / 13.9, at 64 17.8 / 14.4.
bool use_gemm(int64_t in_dim, int64_t out_dim, int64_t n_tok) {
  if (in_dim < 512 || n_tok <= 16) return false;
  return n_tok > 32 || in_dim <= 2048 || out_dim >= 8192;
}

// A wave each, and fewer than 2^32 threads a launch.
constexpr int64_t kMaxRouteTokens = 1 << 25;

int check_route(const float *logits, const float *bias, int64_t n_tok, int32_t n_expert,
                int32_t n_used, int32_t scoring) {
  if (n_tok < 0 || n_expert < 1 || n_expert > MOE_MAX_EXPERTS || n_used < 1 || n_used > n_expert ||
      n_used > MOE_MAX_USED || scoring < MOE_SOFTMAX || scoring > MOE_SQRT_SOFTPLUS)
    return Q8_0_EINVAL;
  if (n_tok > kMaxRouteTokens) return Q8_0_EINVAL;
  if (n_tok == 0) return Q8_0_OK;
  if (!logits) return Q8_0_EINVAL;
  if (!aligned(logits, 4) || !aligned(bias, 4)) return Q8_0_EALIGN;
  return Q8_0_OK;
}

constexpr int64_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxExpertElems = int64_t{1} << 46;
bool layer_sizes_ok(int64_t n_tok, int32_t n_used, int32_t n_expert, int64_t d_model, int64_t d_ff) {
  return n_tok >= 0 && n_tok <= MXFP4_MOE_MAX_TOKENS && n_expert >= 1 &&
         n_expert <= MXFP4_MOE_MAX_EXPERTS && n_used >= 1 && n_used <= n_expert &&
         n_used <= MOE_MAX_USED && d_model > 0 && d_model <= kMaxWidth && d_ff > 0 &&
         d_ff <= kMaxWidth && d_model % MXFP4_BLOCK_ELEMS == 0 && d_ff % MXFP4_BLOCK_ELEMS == 0 &&
         d_model * d_ff <= kMaxExpertElems / n_expert;
}

int run_layer(const mxfp4_moe_layer_args *a, void *workspace, size_t workspace_bytes,
              hipStream_t stream) {
  if (!a || !layer_sizes_ok(a->n_tok, a->n_used, a->n_expert, a->d_model, a->d_ff) ||
      !type_ok(a->out_type) || !type_ok(a->x_type))
    return Q8_0_EINVAL;
  int st = check_route(a->logits, a->bias, a->n_tok, a->n_expert, a->n_used, a->scoring);
  if (st != Q8_0_OK || a->n_tok == 0) return st;
  if (!a->out || !a->x) return Q8_0_EINVAL;
  for (const void *p : {a->gate_codes, a->gate_scales, a->up_codes, a->up_scales, a->down_codes,
                        a->down_scales})
    if (!p) return Q8_0_EINVAL;
  for (const void *p : {a->gate_codes, a->up_codes, a->down_codes, a->x, (const void *)a->out})
    if (!aligned(p, 16)) return Q8_0_EALIGN;
  if (!aligned(a->selected, 4) || !aligned(a->weights, 4)) return Q8_0_EALIGN;
  if (!workspace || workspace_bytes < mx::moe_layer_workspace_bytes(a->n_tok, a->n_used, a->n_expert, a->d_model, a->d_ff))
    return Q8_0_EWORKSPACE;
  if (!aligned(workspace, 256)) return Q8_0_EALIGN;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  const mx::RouteArgs route{a->logits, a->bias, a->n_expert, a->n_used, a->scoring,
                            a->renormalize != 0, a->scale};
  auto u8 = [](const void *p) { return static_cast<const uint8_t *>(p); };
  const mx::MoeLayer m{a->out, a->out_type, a->x, a->x_type, &route,
                       u8(a->gate_codes), u8(a->gate_scales), u8(a->up_codes), u8(a->up_scales),
                       u8(a->down_codes), u8(a->down_scales), a->d_model, a->d_ff, a->n_tok,
                       a->clamp, a->selected, a->weights};
  return status_of(mx::launch_moe_layer(m, static_cast<uint8_t *>(workspace), stream));
}

}  // namespace

extern "C" {

int mxfp4_quantize(void *codes, void *scales, const void *x, int32_t x_type, int64_t x_stride,
                   int64_t n_rows, int64_t in_dim, hipStream_t stream) {
  int st = check_matrix(n_rows, in_dim);
  if (st != Q8_0_OK || !type_ok(x_type) || x_stride < in_dim) return Q8_0_EINVAL;
  if (n_rows == 0 || in_dim == 0) return Q8_0_OK;
  if (!codes || !scales || !x) return Q8_0_EINVAL;
  if (!aligned(codes, 16) || !aligned(x, type_size(x_type))) return Q8_0_EALIGN;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  return status_of(mx::launch_quantize(static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales),
                                       x, x_type, x_stride, n_rows, in_dim, stream));
}

int mxfp4_dequantize(void *out, int32_t out_type, const void *codes, const void *scales,
                     int64_t n_rows, int64_t in_dim, hipStream_t stream) {
  int st = check_matrix(n_rows, in_dim);
  if (st != Q8_0_OK || !type_ok(out_type)) return Q8_0_EINVAL;
  if (n_rows == 0 || in_dim == 0) return Q8_0_OK;
  if (!out || !codes || !scales) return Q8_0_EINVAL;
  if (!aligned(codes, 16) || !aligned(out, 16)) return Q8_0_EALIGN;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  return status_of(mx::launch_dequantize(out, out_type, static_cast<const uint8_t *>(codes),
                                         static_cast<const uint8_t *>(scales), n_rows, in_dim,
                                         stream));
}

size_t mxfp4_matmul_workspace_bytes(int64_t in_dim, int64_t out_dim, int64_t n_tok) {
  if (check_product(in_dim, out_dim, n_tok) != Q8_0_OK || in_dim == 0 || out_dim == 0 || n_tok == 0)
    return 0;
  return use_gemm(in_dim, out_dim, n_tok) ? mx::gemm_workspace_bytes(in_dim, out_dim, n_tok)
                                          : mx::stream_workspace_bytes(in_dim, out_dim, n_tok);
}

int mxfp4_matmul(void *out, int32_t out_type, const void *w_codes, const void *w_scales,
                 int64_t in_dim, int64_t out_dim, const void *x_codes, const void *x_scales,
                 int64_t n_tok, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_product(in_dim, out_dim, n_tok);
  if (st != Q8_0_OK || !type_ok(out_type)) return Q8_0_EINVAL;
  if (n_tok == 0 || out_dim == 0) return Q8_0_OK;
  if (in_dim == 0 || !out || !w_codes || !w_scales || !x_codes || !x_scales) return Q8_0_EINVAL;
  if (!aligned(w_codes, 16) || !aligned(x_codes, 16) || !aligned(out, type_size(out_type)) ||
      !aligned(workspace, 16))
    return Q8_0_EALIGN;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  const auto *w = static_cast<const uint8_t *>(w_codes), *ws = static_cast<const uint8_t *>(w_scales);
  const auto *x = static_cast<const uint8_t *>(x_codes), *xs = static_cast<const uint8_t *>(x_scales);
  if (!workspace) workspace_bytes = 0;
  if (use_gemm(in_dim, out_dim, n_tok)) {
    const mx::GemmPlan p = mx::gemm_plan(in_dim, out_dim, n_tok, workspace_bytes);
    return status_of(mx::launch_gemm(p, out, out_type, w, ws, in_dim, out_dim, x, xs, n_tok,
                                     workspace, stream));
  }
  const mx::StreamPlan p = mx::stream_plan(in_dim, out_dim, n_tok, workspace_bytes);
  return status_of(mx::launch_stream(p, out, out_type, w, ws, in_dim, out_dim, x, xs, n_tok,
                                     workspace, stream));
}

int moe_topk(int32_t *selected, float *weights, const float *logits, const float *bias,
             int64_t n_tok, int32_t n_expert, int32_t n_used, int32_t scoring,
             int32_t renormalize, float scale, hipStream_t stream) {
  int st = check_route(logits, bias, n_tok, n_expert, n_used, scoring);
  if (st != Q8_0_OK || n_tok == 0) return st;
  if (!selected || !weights) return Q8_0_EINVAL;
  if (!aligned(selected, 4) || !aligned(weights, 4)) return Q8_0_EALIGN;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  const mx::RouteArgs a{logits, bias, n_expert, n_used, scoring, renormalize != 0, scale};
  return status_of(mx::launch_topk(a, n_tok, selected, weights, stream));
}

size_t mxfp4_moe_layer_workspace_bytes(int64_t n_tok, int32_t n_used, int32_t n_expert,
                                       int64_t d_model, int64_t d_ff) {
  if (!layer_sizes_ok(n_tok, n_used, n_expert, d_model, d_ff)) return 0;
  return mx::moe_layer_workspace_bytes(n_tok, n_used, n_expert, d_model, d_ff);
}

int mxfp4_moe_layer(const mxfp4_moe_layer_args *args, void *workspace, size_t workspace_bytes,
                    hipStream_t stream) {
  return run_layer(args, workspace, workspace_bytes, stream);
}

}  // extern "C"
