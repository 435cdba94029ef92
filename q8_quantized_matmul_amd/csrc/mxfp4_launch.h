// mxfp4_launch.h -- internal host-side launchers of the MXFP4 operators.  Each
// returns hipSuccess or the launch error; argument checks happen in
// mxfp4_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;  // MXFP4_F32, MXFP4_BF16, MXFP4_F16

// mxfp4_quantize.hip
hipError_t launch_quantize(uint8_t *codes, uint8_t *scales, const void *x, int x_type,
                           int64_t x_stride, int64_t n_rows, int64_t in_dim, hipStream_t s);
hipError_t launch_dequantize(void *out, int out_type, const uint8_t *codes, const uint8_t *scales,
                             int64_t n_rows, int64_t in_dim, hipStream_t s);

// mxfp4_matmul.hip: weight streaming, for few tokens.
struct StreamPlan {
  int ks, splits, steps_per_split;
};
StreamPlan stream_plan(int64_t in_dim, int64_t out_dim, int64_t n_tok, size_t ws_bytes);
size_t stream_workspace_bytes(int64_t in_dim, int64_t out_dim, int64_t n_tok);
hipError_t launch_stream(const StreamPlan &p, void *out, int out_type, const uint8_t *w,
                         const uint8_t *ws, int64_t in_dim, int64_t out_dim, const uint8_t *x,
                         const uint8_t *xs, int64_t n_tok, void *workspace, hipStream_t s);

// mxfp4_gemm.hip: for many tokens.  in_dim >= 512 (a row's scales are read sixteen at a time).
struct GemmPlan {
  int tile, splits, stages_per_split;
};
GemmPlan gemm_plan(int64_t in_dim, int64_t out_dim, int64_t n_tok, size_t ws_bytes);
size_t gemm_workspace_bytes(int64_t in_dim, int64_t out_dim, int64_t n_tok);
hipError_t launch_gemm(const GemmPlan &p, void *out, int out_type, const uint8_t *w, const uint8_t *ws,
                       int64_t in_dim, int64_t out_dim, const uint8_t *x, const uint8_t *xs,
                       int64_t n_tok, void *workspace, hipStream_t s);
// out[i] = sum over s < splits, in order, of part[s * elems + i].
hipError_t launch_reduce(void *out, int out_type, const float *part, int64_t elems, int splits,
                         hipStream_t s);

// moe_topk.hip
struct RouteArgs;
hipError_t launch_topk(const RouteArgs &a, int64_t n_tok, int32_t *selected, float *weights,
                       hipStream_t s);

// mxfp4_moe.hip: the whole MoE layer; buffers already validated.
constexpr int kMaxLayerTokens = 64;
constexpr int kMaxLayerExperts = 512;
struct MoeLayer {
  void *out;
  int out_type;
  const void *x;
  int x_type;
  const RouteArgs *route;
  const uint8_t *gate, *gate_s, *up, *up_s, *down, *down_s;
  int64_t d_model, d_ff, n_tok;
  float clamp;
  int32_t *selected;  // optional
  float *weights;     // optional
};
size_t moe_layer_workspace_bytes(int64_t n_tok, int32_t n_used, int32_t n_expert, int64_t d_model,
                                 int64_t d_ff);
hipError_t launch_moe_layer(const MoeLayer &m, uint8_t *ws, hipStream_t s);

}  // namespace mx
