// moe_topk.hip -- the MoE router: a wave per token (moe_topk.h).
#include "moe_topk.h"

namespace mx {
namespace {

constexpr int kWaves = 4;

template <int EPL>
__global__ __launch_bounds__(64 * kWaves) void topk_kernel(const RouteArgs a, int64_t n_tok,
                                                           int32_t *__restrict__ selected,
                                                           float *__restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= n_tok) return;
  int id;
  float w;
  route_token<EPL>(a, t, lane, id, w);
  if (lane < a.n_used) {
    selected[t * a.n_used + lane] = id;
    weights[t * a.n_used + lane] = w;
  }
}

}  // namespace

hipError_t launch_topk(const RouteArgs &a, int64_t n_tok, int32_t *selected, float *weights,
                       hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((n_tok + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0,
                       s, a, n_tok, selected, weights);
  };
  if (a.n_expert <= 64) go(topk_kernel<1>);
  else if (a.n_expert <= 128) go(topk_kernel<2>);
  else if (a.n_expert <= 256) go(topk_kernel<4>);
  else if (a.n_expert <= 512) go(topk_kernel<8>);
  else go(topk_kernel<16>);
  return hipGetLastError();
}

}  // namespace mx
