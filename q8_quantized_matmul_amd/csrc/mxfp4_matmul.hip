// mxfp4_matmul.hip -- the product of MXFP4 weights and MXFP4 rows,
//   out[t][o] = sum_b 2^(sw[o][b] + sx[t][b] - 254) sum_i w[o][b][i] x[t][b][i].
//
// Streaming kernel.  With few tokens the product is bound by reading the
// weights, 17 bytes per 32 values.  A wave takes 16 weight rows as the A operand
// straight from memory to registers, steps of 512 values apart, and 16 tokens as
// B (16x16x128 instructions: 16 of their 16 columns idle at one token, but the
// matrix core still takes weights ten times faster than memory gives them).
// ks waves of a workgroup split a row's steps and are joined in LDS in wave
// order, so that few rows still give the memory enough waves.  A compute unit takes
// about 25 bytes a nanosecond from memory however many waves wait for them, so long
// rows with too few of them for every unit are split between workgroups too (32768 ->
// 1024 at one token 14.2 us with 64 workgroups, 8.7 with 256 and the join).  1024 ->
// 32768 at one token: 5.5 us, 18 MB, of which 2 are the launch.
#include <algorithm>
#include <type_traits>

#include "mxfp4_mfma.h"

namespace mx {
namespace {

constexpr int kWaves = 8;

struct MatmulArgs {
  void *out;
  const uint8_t *w, *ws, *x, *xs;
  int32_t nb;        // blocks of a row
  int64_t n, t;      // weight rows, tokens
  int32_t ks;        // waves along K: a power of two <= kWaves
  int32_t steps_per_split;
  int32_t row_groups, tok_groups;  // workgroups: row groups, token groups, splits
  bool wide;         // rows of out are aligned for stores of four values
};

// NT: tiles of 16 tokens a workgroup takes.  AHEAD: steps of a wave whose loads are
// issued together, for waves of several steps.
template <int NT, int AHEAD, bool SHORT, int TYPE>
__global__ __launch_bounds__(64 * kWaves, 2) void stream_kernel(const MatmulArgs a) {
  __shared__ f32x4 part[kWaves * NT * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kq = wave & (a.ks - 1), rt = wave / a.ks;
  const int tiles = kWaves / a.ks;  // row tiles of the workgroup
  const int row = lane & 15, g = lane >> 4;
  const int rg = blockIdx.x % a.row_groups, rest = blockIdx.x / a.row_groups;
  const int tg = rest % a.tok_groups, split = rest / a.tok_groups;
  const int64_t o0 = ((int64_t)rg * tiles + rt) * 16;
  const int64_t t0 = (int64_t)tg * (16 * NT);
  // Rows past the ends are read as the last row; what they give is not stored.
  const uint8_t *wc = a.w + o0 * (a.nb * 16), *wsc = a.ws + o0 * a.nb;
  const uint8_t *xc = a.x + t0 * (a.nb * 16), *xsc = a.xs + t0 * a.nb;
  const uint32_t wr = (uint32_t)min<int64_t>(row, a.n - 1 - o0);
  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4{0, 0, 0, 0};

  const int steps_all = (a.nb + kStepBlocks - 1) / kStepBlocks;
  const int first = split * a.steps_per_split, steps = min(first + a.steps_per_split, steps_all);
  if (o0 < a.n) {
    for (int s = first + kq; s < steps; s += AHEAD * a.ks) {
      Blocks4 A[AHEAD], B[AHEAD][NT];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int b0 = (s + u * a.ks) * kStepBlocks;
        if (u == 0 || s + u * a.ks < steps) {
          load_blocks<SHORT>(wc, wsc, Offsets4<SHORT>(wr, b0, a.nb), a.nb, A[u]);
#pragma unroll
          for (int j = 0; j < NT; ++j)
            load_blocks<SHORT>(xc, xsc, Offsets4<SHORT>((uint32_t)min<int64_t>(16 * j + row, a.t - 1 - t0), b0, a.nb), a.nb, B[u][j]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // all of them are on their way before any is used
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int b0 = (s + u * a.ks) * kStepBlocks;
        if (u == 0 || s + u * a.ks < steps) {
          const Offsets4<SHORT> end(0, b0, a.nb);
          finish_blocks(end, A[u]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            finish_blocks(end, B[u][j]);
            acc[j] = mfma_blocks4(A[u], B[u][j], acc[j]);
          }
        }
      }
    }
  }
  if (a.ks > 1) {
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(wave * NT + j) * 64 + lane] = acc[j];
    __syncthreads();
  }
  // Wave kq of a row tile's ks waves joins and stores token tiles kq, kq + ks, ...
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if ((j & (a.ks - 1)) != kq) continue;
    f32x4 v = acc[j];
    if (a.ks > 1) {
      v = part[((wave - kq) * NT + j) * 64 + lane];
      for (int q = 1; q < a.ks; ++q) v += part[((wave - kq + q) * NT + j) * 64 + lane];
    }
    const int64_t t = t0 + 16 * j + row, o = o0 + 4 * g;
    if (t < a.t && o < a.n) store4<TYPE>(a.out, (split * a.t + t) * a.n + o, v, (int)min<int64_t>(4, a.n - o), a.wide);
  }
}

int64_t tiles_of(int64_t out_dim) { return (out_dim + 15) / 16; }
int tok_tiles(int64_t n_tok) { return n_tok <= 16 ? 1 : n_tok <= 32 ? 2 : 4; }

}  // namespace

StreamPlan stream_plan(int64_t in_dim, int64_t out_dim, int64_t n_tok, size_t ws_bytes) {
  const int64_t tiles = tiles_of(out_dim), steps = (in_dim / kBlock + kStepBlocks - 1) / kStepBlocks;
  StreamPlan p{1, 1, (int)steps};
  while (p.ks < kWaves && p.ks < steps && tiles * p.ks < 4096) p.ks *= 2;
  // Splits: a workgroup a compute unit, two steps a wave at least.
  const int64_t per_wg = kWaves / p.ks, nt = 16 * tok_tiles(n_tok);
  const int64_t groups = (tiles + per_wg - 1) / per_wg * ((n_tok + nt - 1) / nt);
  const int64_t fit = (int64_t)(ws_bytes / ((size_t)out_dim * n_tok * 4));
  p.splits = (int)std::max<int64_t>(1, std::min({256 / groups, steps / (2 * p.ks), fit}));
  p.steps_per_split = (int)((steps + p.splits - 1) / p.splits);
  p.splits = (int)((steps + p.steps_per_split - 1) / p.steps_per_split);
  return p;
}

size_t stream_workspace_bytes(int64_t in_dim, int64_t out_dim, int64_t n_tok) {
  const StreamPlan p = stream_plan(in_dim, out_dim, n_tok, SIZE_MAX);
  return p.splits > 1 ? (size_t)p.splits * out_dim * n_tok * 4 : 0;
}

hipError_t launch_stream(const StreamPlan &p, void *out, int out_type, const uint8_t *w, const uint8_t *ws,
                         int64_t in_dim, int64_t out_dim, const uint8_t *x, const uint8_t *xs,
                         int64_t n_tok, void *workspace, hipStream_t s) {
  const int nb = (int)(in_dim / kBlock);
  const bool split = p.splits > 1;
  const int type = split ? kF32 : out_type, size = type == kF32 ? 4 : 2;
  void *dst = split ? workspace : out;
  const int nt = tok_tiles(n_tok);
  const int64_t per_wg = kWaves / p.ks;
  MatmulArgs a{dst, w, ws, x, xs, nb, out_dim, n_tok, p.ks, p.steps_per_split,
               (int32_t)((tiles_of(out_dim) + per_wg - 1) / per_wg),
               (int32_t)((n_tok + 16 * nt - 1) / (16 * nt)), false};
  a.wide = out_dim % 4 == 0 && (reinterpret_cast<uintptr_t>(dst) & (4 * size - 1)) == 0;
  const dim3 grid((uint32_t)((int64_t)a.row_groups * a.tok_groups * p.splits));
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), 0, s, a); };
  const bool ahead = p.steps_per_split > p.ks;
  auto by_type = [&](auto nt_c, auto ahead_c, auto short_c) {
    constexpr int NT = decltype(nt_c)::value, A = decltype(ahead_c)::value;
    constexpr bool S = decltype(short_c)::value;
    if (type == kF32) go(stream_kernel<NT, A, S, kF32>);
    else if (type == kBF16) go(stream_kernel<NT, A, S, kBF16>);
    else go(stream_kernel<NT, A, S, kF16>);
  };
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 4> four{};
  auto by_nt = [&](auto ahead_c, auto short_c) {
    if (nt == 1) by_type(one, ahead_c, short_c);
    else if (nt == 2) by_type(two, ahead_c, short_c);
    else by_type(four, ahead_c, short_c);
  };
  if (nb < 4) by_nt(one, std::true_type{});
  else if (!ahead) by_nt(one, std::false_type{});
  else if (nt == 1) by_type(one, four, std::false_type{});
  else if (nt == 2) by_type(two, two, std::false_type{});
  else by_type(four, two, std::false_type{});
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !split) return err;
  return launch_reduce(out, out_type, static_cast<const float *>(workspace), out_dim * n_tok, p.splits, s);
}

}  // namespace mx
