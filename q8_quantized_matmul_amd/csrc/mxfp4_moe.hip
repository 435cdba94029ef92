// mxfp4_moe.hip -- the whole MoE layer for a few tokens, in two kernels:
//   1. route, quantize x, gate and up of every (token, expert) pair, SwiGLU,
//      quantize mid;
//   2. down of every pair, weighted sum over a token's experts.
// At these sizes the layer is bound by reading each touched expert's matrices
// once (17 bytes per 32 weights), and at one token by latency, so routing is not
// a launch of its own: every workgroup of kernel 1 routes all tokens for itself
// (a wave per token, moe_topk.h) and finds the touched experts from per-expert
// token masks in LDS; workgroup 0 also leaves the tables for kernel 2.
//
// A touched expert's tokens are the columns of 16x16x128 matrix instructions,
// 16 of them a tile, so its weights are read once however many tokens share
// it (mxfp4_mfma.h has the operand layout).
#include <algorithm>

#include "moe_topk.h"
#include "mxfp4_mfma.h"

namespace mx {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// Tables that kernel 1 leaves for kernel 2, and the quantized mid, in the
// workspace.  Pairs are numbered expert-major, tokens ascending.
struct Tables {
  int32_t *head;     // [0]: touched experts
  int32_t *expert;   // [touched]
  int32_t *first;    // [touched + 1]: first pair of each
  int32_t *tok;      // [pairs]
  float *weight;     // [pairs]
  uint8_t *mid;      // [pairs][d_ff/2]
  uint8_t *mid_s;    // [pairs][d_ff/32]
};

struct Args {
  RouteArgs route;
  Tables tab;
  const void *x;
  int32_t x_type;
  const uint8_t *gate, *gate_s, *up, *up_s, *down, *down_s;
  int32_t d_model, d_ff, n_tok;
  float clamp;
  int32_t *selected;  // optional outputs
  float *weights;
  void *out;
};

__device__ __forceinline__ int bit_rank(uint64_t mask, int t) {
  return __popcll(mask & ((1ull << t) - 1));
}

// A lane's block of 32 unquantized values, quantized in the lane.
template <int TYPE>
__device__ __forceinline__ void quantize_block(const void *x, int64_t elem, u32x4 &codes, uint32_t &byte) {
  Eight<TYPE> v[4];
  const uint8_t *p = static_cast<const uint8_t *>(x) + elem * (TYPE == kF32 ? 4 : 2);
  constexpr int N = (TYPE == kF32 ? 8 : 4) / 4;
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const u32x4 t = ((global_u32x4 *)p)[q * N + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[q].d[4 * i + j] = t[j];
    }
    m = max(m, amax_bits<TYPE>(v[q]));
  }
  byte = scale_byte(m);
#pragma unroll
  for (int q = 0; q < 4; ++q) codes[q] = encode<TYPE>(v[q], byte);
}

// Blocks b0..b0+3 of token row `row` of x, quantized; zero past the row and where !valid.
__device__ __forceinline__ void load_x(const Args &a, int row, bool valid, int b0, int nb, Blocks4 &r) {
  r.s = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.c[i] = u32x4{0, 0, 0, 0};
    if (valid && b0 + i < nb) {
      const int64_t elem = (int64_t)row * a.d_model + (b0 + i) * kBlock;
      uint32_t byte;
      if (a.x_type == kF32) quantize_block<kF32>(a.x, elem, r.c[i], byte);
      else if (a.x_type == kBF16) quantize_block<kBF16>(a.x, elem, r.c[i], byte);
      else quantize_block<kF16>(a.x, elem, r.c[i], byte);
      r.s |= byte << (8 * i);
    }
  }
}

__device__ __forceinline__ float swiglu(float g, float u, float clamp) {
  if (clamp > 0.0f) {
    // Comparisons, not fmin/fmax, so that a NaN stays one.
    g = g > clamp ? clamp : g;
    u = u > clamp ? clamp : (u < -clamp ? -clamp : u);
  }
  return g / (1.0f + expf(-g)) * u;
}

// NT: tiles of 16 tokens (n_tok <= 16 NT).  EPL: experts per lane of the router.
template <int NT, int EPL, bool WHOLE>
__global__ __launch_bounds__(kThreads) void up_kernel(const Args a) {
  __shared__ uint32_t mask_lo[64 * EPL], mask_hi[64 * EPL];
  __shared__ int32_t touched[64 * EPL], first[64 * EPL + 1];
  __shared__ int32_t n_touched;
  __shared__ f32x4 part[kWaves][4][64];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n_expert = a.route.n_expert, n_used = a.route.n_used;
  for (int e = tid; e < 64 * EPL; e += kThreads) mask_lo[e] = mask_hi[e] = 0;
  __syncthreads();
  for (int t = wave; t < a.n_tok; t += kWaves) {
    int id;
    float w;
    route_token<EPL>(a.route, t, lane, id, w);
    if (lane < n_used) {
      if (id >= 0) atomicOr(t < 32 ? &mask_lo[id] : &mask_hi[id], 1u << (t & 31));
      if (blockIdx.x == 0) {
        a.selected[t * n_used + lane] = id;
        a.weights[t * n_used + lane] = w;
      }
    }
  }
  __syncthreads();
  auto mask_of = [&](int e) { return ((uint64_t)mask_hi[e] << 32) | mask_lo[e]; };
  if (wave == 0) {  // compact the touched experts, in order
    int count = 0, pairs = 0;
    for (int e0 = 0; e0 < n_expert; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < n_expert ? __popcll(mask_of(e)) : 0;
      const uint64_t live = __ballot(c > 0);
      int before = c;  // inclusive prefix sum of the pair counts
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int u = __shfl_up(before, off, 64);
        if (lane >= off) before += u;
      }
      const int total = __shfl(before, 63, 64);
      if (c > 0) {
        const int i = count + __popcll(live & ((1ull << lane) - 1));
        touched[i] = e;
        first[i] = pairs + before - c;
      }
      count += __popcll(live);
      pairs += total;
    }
    if (lane == 0) {
      n_touched = count;
      first[count] = pairs;
    }
  }
  __syncthreads();
  const int count = n_touched;
  if (blockIdx.x == 0) {
    if (tid == 0) a.tab.head[0] = count;
    for (int i = tid; i < count; i += kThreads) a.tab.expert[i] = touched[i];
    for (int i = tid; i <= count; i += kThreads) a.tab.first[i] = first[i];
    // Pair (t, slot): the rank of t among its expert's tokens.
    for (int i = wave; i < count; i += kWaves) {
      const uint64_t m = mask_of(touched[i]);
      if ((m >> lane) & 1) {
        const int p = first[i] + bit_rank(m, lane);
        a.tab.tok[p] = lane;
        for (int j = 0; j < n_used; ++j)
          if (a.selected[lane * n_used + j] == touched[i]) a.tab.weight[p] = a.weights[lane * n_used + j];
      }
    }
  }

  // Work items: 32 rows of d_ff (one block of mid) of one touched expert, gate
  // and up together, the eight waves splitting d_model.
  const int nb = a.d_model / kBlock, nbf = a.d_ff / kBlock;
  const int steps = (nb + kStepBlocks - 1) / kStepBlocks;
  const int row = lane & 15, g = lane >> 4;
  const int items = count * nbf;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = it / nbf, blk = it - i * nbf;
    const int e = touched[i];
    const uint64_t m = mask_of(e);
    const int n = first[i + 1] - first[i];
    // Token of column c of tile j: the (16 j + c)-th set bit of the mask.
    int column = 0;
    {
      const bool on = (m >> lane) & 1;
      column = __builtin_amdgcn_ds_permute(on ? 4 * bit_rank(m, lane) : 4 * 63, on ? lane : 0);
    }
    const int64_t r0 = (int64_t)e * a.d_ff + blk * 32;
    const uint8_t *wc[4], *wsc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t r = r0 + 16 * (q & 1) + row;
      wc[q] = (q < 2 ? a.gate : a.up) + r * (nb * 16);
      wsc[q] = (q < 2 ? a.gate_s : a.up_s) + r * nb;
    }
    f32x4 acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[j][q] = f32x4{0, 0, 0, 0};
    for (int s = wave; s < steps; s += kWaves) {
      const int b0 = s * kStepBlocks + 4 * g;
      Blocks4 A[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) load_blocks<WHOLE>(wc[q], wsc[q], b0, nb, A[q]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (16 * j < n) {
          Blocks4 B;
          const int tok = __shfl(column, 16 * j + row, 64);
          load_x(a, tok, 16 * j + row < n, b0, nb, B);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[j][q] = mfma_blocks4(A[q], B, acc[j][q]);
        }
      }
    }
    // Join the waves, one token tile at a time; wave 0 then holds 32 rows of mid
    // (lane: rows 4g..4g+3 of both halves) of 16 tokens: one block each.
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (16 * j < n) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; ++q) part[wave][q][lane] = acc[j][q];
        __syncthreads();
        if (wave == 0) {
          f32x4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[q] = part[0][q][lane];
            for (int w = 1; w < kWaves; ++w) v[q] += part[w][q][lane];
          }
          Eight<kF32> mid;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              mid.d[4 * h + r] = __builtin_bit_cast(uint32_t, swiglu(v[h][r], v[2 + h][r], a.clamp));
          uint32_t am = amax_bits<kF32>(mid);
          am = max(am, (uint32_t)__shfl_xor((int)am, 16, 64));
          am = max(am, (uint32_t)__shfl_xor((int)am, 32, 64));
          const uint32_t byte = scale_byte(am);
          const uint32_t c = encode<kF32>(mid, byte);
          if (16 * j + row < n) {
            const int64_t p = first[i] + 16 * j + row;
            uint16_t *o = reinterpret_cast<uint16_t *>(a.tab.mid + p * (a.d_ff / 2) + blk * 16);
            o[g] = (uint16_t)c;
            o[4 + g] = (uint16_t)(c >> 16);
            if (g == 0) a.tab.mid_s[p * nbf + blk] = (uint8_t)byte;
          }
        }
      }
    }
  }
}

// A workgroup owns 16 rows of d_model for all tokens; its waves share out the
// touched experts and add weight * down into sums of their own in LDS (lanes
// hold different tokens, so no two add to one place), joined in wave order.
template <int NT, bool WHOLE, int TYPE>
__global__ __launch_bounds__(kThreads) void down_kernel(const Args a) {
  __shared__ f32x4 sum[kWaves][16 * NT][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, g = lane >> 4;
  for (int i = tid; i < kWaves * 16 * NT * 4; i += kThreads) (&sum[0][0][0])[i] = f32x4{0, 0, 0, 0};
  __syncthreads();
  const int count = a.tab.head[0];
  const int nb = a.d_ff / kBlock;
  const int steps = (nb + kStepBlocks - 1) / kStepBlocks;
  const int64_t o0 = (int64_t)blockIdx.x * 16;
  for (int i = wave; i < count; i += kWaves) {
    const int e = a.tab.expert[i], p0 = a.tab.first[i], n = a.tab.first[i + 1] - p0;
    const int64_t r = (int64_t)e * a.d_model + o0 + row;
    const uint8_t *wc = a.down + r * (nb * 16), *wsc = a.down_s + r * nb;
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0, 0, 0, 0};
    for (int s = 0; s < steps; ++s) {
      const int b0 = s * kStepBlocks + 4 * g;
      Blocks4 A;
      load_blocks<WHOLE>(wc, wsc, b0, nb, A);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (16 * j < n) {
          Blocks4 B;
          const int64_t p = p0 + min(16 * j + row, n - 1);
          load_blocks<WHOLE>(a.tab.mid + p * (nb * 16), a.tab.mid_s + p * nb, b0, nb, B);
          acc[j] = mfma_blocks4(A, B, acc[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (16 * j + row < n) {
        const int p = p0 + 16 * j + row;
        f32x4 &d = sum[wave][a.tab.tok[p]][g];
        d += a.tab.weight[p] * acc[j];
      }
    }
  }
  __syncthreads();
  const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;  // d_model is a multiple of 32
  for (int i = tid; i < a.n_tok * 4; i += kThreads) {
    const int t = i >> 2, q = i & 3;
    f32x4 v = sum[0][t][q];
    for (int w = 1; w < kWaves; ++w) v += sum[w][t][q];
    store4<TYPE>(a.out, (int64_t)t * a.d_model + o0 + 4 * q, v, 4, wide);
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Byte offsets in the workspace.
struct Layout {
  size_t head, expert, first, tok, weight, sel, selw, mid, mid_s, total;
};
Layout layout(int64_t n_tok, int32_t n_used, int32_t n_expert, int64_t d_ff) {
  const size_t pairs = (size_t)n_tok * n_used, touched = std::min<size_t>(pairs, n_expert);
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  l.head = take(4);
  l.expert = take(4 * touched);
  l.first = take(4 * (touched + 1));
  l.tok = take(4 * pairs);
  l.weight = take(4 * pairs);
  l.sel = take(4 * pairs);
  l.selw = take(4 * pairs);
  l.mid = take(pairs * (size_t)(d_ff / 2));
  l.mid_s = take(pairs * (size_t)(d_ff / kBlock));
  l.total = at;
  return l;
}

}  // namespace

size_t moe_layer_workspace_bytes(int64_t n_tok, int32_t n_used, int32_t n_expert, int64_t d_ff) {
  return layout(n_tok, n_used, n_expert, d_ff).total;
}

hipError_t launch_moe_layer(const MoeLayer &m, uint8_t *ws, hipStream_t s) {
  const Layout l = layout(m.n_tok, m.route->n_used, m.route->n_expert, m.d_ff);
  Args a{};
  a.route = *m.route;
  a.tab = Tables{reinterpret_cast<int32_t *>(ws + l.head),  reinterpret_cast<int32_t *>(ws + l.expert),
                 reinterpret_cast<int32_t *>(ws + l.first), reinterpret_cast<int32_t *>(ws + l.tok),
                 reinterpret_cast<float *>(ws + l.weight),  ws + l.mid, ws + l.mid_s};
  a.x = m.x;
  a.x_type = m.x_type;
  a.gate = m.gate;
  a.gate_s = m.gate_s;
  a.up = m.up;
  a.up_s = m.up_s;
  a.down = m.down;
  a.down_s = m.down_s;
  a.d_model = (int32_t)m.d_model;
  a.d_ff = (int32_t)m.d_ff;
  a.n_tok = (int32_t)m.n_tok;
  a.clamp = m.clamp;
  a.selected = m.selected ? m.selected : reinterpret_cast<int32_t *>(ws + l.sel);
  a.weights = m.weights ? m.weights : reinterpret_cast<float *>(ws + l.selw);
  a.out = m.out;

  auto a4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; };
  const bool whole1 = m.d_model % 128 == 0 && a4(m.gate_s) && a4(m.up_s);
  const bool whole2 = m.d_ff % 128 == 0 && a4(m.down_s);
  const int64_t touched = std::min<int64_t>(m.n_tok * m.route->n_used, m.route->n_expert);
  const int64_t items = touched * (m.d_ff / kBlock);
  const dim3 grid1((uint32_t)std::min<int64_t>(items, 512)), grid2((uint32_t)(m.d_model / 16));
  const int nt = m.n_tok <= 16 ? 1 : m.n_tok <= 32 ? 2 : 4;
  auto with_nt = [&](auto f) {
    if (nt == 1) f(std::integral_constant<int, 1>{});
    else if (nt == 2) f(std::integral_constant<int, 2>{});
    else f(std::integral_constant<int, 4>{});
  };
  auto with_bool = [&](bool b, auto f) {
    if (b) f(std::true_type{});
    else f(std::false_type{});
  };
  with_nt([&](auto nt_c) {
    with_bool(whole1, [&](auto whole_c) {
      constexpr int NT = decltype(nt_c)::value;
      constexpr bool W = decltype(whole_c)::value;
      if (m.route->n_expert <= 256) hipLaunchKernelGGL((up_kernel<NT, 4, W>), grid1, dim3(kThreads), 0, s, a);
      else hipLaunchKernelGGL((up_kernel<NT, 8, W>), grid1, dim3(kThreads), 0, s, a);
    });
  });
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  with_nt([&](auto nt_c) {
    with_bool(whole2, [&](auto whole_c) {
      constexpr int NT = decltype(nt_c)::value;
      constexpr bool W = decltype(whole_c)::value;
      if (m.out_type == kF32) hipLaunchKernelGGL((down_kernel<NT, W, kF32>), grid2, dim3(kThreads), 0, s, a);
      else if (m.out_type == kBF16) hipLaunchKernelGGL((down_kernel<NT, W, kBF16>), grid2, dim3(kThreads), 0, s, a);
      else hipLaunchKernelGGL((down_kernel<NT, W, kF16>), grid2, dim3(kThreads), 0, s, a);
    });
  });
  return hipGetLastError();
}

}  // namespace mx
