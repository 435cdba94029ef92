// mxfp4_moe.hip -- the whole MoE layer for a few tokens:
//   up_kernel    route, quantize x, gate and up of every (token, expert) pair, SwiGLU,
//                quantize mid;
//   down_kernel  down of every pair, weighted sum over a token's experts.
// At these sizes the layer is bound by reading each touched expert's matrices
// once (17 bytes per 32 weights), and at a few tokens by latency, so with up to
// eight, a wave each, routing and quantizing are not launches of their own: every
// workgroup of the first kernel does both for itself (moe_topk.h; x in LDS).  With
// more tokens a small kernel in front does it once.  2048 x 768, 6 of 64 experts,
// fused and with the front kernel: 31.2 and 32.2 us at 5 tokens, 39.3 and 38.0 at 8
// (whose launch costs the caller 3 us more), 45.5 and 40.0 at 11.
//
// Measured, 4096 x 2048, 8 of 256 experts: one token 27.1 us (107 MB, 3.9 TB/s:
// launches, routing and the tables' chain are 8 us of it), 64 tokens 521 us (3.0 GB
// of 222 experts, 5.7 TB/s of the 5.9 that reading alone reaches).
//
// A touched expert's tokens are the columns of 16x16x128 matrix instructions
// (mxfp4_mfma.h), 16 of them a tile, so its weights are read once for up to 16
// tokens.  An expert with more loads them again for the next 16, from memory: 64
// workgroups of an XCD have 139 KB each under way at 4096 values a row, more than its
// 4 MB of second cache keep.  64 tokens that all use the same 8 experts of 4096 x 2048
// (four tiles each) move 277 of 71 MB in up_kernel and 104 of 36 MB in down_kernel and
// take 96 us, where 107 MB read once are 18.
//
// down_kernel has a workgroup for every 16 of d_model's rows, and each takes every
// touched expert: right at 4096, where that is one a compute unit (5.7 TB/s above), and
// far from the floor where it is fewer.  64 tokens, 64 experts with d_ff 2048, us and
// the time to read their matrices once: d_model 1024 100 and 37, 2048 128 and 73, 5120
// 281 and 183, 7168 337 and 256; 256 experts of d_model 256 245 and 32.
#include <algorithm>
#include <type_traits>

#include "moe_topk.h"
#include "mxfp4_mfma.h"

namespace mx {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kFusedTok = kWaves;         // up to here up_kernel routes and quantizes
constexpr size_t kFusedBytes = 36 * 1024;  // ... if x fits beside the rest of two workgroups' LDS
constexpr int64_t kUpWorkgroups = 512;     // two a compute unit

// A touched expert and its pairs.  Pairs are numbered expert-major, tokens ascending.
struct Touched {
  int32_t expert, first, n, unused;
};
// What one kernel leaves for the next in the workspace.
struct Tables {
  int32_t *count;     // touched experts
  Touched *touched;   // [count], readable up to kWaves
  int32_t *tok;       // [pairs]
  float *weight;      // [pairs]
  uint8_t *x, *x_s;   // [n_tok][d_model] quantized, from front_kernel
  uint8_t *mid, *mid_s;  // [pairs][d_ff] quantized
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

// x rows quantized by a workgroup of `threads`: rows t0, t0 + step, ... below n_tok
// to codes + t * pitch and scales + t * scale_pitch.  Four lanes a block.
template <int TYPE>
__device__ __forceinline__ void quantize_rows(const Args &a, int t0, int step, uint8_t *codes, int64_t pitch,
                                              uint8_t *scales, int64_t scale_pitch, int tid, int threads) {
  const int per_row = a.d_model / 8;
  for (int t = t0; t < a.n_tok; t += step) {
    for (int g = tid; g < per_row; g += threads) {  // per_row is a multiple of 4: quads stay whole
      Eight<TYPE> v;
      constexpr int N = TYPE == kF32 ? 2 : 1;
      const uint8_t *p = static_cast<const uint8_t *>(a.x) + ((int64_t)t * a.d_model + g * 8) * (TYPE == kF32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const u32x4 q = ((global_u32x4 *)p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v.d[4 * i + j] = q[j];
      }
      const uint32_t byte = scale_byte(max_quad(amax_bits<TYPE>(v)));
      *reinterpret_cast<uint32_t *>(codes + t * pitch + g * 4) = encode<TYPE>(v, byte);
      if ((g & 3) == 0) scales[t * scale_pitch + g / 4] = (uint8_t)byte;
    }
  }
}
__device__ __forceinline__ void quantize_x(const Args &a, int t0, int step, uint8_t *codes, int64_t pitch,
                                           uint8_t *scales, int64_t scale_pitch, int tid, int threads) {
  if (a.x_type == kF32) quantize_rows<kF32>(a, t0, step, codes, pitch, scales, scale_pitch, tid, threads);
  else if (a.x_type == kBF16) quantize_rows<kBF16>(a, t0, step, codes, pitch, scales, scale_pitch, tid, threads);
  else quantize_rows<kF16>(a, t0, step, codes, pitch, scales, scale_pitch, tid, threads);
}

__device__ __forceinline__ float swiglu(float g, float u, float clamp) {
  if (clamp > 0.0f) {
    // Comparisons, not fmin/fmax, so that a NaN stays one.
    g = g > clamp ? clamp : g;
    u = u > clamp ? clamp : (u < -clamp ? -clamp : u);
  }
  return g / (1.0f + expf(-g)) * u;
}

// In front of up_kernel for more than kFusedTok tokens: a workgroup per token.
template <int EPL>
__global__ __launch_bounds__(256) void front_kernel(const Args a) {
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  if (tid < 64) {
    int id;
    float w;
    route_token<EPL>(a.route, t, lane, id, w);
    if (lane < a.route.n_used) {
      a.selected[t * a.route.n_used + lane] = id;
      a.weights[t * a.route.n_used + lane] = w;
    }
  }
  quantize_x(a, t, kMaxLayerTokens, a.tab.x, a.d_model / 2, a.tab.x_s, a.d_model / kBlock, tid, 256);
}

// Bytes between the quantized x rows in LDS: off the banks' period, 16-byte aligned.
__host__ __device__ __forceinline__ int x_pitch(int d_model) { return d_model / 2 + 16; }
__host__ __device__ __forceinline__ int x_scale_pitch(int d_model) { return (d_model / kBlock + 3) / 4 * 4 + 4; }

// The lane's blocks of a step of a quantized x row in LDS, as load_blocks.
__device__ __forceinline__ void load_x(const uint8_t *codes, const uint8_t *scales, int b0, int nb, Blocks4 &r) {
  const int g = (threadIdx.x >> 4) & 3, b = b0 + 4 * g;
  const uint32_t s = *reinterpret_cast<const uint32_t *>(scales + min(b, (nb + 3) / 4 * 4 - 4));
  const int past = min(max(b + 4 - nb, 0), 4);
  r.s = spread_scales(past == 4 ? 0u : s & (0xFFFFFFFFu >> (8 * past)));
#pragma unroll
  for (int i = 0; i < 4; ++i) r.c[i] = *reinterpret_cast<const u32x4 *>(codes + min(b0 + 4 * i + g, nb - 1) * 16);
}

// EPL: experts per lane of the router where this kernel routes, 0 where
// front_kernel has.  A workgroup routes, or reads the routing, and then takes items:
// 32 rows of d_ff (one block of mid) of one touched expert, gate and up together,
// its eight waves splitting d_model.  128 registers, so that two workgroups share
// a compute unit and one reads while the other joins its waves.
template <int EPL, bool SHORT>
__global__ __launch_bounds__(kThreads, SHORT ? 2 : 4) void up_kernel(const Args a) {
  __shared__ uint32_t mask_lo[kMaxLayerExperts], mask_hi[kMaxLayerExperts];
  __shared__ int32_t touched[kMaxLayerExperts], first_of[kMaxLayerExperts];
  __shared__ int32_t n_touched;
  __shared__ f32x4 part[kWaves][4][64];
  __shared__ int32_t slot_id[kFusedTok * kMaxUsed];
  __shared__ float slot_weight[kFusedTok * kMaxUsed];
  extern __shared__ __attribute__((aligned(16))) uint8_t x_lds[];  // [n_tok][x_pitch], then the scales

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_expert = a.route.n_expert, n_used = a.route.n_used;
  uint8_t *xs_lds = x_lds + a.n_tok * x_pitch(a.d_model);
  const bool single = EPL > 0 && a.n_tok == 1;  // its slots are the touched experts: no table to build
  if (!single) {
    for (int e = tid; e < n_expert; e += kThreads) mask_lo[e] = mask_hi[e] = 0;
    __syncthreads();
  }
  if constexpr (EPL > 0) {
    for (int t = wave; t < a.n_tok; t += kWaves) {
      int id;
      float w;
      route_token<EPL>(a.route, t, lane, id, w);
      if (lane < n_used) {
        if (single && id >= 0) {
          mask_lo[id] = 1;
          mask_hi[id] = 0;
          touched[lane] = id;
          first_of[id] = lane;
        } else if (id >= 0) {
          atomicOr(&mask_lo[id], 1u << t);
        }
        slot_id[t * n_used + lane] = id;
        slot_weight[t * n_used + lane] = w;
      }
      if (single) {
        const uint64_t live = __ballot(lane < n_used && id >= 0);
        if (lane == 0) n_touched = __popcll(live);
      }
    }
    // The waves that do not route, if half of them are free; else all.
    const int busy = a.n_tok <= kWaves / 2 ? a.n_tok : 0;
    if (wave >= busy) {
      quantize_x(a, 0, 1, x_lds, x_pitch(a.d_model), xs_lds, x_scale_pitch(a.d_model), tid - 64 * busy,
                 kThreads - 64 * busy);
    }
  } else {
    for (int p = tid; p < a.n_tok * n_used; p += kThreads) {
      const int id = a.selected[p], t = p / n_used;
      if (id >= 0) atomicOr(t < 32 ? &mask_lo[id] : &mask_hi[id], 1u << (t & 31));
    }
  }
  __syncthreads();
  auto mask_of = [&](int e) { return ((uint64_t)mask_hi[e] << 32) | mask_lo[e]; };
  if (!single && wave == 0) {  // compact the touched experts, in order
    int count = 0, pairs = 0;
    for (int e0 = 0; e0 < n_expert; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < n_expert ? __popcll(mask_of(e)) : 0;
      const uint64_t live = __ballot(c > 0);
      if (live == 0) continue;
      int before = c;  // inclusive prefix sum of the pair counts
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int u = __shfl_up(before, off, 64);
        if (lane >= off) before += u;
      }
      const int total = __shfl(before, 63, 64);
      if (c > 0) {
        touched[count + __popcll(live & ((1ull << lane) - 1))] = e;
        first_of[e] = pairs + before - c;
      }
      count += __popcll(live);
      pairs += total;
    }
    if (lane == 0) n_touched = count;
  }
  if (!single) __syncthreads();
  const int count = __builtin_amdgcn_readfirstlane(n_touched);

  const int nb = a.d_model / kBlock, nbf = a.d_ff / kBlock;
  const int steps = (nb + kStepBlocks - 1) / kStepBlocks;
  const int row = lane & 15, g = lane >> 4;
  const int items = count * nbf;
  int turn = 0;  // the wave that joins, in turn
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = it / nbf, blk = it - i * nbf;
    const int e = __builtin_amdgcn_readfirstlane(touched[i]);
    const uint64_t m = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)mask_hi[e]) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)mask_lo[e]);
    const int n = __popcll(m);
    // Token of column c of tile j: the (16 j + c)-th set bit of the mask.
    const bool on = (m >> lane) & 1;
    const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
    const int column = __builtin_amdgcn_ds_permute(on ? 4 * rank : 4 * 63, on ? lane : 0);
    const int64_t r0 = (int64_t)e * a.d_ff + blk * 32;
    for (int j = 0; 16 * j < n; ++j) {
      const int of = __builtin_amdgcn_ds_bpermute(4 * (16 * j + row), column);
      const int tok = 16 * j + row < n ? of : 0;  // idle columns: any row, not stored
      f32x4 acc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = f32x4{0, 0, 0, 0};
      for (int s = wave; s < steps; s += kWaves) {
        const int b0 = s * kStepBlocks;
        Blocks4 A[4], B;
        const Offsets4<SHORT> off((uint32_t)row, b0, nb);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t r = r0 + 16 * (q & 1);
          load_blocks<SHORT>((q < 2 ? a.gate : a.up) + r * (nb * 16), (q < 2 ? a.gate_s : a.up_s) + r * nb, off, nb, A[q]);
        }
        if constexpr (EPL == 0) load_blocks<SHORT>(a.tab.x, a.tab.x_s, Offsets4<SHORT>((uint32_t)tok, b0, nb), nb, B);
        __builtin_amdgcn_sched_barrier(0);  // all of them are on their way before any is used
        if constexpr (EPL > 0) load_x(x_lds + tok * x_pitch(a.d_model), xs_lds + tok * x_scale_pitch(a.d_model), b0, nb, B);
        else finish_blocks(off, B);
#pragma unroll
        for (int q = 0; q < 4; ++q) finish_blocks(off, A[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = mfma_blocks4(A[q], B, acc[q]);
      }
      __syncthreads();  // the last tile has been joined
#pragma unroll
      for (int q = 0; q < 4; ++q) part[wave][q][lane] = acc[q];
      __syncthreads();
      // One wave joins them, the others go on to read the next weights.  It then holds
      // 32 rows of mid (a lane: rows 4g..4g+3 of both halves) of 16 tokens: a block each.
      if (wave == turn) {
        f32x4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = part[0][q][lane];
#pragma unroll
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
          // 32 bits: at most 64 * 32 pairs of 2^15 blocks.
          const uint32_t at = (uint32_t)(first_of[e] + 16 * j + row) * (uint32_t)nbf + (uint32_t)blk;
          *reinterpret_cast<uint16_t *>(a.tab.mid + (at * 16 + 2 * g)) = (uint16_t)c;
          *reinterpret_cast<uint16_t *>(a.tab.mid + (at * 16 + 2 * g + 8)) = (uint16_t)(c >> 16);
          if (g == 0) a.tab.mid_s[at] = (uint8_t)byte;
        }
      }
      turn = (turn + 1) % kWaves;
    }
  }

  // The last workgroup (of the fewest items) leaves the routing and the tables.
  if (blockIdx.x == gridDim.x - 1) {
    if (tid == 0) *a.tab.count = count;
    for (int i = tid; i < count; i += kThreads) {
      const int e = touched[i];
      a.tab.touched[i] = Touched{e, first_of[e], (int32_t)__popcll(mask_of(e)), 0};
    }
    for (int p = tid; p < a.n_tok * n_used; p += kThreads) {
      const int t = p / n_used;
      const int id = EPL > 0 ? slot_id[p] : a.selected[p];
      const float w = EPL > 0 ? slot_weight[p] : a.weights[p];
      if constexpr (EPL > 0) {
        a.selected[p] = id;
        a.weights[p] = w;
      }
      if (id >= 0) {
        const int at = first_of[id] + bit_rank(mask_of(id), t);
        a.tab.tok[at] = t;
        a.tab.weight[at] = w;
      }
    }
  }
}

// A workgroup owns 16 rows of d_model for all tokens; its waves share out the
// touched experts and add weight * down into sums of their own in LDS (lanes
// hold different tokens, so no two add to one place), joined in wave order.
constexpr int kAhead = 4;  // steps whose loads are issued together: 17 KB a wave

template <bool SHORT, int TYPE>
__global__ __launch_bounds__(kThreads, 2) void down_kernel(const Args a) {
  extern __shared__ f32x4 sum[];  // [kWaves][n_tok][4]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15, g = lane >> 4;
  const int count = *a.tab.count;
  Touched next = a.tab.touched[wave];  // nothing, past the count
  for (int i = tid; i < kWaves * a.n_tok * 4; i += kThreads) sum[i] = f32x4{0, 0, 0, 0};
  const int nb = a.d_ff / kBlock;
  const int steps = (nb + kStepBlocks - 1) / kStepBlocks;
  const int64_t o0 = (int64_t)blockIdx.x * 16;
  __syncthreads();
  for (int i = wave; i < count; i += kWaves) {
    const Touched at = next;
    next = a.tab.touched[min(i + kWaves, count - 1)];
    const int64_t r = (int64_t)at.expert * a.d_model + o0;
    const uint8_t *wc = a.down + r * (nb * 16), *wsc = a.down_s + r * nb;
    for (int j = 0; 16 * j < at.n; ++j) {
      const int p = at.first + min(16 * j + row, at.n - 1);
      const int t = a.tab.tok[p];
      const float weight = a.tab.weight[p];
      f32x4 acc = {0, 0, 0, 0};
      for (int s = 0; s < steps; s += kAhead) {
        Blocks4 A[kAhead], B[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (s + u < steps) {
            const int b0 = (s + u) * kStepBlocks;
            load_blocks<SHORT>(wc, wsc, Offsets4<SHORT>((uint32_t)row, b0, nb), nb, A[u]);
            load_blocks<SHORT>(a.tab.mid, a.tab.mid_s, Offsets4<SHORT>((uint32_t)p, b0, nb), nb, B[u]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // all of them are on their way before any is used
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (s + u < steps) {
            const Offsets4<SHORT> off(0, (s + u) * kStepBlocks, nb);
            finish_blocks(off, A[u]);
            finish_blocks(off, B[u]);
            acc = mfma_blocks4(A[u], B[u], acc);
          }
        }
      }
      if (16 * j + row < at.n) {
        f32x4 &d = sum[(wave * a.n_tok + t) * 4 + g];
        d += weight * acc;
      }
    }
  }
  __syncthreads();
  const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;  // d_model is a multiple of 32
  for (int i = tid; i < a.n_tok * 4; i += kThreads) {
    f32x4 v = sum[i];
    for (int w = 1; w < kWaves; ++w) v += sum[w * a.n_tok * 4 + i];
    store4<TYPE>(a.out, (int64_t)(i >> 2) * a.d_model + o0 + 4 * (i & 3), v, 4, wide);
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Byte offsets in the workspace.
struct Layout {
  size_t count, touched, tok, weight, sel, selw, x, x_s, mid, mid_s, total;
};
Layout layout(int64_t n_tok, int32_t n_used, int32_t n_expert, int64_t d_model, int64_t d_ff) {
  const size_t pairs = (size_t)n_tok * n_used, touched = std::min<size_t>(pairs, n_expert);
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  l.count = take(4);
  l.touched = take(sizeof(Touched) * std::max<size_t>(touched, kWaves));
  l.tok = take(4 * pairs);
  l.weight = take(4 * pairs);
  l.sel = take(4 * pairs);
  l.selw = take(4 * pairs);
  l.x = take((size_t)n_tok * (d_model / 2));
  l.x_s = take((size_t)n_tok * (d_model / kBlock));
  l.mid = take(pairs * (size_t)(d_ff / 2));
  l.mid_s = take(pairs * (size_t)(d_ff / kBlock));
  l.total = at;
  return l;
}

}  // namespace

size_t moe_layer_workspace_bytes(int64_t n_tok, int32_t n_used, int32_t n_expert, int64_t d_model,
                                 int64_t d_ff) {
  return layout(n_tok, n_used, n_expert, d_model, d_ff).total;
}

hipError_t launch_moe_layer(const MoeLayer &m, uint8_t *ws, hipStream_t s) {
  const Layout l = layout(m.n_tok, m.route->n_used, m.route->n_expert, m.d_model, m.d_ff);
  Args a{};
  a.route = *m.route;
  a.tab.count = reinterpret_cast<int32_t *>(ws + l.count);
  a.tab.touched = reinterpret_cast<Touched *>(ws + l.touched);
  a.tab.tok = reinterpret_cast<int32_t *>(ws + l.tok);
  a.tab.weight = reinterpret_cast<float *>(ws + l.weight);
  a.tab.x = ws + l.x;
  a.tab.x_s = ws + l.x_s;
  a.tab.mid = ws + l.mid;
  a.tab.mid_s = ws + l.mid_s;
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

  const size_t x_bytes = (size_t)m.n_tok * (x_pitch(a.d_model) + x_scale_pitch(a.d_model));
  const bool few = m.route->n_expert <= 256;  // four experts a lane of the router
  const bool fused = m.n_tok <= kFusedTok && few && x_bytes <= kFusedBytes;
  const int64_t touched = std::min<int64_t>(m.n_tok * m.route->n_used, m.route->n_expert);
  const dim3 grid1((uint32_t)std::min<int64_t>(touched * (m.d_ff / kBlock), kUpWorkgroups));
  const dim3 grid2((uint32_t)(m.d_model / 16));
  hipError_t err = hipSuccess;
  if (!fused) {
    if (few) hipLaunchKernelGGL(front_kernel<4>, dim3((uint32_t)m.n_tok), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(front_kernel<8>, dim3((uint32_t)m.n_tok), dim3(256), 0, s, a);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  auto up = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid1, dim3(kThreads), fused ? x_bytes : 0, s, a);
  };
  auto by_route = [&](auto short_c) {
    constexpr bool S = decltype(short_c)::value;
    if (!fused) up(up_kernel<0, S>);
    else up(up_kernel<4, S>);
  };
  if (m.d_model / kBlock < 4) by_route(std::true_type{});
  else by_route(std::false_type{});
  if ((err = hipGetLastError()) != hipSuccess) return err;
  auto down = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid2, dim3(kThreads), (size_t)kWaves * m.n_tok * 64, s, a);
  };
  auto by_type = [&](auto short_c) {
    constexpr bool S = decltype(short_c)::value;
    if (m.out_type == kF32) down(down_kernel<S, kF32>);
    else if (m.out_type == kBF16) down(down_kernel<S, kBF16>);
    else down(down_kernel<S, kF16>);
  };
  if (m.d_ff / kBlock < 4) by_type(std::true_type{});
  else by_type(std::false_type{});
  return hipGetLastError();
}

}  // namespace mx
