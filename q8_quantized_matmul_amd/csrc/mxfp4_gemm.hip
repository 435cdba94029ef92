// mxfp4_gemm.hip -- the MXFP4 product for many tokens, on 32x32x64 scaled matrix
// instructions (mxfp4_mfma.h).
//
// A workgroup of WM x WN waves computes 32 TM WM weight rows x 32 TN WN tokens.
// A stage is 256 values of every row, one 128-byte line: the copies go straight
// from memory to LDS, 1 KB (eight rows) an instruction, and two stages take
// turns, so the copies of the next one are in flight while one is multiplied,
// with one barrier a stage.
//
// LDS: 128 bytes a row; the 16-byte block c of row r lies at position c ^ (r % 8),
// which the copies get by reading that block from memory (a lane's place in LDS
// is fixed, its address in memory is not) and which makes the eight rows that are
// read together use all banks once.
//
// A lane's block of instruction s (of a stage's four) is block 4 h + s, h its half,
// so the four scale bytes it needs are one dword, the scale operand.  They go
// straight to registers: scattered loads, a row each, that cost as many cache
// lookups whatever they fetch, so a lane fetches eight bytes for two stages and
// trades one dword with the lane of the other half.
//
// Blocks past the end of a row are read from inside the row and given the scale
// byte 0 on both sides, whose products (below 2^-240) vanish in fp32; rows past
// the end of a matrix are read as its last row and not stored.
#include <algorithm>

#include "mxfp4_mfma.h"

namespace mx {
namespace {

constexpr int kStageBlocks = 8;
constexpr int kRowBytes = 128;  // of a stage
constexpr int kXcds = 8;

struct GemmArgs {
  void *out;  // or the partial sums [split][t][n]
  const uint8_t *w, *ws, *x, *xs;
  int32_t nb, n, t;
  int32_t tiles_n, tiles_t, splits, stages_per_split;
  bool wide;
};

// 64 lanes' 16 bytes to the 1 KB at `dst`, lane l's at dst + 16 l.
__device__ __forceinline__ void copy_to_lds(const uint8_t *src, uint8_t *dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
}

// Eight scale bytes at any address.  A lane reads those of blocks b..b+7, or, near
// the end of a row of nb >= 8 blocks, of the row's last eight, and shifts them
// down to b when it uses them (zero past the end).
__device__ __forceinline__ uint64_t load_scales(const uint8_t *p) {
  typedef uint64_t u64_a1 __attribute__((aligned(1)));
  return *reinterpret_cast<const u64_a1 *>(p);
}
__device__ __forceinline__ uint64_t shift_scales(uint64_t v, int b, int nb) {
  const int half = 4 * min(max(b + 8 - nb, 0), 8);  // bits; in two steps, so that 64 gives zero
  return (v >> half) >> half;
}
// Half h of the wave holds the scales of blocks 8 h + 0..7 of its row's sixteen;
// it needs blocks 4 h + 0..3 of the first eight (first) and of the last eight.
__device__ __forceinline__ void split_scales(uint64_t v, uint32_t &first, uint32_t &second) {
  const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)(v >> 32), false, false);
  first = r[0];
  second = r[1];
}

// Workgroups of one XCD (consecutive ids go round the eight) take neighbouring
// tiles, which share rows in its L2: bands of eight weight tiles, all token tiles
// of a band in turn.
__device__ __forceinline__ void tile_of(const GemmArgs &a, int &tn, int &tt, int &ts) {
  const int total = a.tiles_n * a.tiles_t * a.splits;
  int l = blockIdx.x;
  if (total % kXcds == 0) l = (l % kXcds) * (total / kXcds) + l / kXcds;
  const int per_split = a.tiles_n * a.tiles_t;
  ts = l / per_split;
  const int r = l - ts * per_split;
  constexpr int kBand = 8;
  const int band = r / (kBand * a.tiles_t), n0 = band * kBand;
  const int width = min(kBand, a.tiles_n - n0);
  const int q = r - n0 * a.tiles_t;
  tn = n0 + q % width;
  tt = q / width;
}

template <int WM, int WN, int TM, int TN, int TYPE>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_kernel(const GemmArgs a) {
  constexpr int kW = WM * WN;
  constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, ROWS = BM + BN;
  constexpr int COPIES = ROWS / 8 / kW;  // copy instructions of a wave per stage
  static_assert(ROWS % (8 * kW) == 0 && BM % (8 * kW) == 0, "whole copies per wave and matrix");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][ROWS * kRowBytes];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tn, tt, ts;
  tile_of(a, tn, tt, ts);
  const int n0 = tn * BM, t0 = tt * BN;
  const int st0 = ts * a.stages_per_split;
  const int stages_all = (a.nb + kStageBlocks - 1) / kStageBlocks;
  const int st1 = min(st0 + a.stages_per_split, stages_all);
  const int64_t row_bytes = (int64_t)a.nb * 16;

  // Copy i of the wave: rows 8 (wave + kW i) .. + 7 of the stage, weights first.
  const int lr = lane >> 3;
  const int chunk = (lane & 7) ^ lr;
  uint32_t off[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    const int r = 8 * (wave + kW * i) + lr;
    const int at = r < BM ? min(n0 + r, a.n - 1) - n0 : min(t0 + r - BM, a.t - 1) - t0;
    off[i] = (uint32_t)at * (uint32_t)row_bytes;
  }
  const uint8_t *wbase = a.w + n0 * row_bytes, *xbase = a.x + t0 * row_bytes;
  auto copy = [&](int st, int buf, auto from_c, auto to_c) {  // copies FROM..TO-1
    const int b0 = st * kStageBlocks;
    const uint32_t c = (uint32_t)min(chunk, a.nb - 1 - b0) * 16u;
    const uint8_t *w = wbase + (int64_t)b0 * 16, *x = xbase + (int64_t)b0 * 16;
#pragma unroll
    for (int i = decltype(from_c)::value; i < decltype(to_c)::value; ++i) {
      const uint8_t *src = (kW * i * 8 < BM ? w : x) + (off[i] + c);
      copy_to_lds(src, lds[buf] + (wave + kW * i) * 1024);
    }
  };
  constexpr std::integral_constant<int, 0> kFirst{};
  constexpr std::integral_constant<int, COPIES / 2> kHalf{};
  constexpr std::integral_constant<int, COPIES> kLast{};

  const int wm = wave % WM, wn = wave / WM;
  const int lrow = lane & 31, h = lane >> 5;
  const uint8_t *wsbase = a.ws + (int64_t)n0 * a.nb, *xsbase = a.xs + (int64_t)t0 * a.nb;
  uint32_t sw[TM], sx[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
    sw[i] = (uint32_t)(min(n0 + 32 * (wm * TM + i) + lrow, a.n - 1) - n0) * (uint32_t)a.nb;
#pragma unroll
  for (int j = 0; j < TN; ++j)
    sx[j] = (uint32_t)(min(t0 + 32 * (wn * TN + j) + lrow, a.t - 1) - t0) * (uint32_t)a.nb;
  uint64_t nw[TM], nx[TN];              // scales of the next two stages
  uint32_t dw[2][TM], dx[2][TN];        // of these two
  auto load_next_scales = [&](int st) {
    const uint32_t b = (uint32_t)min(st * kStageBlocks + 8 * h, a.nb - 8);
#pragma unroll
    for (int i = 0; i < TM; ++i) nw[i] = load_scales(wsbase + (sw[i] + b));
#pragma unroll
    for (int j = 0; j < TN; ++j) nx[j] = load_scales(xsbase + (sx[j] + b));
  };
  auto take_scales = [&](int st) {
    const int b = st * kStageBlocks + 8 * h;
#pragma unroll
    for (int i = 0; i < TM; ++i) split_scales(shift_scales(nw[i], b, a.nb), dw[0][i], dw[1][i]);
#pragma unroll
    for (int j = 0; j < TN; ++j) split_scales(shift_scales(nx[j], b, a.nb), dx[0][j], dx[1][j]);
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Block 4 h + s of the lane's row, s = 0..3, in a 32-row tile.
  const uint32_t rd = (uint32_t)lrow * kRowBytes + (uint32_t)(((4 * h) ^ (lane & 7)) * 16);
  const uint32_t rw = (uint32_t)wm * (TM * 32 * kRowBytes);
  const uint32_t rx = BM * kRowBytes + (uint32_t)wn * (TN * 32 * kRowBytes);
  u32x4 A[2][TM], B[2][TN];
  auto read = [&](int buf, auto s_c) {  // operands of instruction S of a stage
    constexpr int S = decltype(s_c)::value;
    const uint8_t *p = lds[buf] + (rd ^ (S * 16));
#pragma unroll
    for (int j = 0; j < TN; ++j) B[S & 1][j] = *reinterpret_cast<const u32x4 *>(p + rx + j * (32 * kRowBytes));
#pragma unroll
    for (int i = 0; i < TM; ++i) A[S & 1][i] = *reinterpret_cast<const u32x4 *>(p + rw + i * (32 * kRowBytes));
  };
  auto multiply = [&](auto s_c, auto buf_c) {
    constexpr int S = decltype(s_c)::value, U = decltype(buf_c)::value;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = mfma32<S>(A[S & 1][i], dw[U][i], B[S & 1][j], dx[U][j], acc[i][j]);
  };
  // The next step's reads, then the copies where there are some, one at a time
  // between the matrix instructions of this step, so that none waits for another.
  auto interleave = [&](auto copies_c) {
    constexpr int kCopies = decltype(copies_c)::value, kMfma = TM * TN, kReads = TM + TN;
    constexpr int kGap = kMfma / (kReads + kCopies) > 0 ? kMfma / (kReads + kCopies) : 1;
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, kGap, 0);  // matrix
    }
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // memory
      __builtin_amdgcn_sched_group_barrier(0x008, kGap, 0);
    }
  };
  constexpr std::integral_constant<int, 0> s0{};
  constexpr std::integral_constant<int, 1> s1{};
  constexpr std::integral_constant<int, 2> s2{};
  constexpr std::integral_constant<int, 3> s3{};

  // The copies of a stage are issued in the last step of the stage two before it
  // (the barrier there says that its buffer has been read) and in the step after.
  // Past the last stage they repeat it, into buffers that nobody reads any more, so
  // that the loop is one straight line for the scheduler; its scales are zero there.
  const int last = stages_all - 1;
  copy(st0, 0, kFirst, kLast);
  load_next_scales(st0);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __builtin_amdgcn_s_barrier();
  copy(min(st0 + 1, last), 1, kFirst, kHalf);
  read(0, s0);
  auto stage = [&](int st, auto buf_c) {
    constexpr int buf = decltype(buf_c)::value;
    if constexpr (buf == 0) {
      take_scales(st);
      load_next_scales(st + 2);
    }
    __builtin_amdgcn_sched_barrier(0);
    read(buf, s1);
    copy(min(st + 1, last), buf ^ 1, kHalf, kLast);
    multiply(s0, buf_c);
    interleave(kHalf);
    __builtin_amdgcn_sched_barrier(0);
    read(buf, s2);
    multiply(s1, buf_c);
    interleave(s0);
    __builtin_amdgcn_sched_barrier(0);
    read(buf, s3);
    multiply(s2, buf_c);
    interleave(s0);
    __builtin_amdgcn_sched_barrier(0);
    // The stage has been read (lgkmcnt), the next one's copies have landed (vmcnt).
    __builtin_amdgcn_s_waitcnt(0x0070);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(buf ^ 1, s0);
    copy(min(st + 2, last), buf, kFirst, kHalf);
    multiply(s3, buf_c);
    interleave(kHalf);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int st = st0; st < st1; st += 2) {
    stage(st, s0);
    stage(st + 1, s1);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // no copy outlives the workgroup

  const int64_t base = (int64_t)ts * a.t * a.n;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int t = t0 + 32 * (wn * TN + j) + lrow;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int o = n0 + 32 * (wm * TM + i) + 8 * q + 4 * h;
        if (t < a.t && o < a.n) {
          const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          store4<TYPE>(a.out, base + (int64_t)t * a.n + o, v, a.n - o, a.wide);
        }
      }
    }
  }
}

// out[i] = sum over s of part[s][i], in order; `elems` values, four a lane.
template <int TYPE>
__global__ __launch_bounds__(256) void reduce_kernel(void *__restrict__ out, const float *__restrict__ part,
                                                     int64_t elems, int splits, bool wide) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= elems) return;
  if (i + 4 <= elems && elems % 4 == 0) {
    f32x4 v = *reinterpret_cast<const f32x4 *>(part + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4 *>(part + s * elems + i);
    store4<TYPE>(out, i, v, 4, wide);
  } else {
    f32x4 v{};
    for (int j = 0; j < 4 && i + j < elems; ++j) {
      float u = part[i + j];
      for (int s = 1; s < splits; ++s) u += part[s * elems + i + j];
      v[j] = u;
    }
    store4<TYPE>(out, i, v, (int)min<int64_t>(4, elems - i), false);
  }
}

struct Tile {
  int bm, bn;
};
// Tile shapes, largest first.
constexpr Tile kTiles[] = {{256, 256}, {256, 128}, {128, 128}, {128, 64}, {64, 64}};

}  // namespace

GemmPlan gemm_plan(int64_t in_dim, int64_t out_dim, int64_t n_tok, size_t ws_bytes) {
  GemmPlan p{};
  const int64_t stages = (in_dim / kBlock + kStageBlocks - 1) / kStageBlocks;
  int64_t tiles = 0;
  for (int i = 0; i < 5; ++i) {
    p.tile = i;
    tiles = ((out_dim + kTiles[i].bm - 1) / kTiles[i].bm) * ((n_tok + kTiles[i].bn - 1) / kTiles[i].bn);
    if (tiles >= 256) break;
  }
  p.splits = 1;
  const int64_t want = std::min<int64_t>(256 / std::max<int64_t>(tiles, 1), stages / 4);
  const int64_t fit = (int64_t)(ws_bytes / ((size_t)out_dim * n_tok * 4));
  p.splits = (int)std::max<int64_t>(1, std::min({want, fit, (int64_t)16}));
  p.stages_per_split = (int)((stages + p.splits - 1) / p.splits + 1) / 2 * 2;  // taken in twos
  p.splits = (int)((stages + p.stages_per_split - 1) / p.stages_per_split);
  return p;
}

size_t gemm_workspace_bytes(int64_t in_dim, int64_t out_dim, int64_t n_tok) {
  const GemmPlan p = gemm_plan(in_dim, out_dim, n_tok, SIZE_MAX);
  return p.splits > 1 ? (size_t)p.splits * out_dim * n_tok * 4 : 0;
}

hipError_t launch_gemm(const GemmPlan &p, void *out, int out_type, const uint8_t *w, const uint8_t *ws,
                       int64_t in_dim, int64_t out_dim, const uint8_t *x, const uint8_t *xs,
                       int64_t n_tok, void *workspace, hipStream_t s) {
  const Tile tile = kTiles[p.tile];
  const bool split = p.splits > 1;
  const int type = split ? kF32 : out_type;
  void *dst = split ? workspace : out;
  auto wide_of = [&](const void *q, int ty) {
    return out_dim % 4 == 0 && (reinterpret_cast<uintptr_t>(q) & (ty == kF32 ? 15 : 7)) == 0;
  };
  GemmArgs a{dst, w, ws, x, xs, (int32_t)(in_dim / kBlock), (int32_t)out_dim, (int32_t)n_tok,
             (int32_t)((out_dim + tile.bm - 1) / tile.bm), (int32_t)((n_tok + tile.bn - 1) / tile.bn),
             p.splits, p.stages_per_split, wide_of(dst, type)};
  const dim3 grid((uint32_t)((int64_t)a.tiles_n * a.tiles_t * a.splits));
  auto go = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, a); };
  auto by_tile = [&](auto type_c) {
    constexpr int T = decltype(type_c)::value;
    switch (p.tile) {
      case 0: return go(gemm_kernel<2, 2, 4, 4, T>, 256);
      case 1: return go(gemm_kernel<2, 2, 4, 2, T>, 256);
      case 2: return go(gemm_kernel<2, 2, 2, 2, T>, 256);
      case 3: return go(gemm_kernel<2, 2, 2, 1, T>, 256);
      default: return go(gemm_kernel<2, 2, 1, 1, T>, 256);
    }
  };
  if (type == kF32) by_tile(std::integral_constant<int, kF32>{});
  else if (type == kBF16) by_tile(std::integral_constant<int, kBF16>{});
  else by_tile(std::integral_constant<int, kF16>{});
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !split) return err;
  const int64_t elems = out_dim * n_tok;
  const dim3 rgrid((uint32_t)((elems + 1023) / 1024));
  const float *part = static_cast<const float *>(workspace);
  const bool wide = (reinterpret_cast<uintptr_t>(out) & (out_type == kF32 ? 15 : 7)) == 0;
  auto red = [&](auto kernel) { hipLaunchKernelGGL(kernel, rgrid, dim3(256), 0, s, out, part, elems, p.splits, wide); };
  if (out_type == kF32) red(reduce_kernel<kF32>);
  else if (out_type == kBF16) red(reduce_kernel<kBF16>);
  else red(reduce_kernel<kF16>);
  return hipGetLastError();
}

}  // namespace mx
