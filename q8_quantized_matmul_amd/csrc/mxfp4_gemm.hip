// mxfp4_gemm.hip -- the MXFP4 product for many tokens, on 32x32x64 scaled matrix
// instructions (mxfp4_mfma.h).
//
// A workgroup of WM x WN waves computes 32 TM WM weight rows x 32 TN WN tokens.
// A stage is 256 values of every row, one 128-byte line: the copies go straight
// from memory to LDS, 1 KB (eight rows) an instruction, into the RING places that
// stages take in turn, with one barrier a stage; while one stage is multiplied the
// copies of a later one are in flight.
//
// They are so for one stage at most, whatever RING is.  The waits written here are
// counted, but the compiler, to which every place is the same array, adds waits for all
// copies in flight: in the 64x64 kernel in front of each stage's LDS reads (so its ring
// of four runs as one of two), in the 256x256 kernel at the start of three stages in
// four, right behind the issue of their successors' copies.  In the other two no copies
// are in flight where it would.
//
// What bounds it: 256 workgroups of 256^2 tiles take 1.55 us a stage, of which the
// copies alone are 1.3 (the second caches' rate) and the matrix instructions alone
// 1.34 (6.4 PFLOP/s, what the chip holds on random values for its power; 9.6 on
// constant ones); then the waits above, the stores and the join of the splits.  8192^3
// 306 us, 3.6 PFLOP/s (bf16 outputs 283 to 290); 4096^3 47 (43); 32768 -> 1024 at 2048
// tokens 46 us and 7 for the join; 4096 -> 2048 at 200 7.2 us with two sets of weights in
// turn, 9.1 with four: launch, first loads, sixteen stages of 0.4 us, which is the
// latency of their copies behind four matrix instructions, and stores.
//
// LDS: 128 bytes a row; the 16-byte block c of row r lies at position c ^ (r / 2 % 8),
// which the copies get by reading that block from memory (a lane's place in LDS
// is fixed, its address in memory is not) and which makes sixteen rows that are
// read together use all 64 banks once.
//
// A lane's block of instruction s (of a stage's four) is block 4 h + s, h its half,
// so the four scale bytes it needs are one dword, the scale operand.  A row's scales
// of a stage are eight bytes of a cache line that the copies push out of the first
// cache before the next stage wants it, so they are fetched for four stages at once,
// 32 bytes a row by two lanes, and shared by the waves through LDS (fetched by the
// lanes that use them, two stages at a time: 8192^3 335 us for 311).
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

// Sixteen scale bytes at any address.  A lane reads those of blocks b..b+15, or,
// near the end of a row of nb >= 16 blocks, of the row's last sixteen, and shifts
// them down to b when it uses them (zero past the end).
struct Scales16 {
  uint64_t lo, hi;
};
__device__ __forceinline__ Scales16 load_scales(const uint8_t *p) {
  typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
  const u32x4_a1 v = *reinterpret_cast<const u32x4_a1 *>(p);
  return {v.x | ((uint64_t)v.y << 32), v.z | ((uint64_t)v.w << 32)};
}
__device__ __forceinline__ u32x4 shift_scales(Scales16 v, int b, int nb) {
  const int bytes = min(max(b + 16 - nb, 0), 16);
  if (bytes >= 8) v = {v.hi, 0};
  const int half = 4 * (bytes >= 8 ? bytes - 8 : bytes);  // bits; in two steps, so that 64 gives zero
  const uint64_t lo = (v.lo >> half) >> half | (v.hi << (32 - half)) << (32 - half);
  const uint64_t hi = (v.hi >> half) >> half;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
// Waits until at most N of the wave's memory operations, and none of its LDS
// operations, are outstanding.
template <int N>
__device__ __forceinline__ void wait_memory() {
  static_assert(N < 64, "six bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
// Half h of the wave holds dwords 4 h + 0..3 of its row's eight; stage u of the four
// needs dword 2 u + h.
__device__ __forceinline__ void split_scales(const u32x4 &v, uint32_t (&d)[4]) {
  const auto p = __builtin_amdgcn_permlane32_swap(v.x, v.y, false, false);
  const auto q = __builtin_amdgcn_permlane32_swap(v.z, v.w, false, false);
  d[0] = p[0];
  d[1] = q[0];
  d[2] = p[1];
  d[3] = q[1];
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

template <int WM, int WN, int TM, int TN, int RING, int TYPE>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm_kernel(const GemmArgs a) {
  constexpr int kW = WM * WN, kThreads = 64 * kW;
  constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, ROWS = BM + BN;
  constexpr int COPIES = ROWS / 8 / kW;  // copy instructions of a wave per stage
  constexpr int FETCHES = (ROWS * 2 + kThreads - 1) / kThreads;  // scale fetches of a thread per group
  static_assert(ROWS % (8 * kW) == 0 && BM % (8 * kW) == 0 && kW % 2 == 0, "whole copies per wave and matrix");
  __shared__ __attribute__((aligned(16))) uint8_t lds[RING][ROWS * kRowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t lds_scales[FETCHES * kThreads * 16];

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
  const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lr >> 1)) & 7);
  uint32_t off[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    const int r = 8 * (wave + kW * i) + lr;
    const int at = r < BM ? min(n0 + r, a.n - 1) - n0 : min(t0 + r - BM, a.t - 1) - t0;
    off[i] = (uint32_t)at * (uint32_t)row_bytes;
  }
  const uint8_t *wbase = a.w + n0 * row_bytes, *xbase = a.x + t0 * row_bytes;
  auto copy = [&](int st, int buf) {
    const int b0 = st * kStageBlocks;
    const uint32_t c = (uint32_t)min(chunk, a.nb - 1 - b0) * 16u;
    const uint8_t *w = wbase + (int64_t)b0 * 16, *x = xbase + (int64_t)b0 * 16;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const uint8_t *src = (kW * i * 8 < BM ? w : x) + (off[i] + c);
      copy_to_lds(src, lds[buf] + (wave + kW * i) * 1024);
    }
  };

  const int wm = wave % WM, wn = wave / WM;
  const int lrow = lane & 31, h = lane >> 5;
  // Scale fetch i of the thread: half (tid & 1) of the group's 32 bytes of a row.
  const uint8_t *wsbase = a.ws + (int64_t)n0 * a.nb, *xsbase = a.xs + (int64_t)t0 * a.nb;
  const int sh = threadIdx.x & 1;
  uint32_t soff[FETCHES];
#pragma unroll
  for (int i = 0; i < FETCHES; ++i) {
    const int r = min((int)threadIdx.x / 2 + i * (kThreads / 2), ROWS - 1);
    const int at = r < BM ? min(n0 + r, a.n - 1) - n0 : min(t0 + r - BM, a.t - 1) - t0;
    soff[i] = (uint32_t)at * (uint32_t)a.nb;
  }
  Scales16 fetched[FETCHES];
  auto fetch_scales = [&](int st) {
    const uint32_t b = (uint32_t)min(st * kStageBlocks + 16 * sh, a.nb - 16);
#pragma unroll
    for (int i = 0; i < FETCHES; ++i) {
      const bool isw = (int)threadIdx.x / 2 + i * (kThreads / 2) < BM;
      fetched[i] = load_scales((isw ? wsbase : xsbase) + (soff[i] + b));
    }
  };
  auto share_scales = [&](int st) {
#pragma unroll
    for (int i = 0; i < FETCHES; ++i)  // the last may go past the rows, into padding
      *reinterpret_cast<u32x4 *>(lds_scales + (threadIdx.x + i * kThreads) * 16) =
          shift_scales(fetched[i], st * kStageBlocks + 16 * sh, a.nb);
  };
  u32x4 rw_s[TM], rx_s[TN];       // the next group's scales as read
  uint32_t dw[TM][4], dx[TN][4];  // scale operands of the group's stages
  auto read_scales = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
      rw_s[i] = *reinterpret_cast<const u32x4 *>(lds_scales + (32 * (wm * TM + i) + lrow) * 32 + h * 16);
#pragma unroll
    for (int j = 0; j < TN; ++j)
      rx_s[j] = *reinterpret_cast<const u32x4 *>(lds_scales + (BM + 32 * (wn * TN + j) + lrow) * 32 + h * 16);
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i) split_scales(rw_s[i], dw[i]);
#pragma unroll
    for (int j = 0; j < TN; ++j) split_scales(rx_s[j], dx[j]);
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Block 4 h + s of the lane's row, s = 0..3, in a 32-row tile.
  const uint32_t rd = (uint32_t)lrow * kRowBytes + (uint32_t)(((4 * h) ^ ((lrow >> 1) & 7)) * 16);
  const uint32_t rw = (uint32_t)wm * (TM * 32 * kRowBytes);
  const uint32_t rx = BM * kRowBytes + (uint32_t)wn * (TN * 32 * kRowBytes);
  // Two sets of operands: of the stage's instructions in turn, or, for small tiles, of
  // this stage and the next, so that a stage waits for LDS once and not four times.
  constexpr bool kSmall = TM * TN <= 4;
  constexpr int kHeld = kSmall ? 4 : 1;
  u32x4 A[2][kHeld][TM], B[2][kHeld][TN];
  auto read = [&](int buf, auto s_c, auto set_c) {  // operands of instruction S of a stage
    constexpr int S = decltype(s_c)::value, SET = decltype(set_c)::value, AT = kSmall ? S : 0;
    const uint8_t *p = lds[buf] + (rd ^ (S * 16));
#pragma unroll
    for (int j = 0; j < TN; ++j) B[SET][AT][j] = *reinterpret_cast<const u32x4 *>(p + rx + j * (32 * kRowBytes));
#pragma unroll
    for (int i = 0; i < TM; ++i) A[SET][AT][i] = *reinterpret_cast<const u32x4 *>(p + rw + i * (32 * kRowBytes));
  };
  auto multiply = [&](auto s_c, auto u_c, auto set_c) {
    constexpr int S = decltype(s_c)::value, U = decltype(u_c)::value;
    constexpr int SET = decltype(set_c)::value, AT = kSmall ? S : 0;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = mfma32<S>(A[SET][AT][i], dw[i][U], B[SET][AT][j], dx[j][U], acc[i][j]);
  };
  // With one wave a SIMD, whatever is issued between matrix instructions is free
  // and whatever is issued between steps is not.  The next step's reads (and other
  // LDS accesses), then the copies or scale fetches where there are some, go
  // between the matrix instructions of this step, arithmetic over all of them.
  auto interleave = [&](auto reads_c, auto memory_c, auto valu_c) {
    constexpr int kReads = decltype(reads_c)::value, kMemory = decltype(memory_c)::value;
    constexpr int kMfma = TM * TN, kAll = kReads + kMemory, kMost = (kAll + kMfma - 1) / kMfma;
    constexpr int kValu = (decltype(valu_c)::value + kMfma - 1) / kMfma;
#pragma unroll
    for (int k = 0; k < kMfma; ++k) {
      const int from = k * kAll / kMfma, to = (k + 1) * kAll / kMfma;
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        if (from + i < to) {
          if (from + i < kReads) __builtin_amdgcn_sched_group_barrier(0x080, 1, 0);  // LDS
          else __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);                    // memory
        }
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                     // matrix
      if (kValu > 0) __builtin_amdgcn_sched_group_barrier(0x002, kValu, 0);  // arithmetic
    }
  };
  constexpr std::integral_constant<int, 0> s0{};
  constexpr std::integral_constant<int, 1> s1{};
  constexpr std::integral_constant<int, 2> s2{};
  constexpr std::integral_constant<int, 3> s3{};
  constexpr std::integral_constant<int, TM + TN> kReads{};
  constexpr std::integral_constant<int, 2 * (TM + TN)> kMoreReads{};
  constexpr std::integral_constant<int, TM + TN + FETCHES> kReadsWrites{};
  constexpr std::integral_constant<int, COPIES> kCopies{};
  constexpr std::integral_constant<int, FETCHES> kFetches{};
  constexpr std::integral_constant<int, 24 * FETCHES> kShifts{};

  // The copies of a stage are issued in the stage RING before it, behind the barrier
  // that says that its place has been read.  Past the last stage they repeat it, into
  // places that nobody reads any more, so that a stage is one straight line for the
  // scheduler; its scales are zero there.
  const int last = stages_all - 1;
  fetch_scales(st0);
#pragma unroll
  for (int r = 0; r < RING; ++r) copy(min(st0 + r, last), r);
  share_scales(st0);
  wait_memory<(RING - 1) * COPIES>();
  __builtin_amdgcn_s_barrier();
  auto read_stage = [&](int buf, auto set_c) {
    read(buf, s0, set_c);
    read(buf, s1, set_c);
    read(buf, s2, set_c);
    read(buf, s3, set_c);
  };
  if constexpr (kSmall) read_stage(0, s0);
  else read(0, s0, s0);
  read_scales();
  // Stage U of a group of four: fetch the next group's scales, leave them in LDS (the
  // group's own were read three barriers ago), read them.
  auto small_stage = [&](int st, auto u_c) {
    constexpr int U = decltype(u_c)::value, buf = U % RING;
    constexpr std::integral_constant<int, U & 1> now{};
    constexpr std::integral_constant<int, (U & 1) ^ 1> next{};
    // The stage is in registers and the next one's copies have landed; of the counted
    // operations later copies and a scale fetch may be outstanding.
    wait_memory<(RING - 2) * COPIES + (U >= 1 && U < RING ? FETCHES : 0)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_stage((buf + 1) % RING, next);
    if constexpr (U == 3) read_scales();
    copy(min(st + RING, last), buf);
    if constexpr (U == 0) {
      // Behind the copies: the waits of the next stages leave room for it, and not for them.
      __builtin_amdgcn_sched_barrier(0);
      fetch_scales(st + 4);
    }
    __builtin_amdgcn_sched_barrier(0);
    multiply(s0, u_c, now);
    multiply(s1, u_c, now);
    multiply(s2, u_c, now);
    multiply(s3, u_c, now);
    if constexpr (U == 2) share_scales(st + 2);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto large_stage = [&](int st, auto u_c) {
    constexpr int U = decltype(u_c)::value, buf = U & 1;
    __builtin_amdgcn_sched_barrier(0);
    read(buf, s1, s1);
    multiply(s0, u_c, s0);
    interleave(kReads, s0, s0);
    __builtin_amdgcn_sched_barrier(0);
    read(buf, s2, s0);
    if constexpr (U == 0) fetch_scales(st + 4);
    multiply(s1, u_c, s1);
    if constexpr (U == 0) interleave(kReads, kFetches, kFetches);
    else interleave(kReads, s0, s0);
    __builtin_amdgcn_sched_barrier(0);
    read(buf, s3, s1);
    if constexpr (U == 2) share_scales(st + 2);
    multiply(s2, u_c, s0);
    if constexpr (U == 2) interleave(kReadsWrites, s0, kShifts);
    else interleave(kReads, s0, s0);
    __builtin_amdgcn_sched_barrier(0);
    // The stage has been read and the next one's copies have landed; a scale fetch,
    // issued after them, may be outstanding.
    wait_memory<(U == 0 ? FETCHES : 0)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(buf ^ 1, s0, s0);
    if constexpr (U == 3) read_scales();
    copy(min(st + 2, last), buf);
    multiply(s3, u_c, s1);
    if constexpr (U == 3) interleave(kMoreReads, kCopies, kCopies);
    else interleave(kReads, kCopies, kCopies);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto stage = [&](int st, auto u_c) {
    if constexpr (kSmall) small_stage(st, u_c);
    else large_stage(st, u_c);
  };
  // A last group of one or two stages is taken alone, but for the largest tile, whose
  // registers leave no room for a second copy of the code: it multiplies zeros there.
  // gemm_plan gives a split whole pairs, or whole fours, so no split takes the next one's.
  constexpr bool kTail = kSmall;
  int st = st0;
  for (; st + (kTail ? 2 : 0) < st1; st += 4) {
    take_scales();
    stage(st, s0);
    stage(st + 1, s1);
    stage(st + 2, s2);
    stage(st + 3, s3);
  }
  if (kTail && st < st1) {
    take_scales();
    stage(st, s0);
    stage(st + 1, s1);
  }
  wait_memory<0>();
  __builtin_amdgcn_s_barrier();  // every wave's copies have landed, and been read

  // Through LDS, a region a wave, so that a store writes whole lines of out: as the
  // lanes hold them it would write 32 bytes of 32 rows (1024 -> 32768 at 512 tokens 26.9
  // us, so 22.8, with bf16 outputs 24.3 and 20.1; 4096^3 49 and 47, 49 and 43; 8192^3
  // 311 and 306, 304 and 290).  The 16-byte chunk c of row r
  // lies at c ^ (r % 16) (% 8 in rows of eight), which spreads rows over the banks.
  constexpr int kChunks = TM * 8, kSwizzle = (kChunks < 16 ? kChunks : 16) - 1;
  static_assert(kW * 32 * kChunks * 16 <= RING * ROWS * kRowBytes, "the regions fit in the stages' places");
  uint8_t *mine = &lds[0][0] + wave * (32 * kChunks * 16);
  const int64_t base = (int64_t)ts * a.t * a.n;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4 *>(mine + (lrow * kChunks + ((8 * i + 2 * q + h) ^ (lrow & kSwizzle))) * 16) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int k = 0; k < 32 * kChunks / 64; ++k) {
      const int at = k * 64 + lane, r = at / kChunks, c = at % kChunks;
      const f32x4 v = *reinterpret_cast<const f32x4 *>(mine + (r * kChunks + (c ^ (r & kSwizzle))) * 16);
      const int t = t0 + 32 * (wn * TN + j) + r, o = n0 + 32 * wm * TM + 4 * c;
      if (t < a.t && o < a.n) store4<TYPE>(a.out, base + (int64_t)t * a.n + o, v, a.n - o, a.wide);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

// Tile shapes, and what a stage of 256 values takes when `at` workgroups share the
// chip's 256 compute units (microseconds, measured; `slots` of them run at once).
struct Tile {
  int bm, bn, slots;
  float us_full, us_half;  // at slots, at 256 workgroups
};
constexpr Tile kTiles[] = {{256, 256, 256, 1.55f, 1.55f},
                           {128, 128, 512, 1.25f, 1.1f},
                           {128, 64, 512, 0.95f, 0.75f},
                           {64, 64, 512, 0.65f, 0.4f}};
constexpr int kNumTiles = 4, kMaxSplit = 16;
// A split costs a launch and the partial sums' way to memory and back.
constexpr float kSplitUs = 4.0f, kPartialBytesPerUs = 4.0e6f;

}  // namespace

// The tile and split of the smallest estimated time.  Large tiles read each row
// fewer times, small ones give every compute unit work, and a split over K does
// for long rows what small tiles do for many.  Measured, microseconds, fp32 outputs,
// chosen first: 4096 -> 4096 at 4096 tokens 256^2 tiles 47, 128^2 52; 4096 -> 2048 at
// 4096 128^2 28, 256^2 35; at 2048 128x64 18.9, 64^2 22.0; at 1024 64^2 12.4, 128x64
// 14.3; 32768 -> 1024 at 2048 128^2 in 4 splits 54, 256^2 in 8 59, 128x64 in 2 59; 7168
// -> 2048 at 129 64^2 in 2 splits 11.5, unsplit 13.2.
GemmPlan gemm_plan(int64_t in_dim, int64_t out_dim, int64_t n_tok, size_t ws_bytes) {
  const int64_t stages = (in_dim / kBlock + kStageBlocks - 1) / kStageBlocks;
  const double out_bytes = 4.0 * (double)out_dim * (double)n_tok;
  GemmPlan best{};
  double best_us = 0;
  for (int i = 0; i < kNumTiles; ++i) {
    const Tile &t = kTiles[i];
    const int64_t tiles = ((out_dim + t.bm - 1) / t.bm) * ((n_tok + t.bn - 1) / t.bn);
    // The kernels take whole pairs of stages, the largest tile whole groups of four.
    const int64_t whole = i == 0 ? 4 : 2;
    for (int want = 1; want <= kMaxSplit; want *= 2) {
      const int64_t per_split = ((stages + want - 1) / want + whole - 1) / whole * whole;
      const int64_t splits = (stages + per_split - 1) / per_split;
      if (want > 1 && (stages < 4 * want || tiles * want > t.slots)) break;
      if (splits > 1 && splits * out_bytes > (double)ws_bytes) break;
      const double groups = (double)(tiles * splits);
      const double stage_us = groups <= 256 ? t.us_half : t.us_half + (t.us_full - t.us_half) * std::min(1.0, (groups - 256) / (t.slots - 256 + 1.0));
      double us = std::max(1.0, groups / t.slots) * (double)std::min(per_split, stages) * stage_us;
      if (splits > 1) us += kSplitUs + 2.0 * splits * out_bytes / kPartialBytesPerUs;
      if ((i == 0 && want == 1) || us < best_us) {
        best_us = us;
        best = {i, (int)splits, (int)per_split};
      }
    }
  }
  return best;
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
      case 0: return go(gemm_kernel<2, 4, 4, 2, 2, T>, 512);
      case 1: return go(gemm_kernel<2, 2, 2, 2, 2, T>, 256);
      case 2: return go(gemm_kernel<2, 2, 2, 1, 2, T>, 256);
      default: return go(gemm_kernel<2, 2, 1, 1, 4, T>, 256);
    }
  };
  if (type == kF32) by_tile(std::integral_constant<int, kF32>{});
  else if (type == kBF16) by_tile(std::integral_constant<int, kBF16>{});
  else by_tile(std::integral_constant<int, kF16>{});
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !split) return err;
  return launch_reduce(out, out_type, static_cast<const float *>(workspace), out_dim * n_tok, p.splits, s);
}

hipError_t launch_reduce(void *out, int out_type, const float *part, int64_t elems, int splits, hipStream_t s) {
  const dim3 grid((uint32_t)((elems + 1023) / 1024));
  const bool wide = (reinterpret_cast<uintptr_t>(out) & (out_type == kF32 ? 15 : 7)) == 0;
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, out, part, elems, splits, wide); };
  if (out_type == kF32) go(reduce_kernel<kF32>);
  else if (out_type == kBF16) go(reduce_kernel<kBF16>);
  else go(reduce_kernel<kF16>);
  return hipGetLastError();
}

}  // namespace mx
