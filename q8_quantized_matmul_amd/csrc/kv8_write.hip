// kv8_write.hip -- rows into the 8-bit key/value cache and back.
//
// A wave takes 16 tokens of one head, keys or values: the granule in which both
// code layouts are contiguous (16 * d bytes).  The waves of one block of tokens
// sit in one workgroup, so the block's scale is one LDS exchange away.  For
// single tokens both kernels are bound by the chain table -> scale and codes -> store, for
// prompts (2 + 1 bytes a 16-bit value) reading by HBM (16384 tokens of 8 heads of 128 18.5 us, 5.4 TB/s),
// writing at 2.7 TB/s (36.8 us) by one round trip a wave and the exact quotients.
#include "kv8_device.h"

namespace kv {
namespace {

constexpr int kWriteThreads(int block_waves) { return 64 * (block_waves > 4 ? block_waves : 4); }

// A lane's share of 16 tokens: of K 16 dims of one token, of V 4 dims of 4 tokens, for each
// 64 dims of the head; either way 16 values whose codes are 16 adjacent bytes.
struct Share {
  int token0, tokens;  // first token of 16, and how many
  int dim0;            // first dim, of each 64
  __device__ __forceinline__ Share(bool is_k, int lane)
      : token0(is_k ? lane & 15 : lane >> 4 << 2),
        tokens(is_k ? 1 : 4),
        dim0(is_k ? lane >> 4 << 4 : (lane & 15) << 2) {}
};

// x / s to the nearest integer, ties to even, by the exact quotient.  What the callers round in fp32 is off by
// at most 127.5 * 2^-23 < 2^-16 (a reciprocal or ratio and a product, each rounded once), so only quotients
// nearer than 2^-15 to a tie come here: 6 % of the waves have one among 1024 values (with a margin of 2^-12,
// half of them: 16384 tokens of 8 heads of 128 took 39 us).  The difference x - n * s is exact in 64 bits,
// and so is its comparison with s / 2.
__device__ __forceinline__ float settle(float n, double x, double s) {
  const double r2 = 2.0 * __builtin_fma(-(double)n, s, x);
  if (r2 > s || (r2 == s && ((int)n & 1))) n += 1.f;
  if (r2 < -s || (r2 == -s && ((int)n & 1))) n -= 1.f;
  return n;
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: x + kMagic rounds x to an integer, in the low bits
constexpr float kNearTie = 0.5f - 0x1p-15f;

// Codes of 16 values under scale s (finite, not negative), inv = 1 / s.
__device__ __forceinline__ u32x4 encode16(const float (&x)[16], float s, float inv) {
  float m[16], far = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    m[i] = __builtin_fmaf(x[i], inv, kMagic);
    far = fmaxf(far, __builtin_fabsf(__builtin_fmaf(x[i], inv, kMagic - m[i])));
  }
  // subnormal scales: their reciprocals are infinite or inexact
  if (!(far < kNearTie) || s < 0x1p-126f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float n = 0.f;
      if (s >= 0x1p-126f)
        n = settle(m[i] - kMagic, x[i], s);
      else if (s > 0.f)
        n = (float)__builtin_rint((double)x[i] / (double)s);
      m[i] = fminf(fmaxf(n, -127.f), 127.f) + kMagic;
    }
  }
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = __builtin_amdgcn_perm(as<uint32_t>(m[4 * j + 1]), as<uint32_t>(m[4 * j]), 0x0c0c0400u);
    const uint32_t b = __builtin_amdgcn_perm(as<uint32_t>(m[4 * j + 3]), as<uint32_t>(m[4 * j + 2]), 0x04000c0cu);
    w[j] = a | b;
  }
  return w;
}

// 16 codes under scale s0 as codes under the larger s1, nearest even of the exact quotient; those of
// `older` bytes only.
__device__ __forceinline__ u32x4 requantize16(u32x4 codes, float s0, float s1, uint32_t older) {
  const float ratio = s0 / s1;
  float n[16], far = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x = (float)(int8_t)(codes[i >> 2] >> (8 * (i & 3))) * ratio;
    n[i] = __builtin_rintf(x);
    far = fmaxf(far, __builtin_fabsf(x - n[i]));
  }
  if (!(far < kNearTie)) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      n[i] = settle(n[i], (double)(int8_t)(codes[i >> 2] >> (8 * (i & 3))) * (double)s0, s1);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)n[4 * j + i] & 255u) << (8 * i);
    codes[j] = (w & older) | (codes[j] & ~older);
  }
  return codes;
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, false));
}
// The largest of the wave's values, without a detour through LDS.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_with<0xb1>(v);   // lanes 1 apart
  v = max_with<0x4e>(v);   // 2
  v = max_with<0x141>(v);  // the other four of eight
  v = max_with<0x140>(v);  // the other eight of sixteen
  auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// blockIdx.x: a slot of the batch's blocks; blockIdx.y: kUnits of the 2 * n_kv arrays of heads (all of K,
// then all of V).  (Several turns of kUnits in a workgroup, which then looks its block up once for them, took
// 37.5 to 39 us for 16384 tokens of 8 heads of 128 instead of 36.5.)
template <int TYPE, int D, int BLOCK_WAVES>
__global__ __launch_bounds__(kWriteThreads(BLOCK_WAVES)) void write_kernel(Cache c, Batch b, Rows kr, Rows vr) {
  constexpr int kWaves = kWriteThreads(BLOCK_WAVES) / 64, kUnits = kWaves / BLOCK_WAVES;
  constexpr int kBlock = 16 * BLOCK_WAVES, kPasses = D / 64;
  __shared__ uint32_t wave_amax[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % BLOCK_WAVES;

  // which sequence, which of its blocks
  int s = blockIdx.x, nth = 0;
  if (b.max_new > 1) {
    const Slots slots{kBlock, 1, 2};
    s = find_sequence(b, slots, blockIdx.x);
    nth = (int)(blockIdx.x - slots.first(b, s));
    if (nth < 0) return;  // starts that do not ascend from 0: a block before the table's first
  }
  const Span q = span_of(b, c, s);
  const int base = (max(q.first, 0) >> c.block_log << c.block_log) + nth * kBlock;
  const int t0 = max(q.first - base, 0), t1 = min(q.len - base, kBlock);  // new tokens of the block
  if (t0 >= t1) return;
  const int page = page_of(c, b, s, base);
  if (page < 0) return;

  const int mine = blockIdx.y * kUnits + wave / BLOCK_WAVES, unit = min(mine, 2 * c.n_kv - 1);
  const bool idle = mine != unit;  // only passes the barrier
  const bool is_k = unit < c.n_kv;
  const int head = is_k ? unit : unit - c.n_kv;
  // this lane's tokens of the block: first + i
  const Share sh(is_k, lane);
  const int first = 16 * part + sh.token0;
  // bytes of a lane's 16 that are new, or older ones
  uint32_t fresh = 0, older = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = first + (is_k ? 0 : i);
    if (!idle && t >= t0 && t < t1) fresh |= 255u << (8 * i);
    if (!idle && t < t0) older |= 255u << (8 * i);
  }
  const Rows &r = is_k ? kr : vr;
  const int64_t row = ((int64_t)q.row0 + base + first - q.first) * r.token_stride + (int64_t)head * r.head_stride + sh.dim0;
  float *const scale = (is_k ? c.ks : c.vs) + scale_offset(c, page, head, base);
  int8_t *const codes = (is_k ? c.k : c.v) + code_offset(c, page, head, base + 16 * part);
  // K [dims / 16][token][16]: a chunk of 16 dims is 256 bytes, a wave's pass 1024.
  // V [token / 4][dim][4]: four tokens are 4 * D bytes.
  const int at0 = is_k ? 16 * lane : sh.token0 * D + 4 * sh.dim0, at_step = is_k ? 1024 : 256;

  // all loads first: rows, and where the block or this lane's bytes hold others, what they hold
  float s0 = 0.f;
  if (t0 > 0) s0 = *scale;
  u32x4 was[kPasses];
  if (fresh != 0xffffffffu && (fresh | older)) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) was[p] = *reinterpret_cast<const u32x4 *>(codes + at0 + p * at_step);
  }
  float x[kPasses][16];
  if (is_k) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      if (fresh) {
        load_values<TYPE, 16>(r.p, row + 64 * p, r.wide, x[p]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[p][i] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      float t[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (fresh >> (8 * i) & 1) {
          load_values<TYPE, 4>(r.p, row + i * r.token_stride + 64 * p, r.wide, t[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) t[i][j] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) x[p][i] = t[i & 3][i >> 2];  // [dim][token], as V's codes lie
    }
  }
  uint32_t amax = 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max(amax, as<uint32_t>(x[p][i]) & 0x7fffffffu);
  amax = wave_max(amax);
  if constexpr (BLOCK_WAVES > 1) {
    if (lane == 0) wave_amax[wave] = amax;
    __syncthreads();  // also: every wave has read the old scale
#pragma unroll
    for (int i = 0; i < BLOCK_WAVES; ++i) amax = max(amax, wave_amax[wave - part + i]);
  }

  float s1 = as<float>(amax) / 127.f;  // IEEE division
  if (t0 > 0 && s0 > s1) s1 = s0;
  const bool bad = amax >= 0x7f800000u || (t0 > 0 && s0 != s0);
  if (bad) s1 = as<float>(0x7fc00000u);
  if (!(t0 > 0 && s1 > s0)) older = 0;  // the scale did not grow
  if (!idle && part == 0 && lane == 0) *scale = s1;
  if ((fresh | older) == 0) return;

  const float inv = 1.f / s1;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    u32x4 w = {0, 0, 0, 0};
    if (!bad) w = encode16(x[p], s1, inv);
    if (fresh != 0xffffffffu) {
      u32x4 old = was[p];
      if (older) old = requantize16(old, s0, s1, older);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (w[j] & fresh) | (old[j] & ~fresh);
    }
    *reinterpret_cast<u32x4 *>(codes + at0 + p * at_step) = w;
  }
}

template <int TYPE, int D>
__global__ __launch_bounds__(256) void read_kernel(Cache c, Batch b, void *k, void *v) {
  constexpr int kPasses = D / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int heads = (k ? c.n_kv : 0) + (v ? c.n_kv : 0);
  const int unit = blockIdx.y * 4 + wave;
  if (unit >= heads) return;
  const bool is_k = k && unit < c.n_kv;
  const int head = unit >= c.n_kv ? unit - c.n_kv : unit;
  int s = blockIdx.x, nth = 0;
  if (b.max_new > 1) {
    const Slots slots{16, 1, 2};
    s = find_sequence(b, slots, blockIdx.x);
    nth = (int)(blockIdx.x - slots.first(b, s));
  }
  const Span q = span_of(b, c, s);
  // positions below 0 (a sequence with more rows than tokens) make blocks of their own; where nth is below 0, t0 is
  // 16 at least
  const int base = (q.first >> 4 << 4) + nth * 16;
  const int t0 = max(q.first - base, 0), t1 = min(q.len - base, 16);
  if (t0 >= t1) return;
  const int page = base >= 0 ? page_of(c, b, s, base) : -1;
  float scale = base >= 0 ? as<float>(0x7fc00000u) : 0.f;
  if (page >= 0) scale = (is_k ? c.ks : c.vs)[scale_offset(c, page, head, base)];
  const int8_t *codes = (is_k ? c.k : c.v) + (page >= 0 ? code_offset(c, page, head, base) : 0);
  void *out = is_k ? k : v;
  const Share sh(is_k, lane);
  const int64_t stride = (int64_t)c.n_kv * D;
  const int64_t row = ((int64_t)q.row0 + base + sh.token0 - q.first) * stride + (int64_t)head * D + sh.dim0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int at = is_k ? 1024 * p + 16 * lane : sh.token0 * D + 4 * (64 * p + sh.dim0);
    u32x4 w = {0, 0, 0, 0};
    if (page >= 0) w = *reinterpret_cast<const u32x4 *>(codes + at);
    if (is_k) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3))) * scale;
      if (sh.token0 >= t0 && sh.token0 < t1) store_values<TYPE, 16>(out, row + 64 * p, x);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = (float)(int8_t)(w[j] >> (8 * i)) * scale;
        if (sh.token0 + i >= t0 && sh.token0 + i < t1) store_values<TYPE, 4>(out, row + i * stride + 64 * p, x);
      }
    }
  }
}

// Calls f with the head size as a constant.
template <class F>
hipError_t by_dim(int d, F f) {
  switch (d) {
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    case 192: return f(std::integral_constant<int, 192>());
    case 256: return f(std::integral_constant<int, 256>());
    default: return f(std::integral_constant<int, 512>());
  }
}

template <int TYPE, int D, int BW>
hipError_t write_launch(const Cache &c, const Batch &b, const Rows &k, const Rows &v, hipStream_t s) {
  constexpr int kUnits = kWriteThreads(BW) / 64 / BW;
  const uint32_t x = b.max_new > 1 ? (uint32_t)(b.n_tok / (16 * BW) + 2 * b.n_seq) : (uint32_t)b.n_seq;
  const uint32_t y = (uint32_t)((2 * c.n_kv + kUnits - 1) / kUnits);
  write_kernel<TYPE, D, BW><<<dim3(x, y), kWriteThreads(BW), 0, s>>>(c, b, k, v);
  return hipGetLastError();
}

template <int TYPE>
hipError_t write_type(const Cache &c, const Batch &b, const Rows &k, const Rows &v, hipStream_t s) {
  return by_dim(c.d, [&](auto d) {
    switch (c.block_log) {
      case 4: return write_launch<TYPE, d.value, 1>(c, b, k, v, s);
      case 5: return write_launch<TYPE, d.value, 2>(c, b, k, v, s);
      case 6: return write_launch<TYPE, d.value, 4>(c, b, k, v, s);
      default: return write_launch<TYPE, d.value, 8>(c, b, k, v, s);
    }
  });
}

template <int TYPE>
hipError_t read_type(const Cache &c, const Batch &b, void *k, void *v, hipStream_t s) {
  return by_dim(c.d, [&](auto d) {
    const uint32_t x = b.max_new > 1 ? (uint32_t)(b.n_tok / 16 + 2 * b.n_seq) : (uint32_t)b.n_seq;
    const int heads = (k ? c.n_kv : 0) + (v ? c.n_kv : 0);
    read_kernel<TYPE, d.value><<<dim3(x, (uint32_t)((heads + 3) / 4)), 256, 0, s>>>(c, b, k, v);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_write(const Cache &c, const Batch &b, const Rows &k, const Rows &v, hipStream_t s) {
  switch (k.type) {
    case kF32: return write_type<kF32>(c, b, k, v, s);
    case kBF16: return write_type<kBF16>(c, b, k, v, s);
    default: return write_type<kF16>(c, b, k, v, s);
  }
}

hipError_t launch_read(const Cache &c, const Batch &b, void *k, void *v, int type, hipStream_t s) {
  switch (type) {
    case kF32: return read_type<kF32>(c, b, k, v, s);
    case kBF16: return read_type<kBF16>(c, b, k, v, s);
    default: return read_type<kF16>(c, b, k, v, s);
  }
}

}  // namespace kv
