// kv8_attn.h -- what the attention kernels share: query rows as matrix operands, a row's
// running softmax, and how partial results become outputs.
//
// Scores are kept in units of log2.  A row keeps a bound m with every score of it seen so far at
// most m + kSlack; weights are exp2(score - m + kBias), at most 2^15, so that they fit fp16 and
// all but the smallest keep its 11 bits.  The bound moves only when a score passes it by kSlack,
// which is rare, so most steps neither reduce a maximum over lanes nor rescale their sums.
// V's scales enter the weights as vs * 2^-E, at most 1, E being the exponent of the largest
// scale that the row has seen so far; a growth of E rescales the sums exactly.  E belongs to the row:
// blocks that only later rows of a tile see, or that lie before a row's window, may have any scale.
#pragma once

#include "kv8_device.h"

namespace kv {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.f, kBias = 7.f;
constexpr float kLowest = -3.0e38f;  // below every score, and finite: exp2(-inf - kLowest) is 0
constexpr int kNoScale = -200;       // E before any scale (fp32 exponents are above -150)

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_fast(float x) { return __builtin_amdgcn_logf(x); }
__device__ __forceinline__ int exponent_of(float x) { return __builtin_amdgcn_frexp_expf(x); }
__device__ __forceinline__ float ldexp_fast(float x, int e) { return __builtin_amdgcn_ldexpf(x, e); }

__device__ __forceinline__ f32x4 mfma16(h8 a, h8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(h8 a, h8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// f with the type as a constant.
template <class F>
__device__ __forceinline__ auto by_type(int type, F f) {
  switch (type) {
    case kF32: return f(std::integral_constant<int, kF32>());
    case kBF16: return f(std::integral_constant<int, kBF16>());
    default: return f(std::integral_constant<int, kF16>());
  }
}

template <int N>
__device__ __forceinline__ void load_row(const Rows &r, int64_t at, float (&v)[N]) {
  switch (r.type) {
    case kF32: load_values<kF32, N>(r.p, at, r.wide, v); break;
    case kBF16: load_values<kBF16, N>(r.p, at, r.wide, v); break;
    default: load_values<kF16, N>(r.p, at, r.wide, v); break;
  }
}

template <int N>
__device__ __forceinline__ void store_row(void *p, int type, int64_t at, const float (&v)[N]) {
  switch (type) {
    case kF32: store_values<kF32, N>(p, at, v); break;
    case kBF16: store_values<kBF16, N>(p, at, v); break;
    default: store_values<kF16, N>(p, at, v); break;
  }
}

// fp16 operand values of a row whose largest magnitude is amax: v * 2^-e below 2^14, in one
// half, or two whose sum has 22 bits.
struct RowScale {
  int e;
  float factor;  // of the row's integer products: score in log2 units = product * k scale * factor
  __device__ __forceinline__ RowScale(float amax, float scale) {
    const bool finite = as<uint32_t>(amax) < 0x7f800000u;
    e = finite && amax > 0.f ? exponent_of(amax) - 14 : 0;
    factor = finite ? ldexp_fast(scale * kLog2e, e) : as<float>(0x7fc00000u);
  }
};

// A row's result over some keys, its weights summed: value = sum of weights * codes.
// total > 0 or NaN where there were keys.
struct Finish {
  float lse2;    // log2 of the sum of exp2(score), the sink among them
  float factor;  // output = sum * factor
  // m: the row's bound; e: its exponent taken out of V's scales; sink2: log2 units, or -inf
  __device__ __forceinline__ Finish(float m, float total, int e, float sink2) {
    lse2 = total == 0.f ? -INFINITY : m - kBias + log2_fast(total);
    factor = total == 0.f ? 0.f : ldexp_fast(1.f / total, e);
    add_sink(sink2);
  }
  __device__ __forceinline__ void add_sink(float sink2) {
    if (sink2 == -INFINITY) return;
    const float top = fmaxf(lse2, sink2);
    const float all = lse2 != lse2 ? lse2 : top + log2_fast(exp2_fast(lse2 - top) + exp2_fast(sink2 - top));
    if (lse2 > -INFINITY) factor *= exp2_fast(lse2 - all);
    lse2 = all;
  }
};

// Where partial results lie (Plan).
struct Partials {
  float *out, *lse2;
  int64_t rows;
  __device__ __forceinline__ Partials(void *ws, const Batch &b, const Cache &c, int n_q, int splits)
      : out(static_cast<float *>(ws)), lse2(out + (int64_t)splits * b.n_tok * n_q * c.d), rows((int64_t)b.n_tok * n_q) {}
};

}  // namespace kv
