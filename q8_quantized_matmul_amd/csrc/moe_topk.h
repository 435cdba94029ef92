// moe_topk.h -- the MoE router's top-k of one token, on one wave.
//
// Lane l holds experts l, l + 64, ... .  Every expert's key (its score plus
// bias) becomes an unsigned number of the same order, 0 meaning "not
// eligible", and n_used rounds each take the maximum: a register maximum, a
// cross-lane maximum (six DPP moves), and ballots that find the lowest expert
// holding it, which breaks ties towards the lowest index.  Softmax keys order
// by the logits themselves, in 32 bits; sigmoid and sqrt(softplus) scores are
// formed in 64 bits, where neither rounding nor the math functions' last bits
// move an expert across another.
#pragma once

#include "mxfp4_device.h"

namespace mx {

constexpr int kSoftmax = 0, kSigmoid = 1, kSqrtSoftplus = 2;  // MOE_SOFTMAX, ...
constexpr int kMaxRouteExperts = 1024;
constexpr int kMaxUsed = 32;

struct RouteArgs {
  const float *logits;  // [n_tok][n_expert]
  const float *bias;    // [n_expert] or null
  int32_t n_expert, n_used, scoring, renormalize;
  float scale;
};

// Unsigned order of floating keys: negatives reversed, NaN above everything,
// -inf as 0.  Callers add +0 first, so that zeros of both signs are equal.
__device__ __forceinline__ uint32_t order32(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  const uint32_t o = (b >> 31) ? ~b : b | 0x80000000u;
  return b == 0xFF800000u ? 0u : o;
}
__device__ __forceinline__ uint64_t order64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  if ((b & ~(1ull << 63)) > 0x7FF0000000000000ull) return ~0ull;
  const uint64_t o = (b >> 63) ? ~b : b | (1ull << 63);
  return b == 0xFFF0000000000000ull ? 0ull : o;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_max(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
  const uint64_t o = ((uint64_t)hi << 32) | lo;
  return o > v ? o : v;
}
__device__ __forceinline__ uint32_t lane63(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
__device__ __forceinline__ uint64_t lane63(uint64_t v) {
  return ((uint64_t)lane63((uint32_t)(v >> 32)) << 32) | lane63((uint32_t)v);
}
// The wave's maximum, uniform.
template <typename K>
__device__ __forceinline__ K wave_max(K v) {
  v = dpp_max<q8::kDppXor1, 0xF>(v);
  v = dpp_max<q8::kDppXor2, 0xF>(v);
  v = dpp_max<q8::kDppHalfMirror, 0xF>(v);
  v = dpp_max<q8::kDppMirror, 0xF>(v);
  v = dpp_max<q8::kDppBcast15, 0xA>(v);
  v = dpp_max<q8::kDppBcast31, 0xC>(v);
  return lane63(v);
}
__device__ __forceinline__ float readlane_f32(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ float wave_sum(float v) { return readlane_f32(q8::group_sum<64>(v), 63); }

// n_used rounds of maximum: lane j < n_used ends with the id and score of slot
// j, or -1 and 0 if fewer experts are eligible.
template <int EPL, typename K>
__device__ __forceinline__ void take_largest(K (&key)[EPL], const float (&score)[EPL], int n_used,
                                             int lane, int &id, float &sc) {
  id = -1;
  sc = 0.0f;
  for (int j = 0; j < n_used; ++j) {
    K best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = key[i] > best ? key[i] : best;
    best = wave_max(best);
    if (best == 0) break;
    bool found = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint64_t who = __ballot(key[i] == best);
      if (!found && who != 0) {
        found = true;
        const int l = __ffsll((unsigned long long)who) - 1;
        const float s = readlane_f32(score[i], l);
        if (lane == j) {
          id = i * 64 + l;
          sc = s;
        }
        if (lane == l) key[i] = 0;
      }
    }
  }
}

// The routing of token t: lane j < n_used gets slot j's expert and weight.
template <int EPL>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, int lane, int &id,
                                            float &weight) {
  const float inf = __builtin_huge_valf();
  float z[EPL], b[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    z[i] = e < a.n_expert ? a.logits[t * a.n_expert + e] : -inf;
    b[i] = a.bias && e < a.n_expert ? a.bias[e] : 0.0f;
  }
  float sc, total = 1.0f;
  if (a.scoring == kSoftmax) {
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = z[i] == -inf ? 0u : order32(z[i] + b[i] + 0.0f);
    take_largest<EPL>(key, z, a.n_used, lane, id, sc);
    // exp(z - m) over the sum: m the largest chosen logit, or the largest of all
    // where the sum goes over all.  An order-preserving maximum keeps NaN.
    uint32_t top = id >= 0 ? order32(sc) : 0u;
    if (!a.renormalize) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) top = max(top, order32(z[i]));
    }
    top = wave_max(top);
    const float m = top == 0xFFFFFFFFu ? __builtin_nanf("")
                                       : __builtin_bit_cast(float, (top >> 31) ? top ^ 0x80000000u : ~top);
    float all = 0.0f;
    if (!a.renormalize) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) all += z[i] == -inf ? 0.0f : expf(z[i] - m);
    }
    weight = id >= 0 ? expf(sc - m) : 0.0f;
    total = wave_sum(a.renormalize ? weight : all);
  } else {
    uint64_t key[EPL];
    float score[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = 0;
      score[i] = 0.0f;
      if (i * 64 < a.n_expert) {  // uniform
        const double v = z[i];
        const double s = a.scoring == kSigmoid ? 1.0 / (1.0 + exp(-v))
                                               : sqrt(log1p(exp(-fabs(v))) + fmax(v, 0.0));
        score[i] = (float)(v != v ? v : s);
        key[i] = z[i] == -inf ? 0ull : order64((v != v ? v : s) + (double)b[i] + 0.0);
      }
    }
    take_largest<EPL>(key, score, a.n_used, lane, id, sc);
    weight = id >= 0 ? sc : 0.0f;
    if (a.renormalize) total = wave_sum(weight);
  }
  // A NaN sum must reach the weights; an empty row's zero sum must not.
  weight = (total == 0.0f ? weight : weight / total) * a.scale;
}

}  // namespace mx
