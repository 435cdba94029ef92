// moe_topk.h -- the MoE router's top-k of one token, on one wave.
//
// Lane l holds experts l, l + 64, ... .  An expert's key becomes an unsigned number
// of the same order, 0 meaning "not eligible".  Softmax keys are logit plus bias, in
// 32 bits; sigmoid and sqrt(softplus) keys are score plus bias and compared in 64
// bits, where neither rounding nor the math functions' last bits move an expert
// across another.
//
// The n_used-th largest of the lanes' maxima is no more than the n_used-th largest
// key, so the keys from it up hold all that are chosen, and mostly few others.
// These candidates move to a lane each and count the ones before them, which is
// their slot: no chain of n_used dependent maxima over all experts.  For the scores
// that first step needs only bounds from 32-bit math, and the 64-bit exp and log
// are taken once a lane, not once an expert.  Bound by the latency of that chain of
// cross-lane steps (256 experts, 8 of them, a single token 4.2, 4.5 and 5.9 us for
// the three scores) and, for many tokens, by instructions: 4096 tokens 6.2, 7.2 and
// 10.5 us, where n_used rounds of maximum over 64-bit keys of every expert took 5.4,
// 9.3 and 14.1; 1024 experts, 32 of them: 17.8, 21.3, 31.6 against 28.7, 50.1, 68.4.
// A token with more than 64 candidates takes them in turn, some 90 us: with normal
// logits one in 30 000 at 1024 experts and 32 used, and none in 300 000 with fewer of either;
// 4096 tokens of 256 equal logits each, 8 used, 14.8, 17.2 and 23.2.
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
// The wave's maximum, uniform.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<q8::kDppXor1, 0xF>(v);
  v = dpp_max<q8::kDppXor2, 0xF>(v);
  v = dpp_max<q8::kDppHalfMirror, 0xF>(v);
  v = dpp_max<q8::kDppMirror, 0xF>(v);
  v = dpp_max<q8::kDppBcast15, 0xA>(v);
  v = dpp_max<q8::kDppBcast31, 0xC>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t high(uint32_t v) { return v; }
__device__ __forceinline__ uint32_t high(uint64_t v) { return (uint32_t)(v >> 32); }
__device__ __forceinline__ float readlane_f32(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ float wave_sum(float v) { return readlane_f32(q8::group_sum<64>(v), 63); }

// The score of a logit other than -inf, in 64 bits.  NaN stays NaN.
__device__ __forceinline__ double score64(int scoring, double v) {
  const double s = scoring == kSigmoid ? 1.0 / (1.0 + exp(-v)) : sqrt(log1p(exp(-fabs(v))) + fmax(v, 0.0));
  return v != v ? v : s;
}
// ... and in 32 bits, to within 2^-20 of itself (a few roundings and math functions
// of a step or two each) or, where it underflows (exp does at 2^-126, and the root
// of that is 2^-63), 2^-62.
__device__ __forceinline__ float score32(int scoring, float v) {
  const float s = scoring == kSigmoid ? 1.0f / (1.0f + expf(-v)) : sqrtf(log1pf(expf(-fabsf(v))) + fmaxf(v, 0.0f));
  return v != v ? v : s;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int l) {
  return ((uint64_t)lane_value((uint32_t)(v >> 32), l) << 32) | lane_value((uint32_t)v, l);
}
__device__ __forceinline__ int permute(int to, int v) { return __builtin_amdgcn_ds_permute(4 * to, v); }
__device__ __forceinline__ float permute(int to, float v) {
  return __builtin_bit_cast(float, permute(to, __builtin_bit_cast(int, v)));
}

// A score on its way from its expert's lane to its slot: the bits of a double, or, for
// softmax, of the fp32 logit in the high half alone.
typedef uint64_t Score;
__device__ __forceinline__ Score pack(double s) { return __builtin_bit_cast(uint64_t, s); }
__device__ __forceinline__ Score pack(float z) { return (uint64_t)__builtin_bit_cast(uint32_t, z) << 32; }
__device__ __forceinline__ double score_of(Score s) { return __builtin_bit_cast(double, s); }
__device__ __forceinline__ float logit_of(Score s) { return __builtin_bit_cast(float, high(s)); }

// A number that at least n_used of the lanes' keys (or all that are not 0) reach.
__device__ __forceinline__ uint32_t border_of(uint32_t best, int n_used) {
  uint32_t top = 0;
  for (int count = 0; count < n_used;) {
    top = wave_max(best);
    if (top == 0) break;
    count += __popcll(__ballot(best == top));
    best = best == top ? 0u : best;
  }
  return top;
}

// Slots of the candidates, lanes `who` with a key, an expert and its score (softmax: its
// logit) each; of equal keys the lower lane is first.
template <typename K>
__device__ __forceinline__ void place(uint64_t who, K key, int expert, Score score, bool softmax, int n_used,
                                      int lane, int &id, Score &sc) {
  int before = 0;
  for (uint64_t left = who; left != 0; left &= left - 1) {
    const int c = __ffsll((unsigned long long)left) - 1;
    const K k = lane_value(key, c);
    before += k > key || (k == key && c < lane) ? 1 : 0;
  }
  // n_used is at most 32: the others go to lane 63, which is no slot.  Slots that
  // nobody sends to get zeros.
  const int to = ((who >> lane) & 1) && before < n_used ? before : 63;
  id = permute(to, expert + 1) - 1;
  sc = (uint64_t)(uint32_t)permute(to, (int)high(score)) << 32;
  if (!softmax) sc |= (uint32_t)permute(to, (int)(uint32_t)score);
  if (lane >= n_used) id = -1;
  if (id < 0) sc = 0;
}

// The candidates among EPL experts a lane, those with keys (or upper bounds of
// keys) of at least border, moved to lanes 0, 1, ... in the order of their ids.
// Returns how many; above 64 nothing is moved.
template <int EPL>
__device__ __forceinline__ int gather(const uint32_t (&key)[EPL], uint32_t border, const float (&z)[EPL],
                                      const float (&b)[EPL], int lane, float &zc, float &bc, int &ec) {
  int total = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) total += __popcll(__ballot(key[i] != 0 && key[i] >= border));
  if (total > 64) return total;
  int base = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool in = key[i] != 0 && key[i] >= border;
    const uint64_t who = __ballot(in);
    if (who == 0) continue;  // uniform
    const int n = __popcll(who);
    // The others send to a lane past these (or to lane 0 if there is none, which
    // then has its candidate or is one of these alone).
    const int to = in ? base + __popcll(who & ((1ull << lane) - 1)) : (base + n) & 63;
    const float zi = permute(to, z[i]), bi = permute(to, b[i]);
    const int ei = permute(to, i * 64 + lane);
    if (lane >= base && lane < base + n) {
      zc = zi;
      bc = bi;
      ec = ei;
    }
    base += n;
  }
  return total;
}

// An expert's key in 64 bits (0: not eligible), and its score (for softmax its logit).
__device__ __forceinline__ uint64_t key_of(const RouteArgs &a, float z, float b, Score &score) {
  score = pack(z);
  if (z == -__builtin_huge_valf()) return 0;
  if (a.scoring == kSoftmax) return (uint64_t)order32(z + b + 0.0f) << 32;
  const double s = score64(a.scoring, z);
  score = pack(s);
  return order64(s + (double)b + 0.0);
}

// Where more than 64 keys are equal or nearly equal: 64 experts at a time against
// the slots so far, n_used rounds of maximum each.  Few registers, and slow.
__device__ __forceinline__ void take_in_turn(const RouteArgs &a, int64_t t, int lane, int &id, Score &sc) {
  uint64_t kept = 0;  // lane j: the key of slot j
  id = -1;
  sc = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < a.n_expert; e0 += 64) {
    const int e = e0 + lane;
    Score score = 0;
    uint64_t next = 0;
    if (e < a.n_expert) next = key_of(a, a.logits[t * a.n_expert + e], a.bias ? a.bias[e] : 0.0f, score);
    uint64_t old = kept, add = next;
    int from = -1;  // + 64: one of the new ones, whose ids are above the slots'
    for (int j = 0; j < a.n_used; ++j) {
      const uint64_t best = old >= add ? old : add;
      const uint32_t top = wave_max(high(best));  // no eligible key has a zero there
      if (top == 0) break;
      const uint32_t low = wave_max(high(best) == top ? (uint32_t)best : 0u);
      const uint64_t key = ((uint64_t)top << 32) | low;
      const uint64_t slots = __ballot(old == key), fresh = __ballot(add == key);
      const int l = __ffsll((unsigned long long)(slots ? slots : fresh)) - 1;
      if (lane == j) from = slots ? l : 64 + l;
      if (lane == l) (slots ? old : add) = 0;
    }
    const int l = 4 * (from & 63);
    auto pick = [&](int was, int now) {
      const int w = __builtin_amdgcn_ds_bpermute(l, was), n = __builtin_amdgcn_ds_bpermute(l, now);
      return from < 0 ? 0 : from < 64 ? w : n;
    };
    auto pick64 = [&](uint64_t was, uint64_t now) {
      const uint32_t lo = (uint32_t)pick((int)(uint32_t)was, (int)(uint32_t)now);
      return (uint64_t)(uint32_t)pick((int)(was >> 32), (int)(now >> 32)) << 32 | lo;
    };
    id = pick(id + 1, e + 1) - 1;
    sc = pick64(sc, score);
    kept = pick64(kept, next);
  }
}

// The routing of token t: lane j < n_used gets slot j's expert and weight.
template <int EPL>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, int lane, int &id,
                                            float &weight) {
  const float inf = __builtin_huge_valf();
  const bool softmax = a.scoring == kSoftmax;
  float z[EPL], b[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    z[i] = e < a.n_expert ? a.logits[t * a.n_expert + e] : -inf;
    b[i] = a.bias && e < a.n_expert ? a.bias[e] : 0.0f;
  }
  // Keys, or bounds of them: best reaches no higher than the lane's largest, upper no
  // lower than each.
  uint32_t upper[EPL], best = 0;
  float total = 1.0f;
  Score slot, score = 0;
  uint64_t key = 0;  // one expert a lane is its own candidate
  if constexpr (EPL == 1) {
    key = key_of(a, z[0], b[0], score);
    best = upper[0] = high(key);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      upper[i] = 0;
      if (i * 64 < a.n_expert && z[i] != -inf) {
        float s = z[i], off = 0.0f;
        if (!softmax) {
          s = score32(a.scoring, s);
          off = 0x1p-19f * (s + fabsf(b[i])) + 0x1p-62f;
        }
        const float k = s + b[i];
        if (!(fabsf(k) < inf)) off = 0.0f;  // infinite and NaN keys are exact
        best = max(best, order32(k - off + 0.0f));
        upper[i] = order32(k + off + 0.0f);
      }
    }
  }
  const uint32_t border = border_of(best, a.n_used);
  if constexpr (EPL == 1) {
    place(__ballot(best != 0 && best >= border), key, lane, score, softmax, a.n_used, lane, id, slot);
  } else {
    float zc = -inf, bc = 0.0f;
    int ec = 0;
    const int n = gather<EPL>(upper, border, z, b, lane, zc, bc, ec);
    if (n <= 64) {
      key = key_of(a, zc, bc, score);
      place(n == 64 ? ~0ull : (1ull << n) - 1, key, ec, score, softmax, a.n_used, lane, id, slot);
    } else {
      take_in_turn(a, t, lane, id, slot);
    }
  }
  if (softmax) {
    const float sc = logit_of(slot);
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
    weight = (float)score_of(slot);
    if (a.renormalize) total = wave_sum(weight);
    if (a.renormalize && total < 0x1p-20f) {
      // fp32 may hold a few bits of these scores, or none (a sigmoid of -88, of -104).
      // Divided by the power of two of the largest first, they keep their weights.  From
      // 2^-20 on what a score below 2^-126 loses is below 2^-129 of the sum.
      const int top = (int)(wave_max(high(slot)) >> 20);
      weight = (float)ldexp(score_of(slot), 1023 - top);
      total = wave_sum(weight);
    }
  }
  // A NaN sum must reach the weights; an empty row's zero sum must not.
  weight = (total == 0.0f ? weight : weight / total) * a.scale;
}

}  // namespace mx
