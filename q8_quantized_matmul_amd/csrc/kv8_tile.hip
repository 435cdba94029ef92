// kv8_tile.hip -- attention for many query rows a key/value head (prompts, chunks of them, many
// heads on one): keys and values go through LDS as fp16 tiles that all waves multiply with.
//
// A workgroup takes 32 query rows a wave (tokens x the head's query heads) and a stretch of their
// keys, kKeys at a time (heads of 512: two waves share 32 rows, half of the dims each, and add
// their scores through LDS; a wave could not hold the sums and queries of 512 dims).  Codes come
// from HBM or L2 as int8, become fp16 once in the workgroup and lie in LDS in the order of the
// matrix operands, so that every operand is one conflict-free 16-byte read a lane.  Both products
// run on v_mfma_f32_32x32x16_f16, transposed (S^T = K Q^T, O^T = V^T P^T): a lane then holds 16 of
// 32 keys of one row, its weights become the second product's operand without leaving the lane, and
// a row's running bound and sum are one register each.
//
// The matrix core and the vector ALU have about equal work (of 64 keys and 32 rows of 128 values: 32
// instructions of 32 cycles; 32 exp2 and 200 others), so a wave does both at once: in step t it
// multiplies the keys of tile t + 1 while it turns the scores of tile t into weights, then the values of tile
// t while it scales the scores of t + 1 and puts the tiles that come next into LDS.  K is therefore staged
// a tile ahead of V; each has two buffers, and there is one barrier a step.
//
// Measured, causal, 32 heads of 128 on 8, bf16: 8192 tokens 560 to 610 us (900 to 980 TFLOP/s of the live half), 32768
// tokens 8.2 to 8.5 ms (1.0 PFLOP/s); torch's product of two fp16 matrices of 8192 reaches 1.17 on the same card.
// Both run at about 2.0 GHz.  512 tokens over 32768 keys, split in four, 284 to 300 us.  8192 tokens
// of heads of 64 404 to 441 us (640 TFLOP/s), of 192 1660 (495), of 256 1820 (600): those of 192 and 256 hold four waves
// and tiles of 32 keys.  On the way there (8192 tokens): weights, then products, tile by tile 806 us; page ids
// looked up a tile ahead of the codes, which nothing then waits for, 647; both at once 617.  Not taken, all within 5 %
// of it or slower: deeper operand reads, a fixed order of products and vector work with scores of two tiles in
// registers (their spills wait for the loads in flight), sums by dot products (they run on the matrix core), four
// waves instead of eight, wave priorities.
#include <atomic>

#include "kv8_attn.h"

namespace kv {
namespace {

// Scales of V this many powers of two below the largest are not folded into the exponent (put).
constexpr int kFoldBits = 8, kNoFold = -100000;

// The largest sum of a lane's weights of a tile: none is above fp16's 65504 then.
constexpr float kMostSum = 0x1p15f;

// In a branch that is hardly ever taken: what follows is not to be computed ahead of it.
__device__ __forceinline__ void rare() { asm volatile(""); }

// A lane's neighbour's value (0xb1), or that of the lane two on (0x4e), within four lanes.
template <int CTRL>
__device__ __forceinline__ int swapped(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, false);
}

template <int D, bool HALVES>
struct Shape {
  static constexpr int kKeys = D <= 128 ? 64 : 32;         // of a tile
  static constexpr int kWaves = D == 128 && !HALVES ? 8 : 4;
  static constexpr int kParts = D > 256 ? 2 : 1;           // waves that share 32 rows
  static constexpr int kDims = D / kParts;                 // dims of a wave
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRows = 32 * kWaves / kParts;
  static constexpr int kSubs = kKeys / 32;
  static constexpr int kGroups = kKeys / 16;               // of 16 keys, each under one scale
  static constexpr int kTile = kKeys * D;                  // fp16 values of a K or V tile
  static constexpr int kChunks = kKeys * D / 16;           // 16-byte pieces of codes of a K or V tile
  static constexpr int kPasses = (kChunks + kThreads - 1) / kThreads;
  static constexpr int kScaleWords = (4 * kGroups + 2 + 3) / 4 * 4;
  static constexpr int kMeet = kParts > 1 ? kWaves * 16 * 64 : 0;  // fp32 scores of the waves
  static constexpr int kLds = 2 * (2 * kTile * 2 + kScaleWords * 4) + kMeet * 4 + kRows * 4;
};

template <int D, bool HALVES>
__global__ __launch_bounds__((Shape<D, HALVES>::kThreads), (Shape<D, HALVES>::kWaves / 4)) void tile_kernel(
    Cache c, Batch b, Attention a, int splits, void *ws, int tiles) {
  using S = Shape<D, HALVES>;
  constexpr int kSteps = S::kDims / 16, kDimTiles = S::kDims / 32, kParts = S::kParts;
  constexpr int kSubs = S::kSubs, kGroups = S::kGroups, kPasses = S::kPasses;
  extern __shared__ __attribute__((aligned(16))) char lds[];  // S::kLds
  _Float16 *const kt = reinterpret_cast<_Float16 *>(lds);     // [2][kTile]
  _Float16 *const vt = kt + 2 * S::kTile;                     // [2][kTile]
  float *const scales = reinterpret_cast<float *>(vt + 2 * S::kTile);  // [2][kScaleWords], see put
  float *const meet = scales + 2 * S::kScaleWords;                     // [wave][16][64]
  int *const positions = reinterpret_cast<int *>(meet + S::kMeet);     // [kRows]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part_of = wave % kParts, dim0 = part_of * S::kDims;  // this wave's dims
  const int half = lane >> 5, col = lane & 31;
  // late tiles of a sequence have the most keys: they start first
  const int head = blockIdx.x % c.n_kv, w = tiles - 1 - blockIdx.x / c.n_kv, split = blockIdx.y;

  // the rows
  const Slots slots{S::kRows, a.group, 1};
  const int s = find_sequence(b, slots, w);
  const Span q = span_of(b, c, s);
  const int rows = q.n * a.group, r0 = (int)(w - slots.first(b, s)) * S::kRows;
  if (r0 < 0 || r0 >= rows) return;  // below 0: starts that do not ascend from 0
  const int wg_hi = q.first + (min(r0 + S::kRows, rows) - 1) / a.group, wg_lo = q.first + r0 / a.group;
  const int wr0 = r0 + 32 * (wave / kParts);
  const bool wave_ok = wr0 < rows;
  const int tok_hi = (min(wr0 + 32, rows) - 1) / a.group;
  const int row = wr0 + col, tok = min(row / a.group, tok_hi);
  const bool row_ok = row < rows;
  const int q_head = head * a.group + (row_ok ? row - tok * a.group : 0);
  // The row's position is wanted where masks are and at the end: until then it lies in LDS, each wave's own (a
  // register more, and heads of 128 spill).
  positions[wr0 - r0 + col] = row_ok ? q.first + tok : -1;
  auto position = [&] { return positions[wr0 - r0 + (threadIdx.x & 31)]; };
  const int pos_lo = q.first + wr0 / a.group, pos_hi = wave_ok ? q.first + tok_hi : -1;

  // the keys: n tiles from first_key on, counted from 0 below
  const int key0 = a.window ? max(wg_lo - a.window + 1, 0) & ~(S::kKeys - 1) : 0;
  const int key_end = wg_hi + 1;
  const int n_tiles = max(key_end - key0 + S::kKeys - 1, 0) / S::kKeys;
  const int per = (n_tiles + splits - 1) / splits;
  const int t_begin = split * per, n = min(n_tiles, t_begin + per) - t_begin;
  const int first_key = key0 + t_begin * S::kKeys;

  // query operands: lane (half, col) holds dims 16 i + 8 half + 0 .. 7 of the wave's dims of row col
  h8 qh[kSteps], ql[HALVES ? kSteps : 1];
  const int64_t q_at = (int64_t)(q.row0 + tok) * a.q.token_stride + (int64_t)q_head * a.q.head_stride + 8 * half;
  float factor = 0.f;
  auto load_queries = [&] {
    factor = by_type(a.q.type, [&](auto type) {
      Eight<type.value> x[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) x[i].load(a.q.p, q_at + dim0 + 16 * i, a.q.wide);
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) amax = max(amax, x[i].amax_bits());
      if constexpr (kParts > 1) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          Eight<type.value> other;
          other.load(a.q.p, q_at + (S::kDims - dim0) + 16 * i, a.q.wide);
          amax = max(amax, other.amax_bits());
        }
      }
      amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
      const RowScale rs(as<float>(amax), a.scale);
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = ldexp_fast(x[i].get(j), -rs.e);
          qh[i][j] = (_Float16)v;
          if constexpr (HALVES) ql[i][j] = (_Float16)(v - (float)qh[i][j]);
        }
      return rs.factor;
    });
  };

  // ---- staging ----
  // Piece ch of a tile's K (or V) codes: group ch / D of 16 keys, piece ch % D of its 16 * D bytes.
  // Keys behind the last one take its page, and tiles behind the last are fetched like others: no
  // row sees them, and nothing branches.
  const int32_t *const table = b.table + (int64_t)s * b.width;
  const int in_page = (1 << c.page_log) - 1;
  const int64_t page_bytes = (int64_t)(c.n_kv << c.page_log) * D, head_bytes = (int64_t)(head << c.page_log) * D;
  struct Pages {
    int of[kPasses], of_scale;  // as the table has them
  };
  auto look_up = [&](int t) {
    Pages r;
    const int key = first_key + t * S::kKeys;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) r.of[p] = table[min(key + 16 * ((tid + p * S::kThreads) / D), key_end - 1) >> c.page_log];
    r.of_scale = table[min(key + 16 * (lane % kGroups), key_end - 1) >> c.page_log];
    return r;
  };
  struct Codes {
    u32x4 of[kPasses];
  };
  auto fetch = [&](const int8_t *codes, int t, const Pages &pages) {
    Codes r;
    const int key = first_key + t * S::kKeys;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int ch = min(tid + p * S::kThreads, S::kChunks - 1);
      const int page = (uint32_t)pages.of[p] < (uint32_t)c.n_pages ? pages.of[p] : 0;  // its scales will be NaN
      const int at = ((key + 16 * (ch / D)) & in_page) * D + 16 * (ch % D);
      r.of[p] = *reinterpret_cast<const u32x4 *>(codes + (page * page_bytes + head_bytes) + at);
    }
    return r;
  };
  struct Scales {
    float k, v;
  };
  auto fetch_scales = [&](int t, const Pages &pages) {  // lane i: of group i % kGroups
    const bool ok = (uint32_t)pages.of_scale < (uint32_t)c.n_pages;
    const int64_t at = scale_offset(c, ok ? pages.of_scale : 0, head, first_key + t * S::kKeys + 16 * (lane % kGroups));
    Scales r{c.ks[at], c.vs[at]};
    if (!ok) r.k = r.v = as<float>(0x7fc00000u);
    return r;
  };
  auto put_k = [&](int t, const Codes &g) {
    _Float16 *const kb = kt + (t & 1) * S::kTile;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int ch = tid + p * S::kThreads, group = ch / D, piece = ch % D;
      if (S::kChunks % S::kThreads != 0 && ch >= S::kChunks) break;
      // 16 dims of one key -> operand (32 keys, 16 dims), halves of 8 dims
      _Float16 *kd = kb + ((group >> 1) * (D / 16) + (piece >> 4)) * 512 + (16 * (group & 1) + (piece & 15)) * 8;
      *reinterpret_cast<h8 *>(kd) = codes_f16(g.of[p][0], g.of[p][1]);
      *reinterpret_cast<h8 *>(kd + 256) = codes_f16(g.of[p][2], g.of[p][3]);
    }
  };
  auto put_v = [&](int t, const Codes &g) {
    _Float16 *const vb = vt + (t & 1) * S::kTile;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int ch = tid + p * S::kThreads, group = ch / D, piece = ch % D;
      if (S::kChunks % S::kThreads != 0 && ch >= S::kChunks) break;
      // 4 dims of 4 keys -> operand (32 dims, 16 keys) of this group.  Of the N dims of a wave, operand
      // row r holds dim 4 (r % (N / 4)) + r / (N / 4), so that the dims that adjacent lanes write at
      // once are adjacent rows
      const int quad = piece / (D / 4), d4 = piece % (D / 4);
      _Float16 *vd = vb + group * (D / 32) * 512 + (quad & 1) * 256 + (quad >> 1) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = d4 / (S::kDims / 4) * S::kDims + j * (S::kDims / 4) + d4 % (S::kDims / 4);
        *reinterpret_cast<h4 *>(vd + (r >> 5) * 512 + (r & 31) * 8) = codes_f16(g.of[p][j]);
      }
    }
  };
  // Of each group: K's scale; with E the largest exponent of the tile's scales of V, log2(V's / 2^E), which goes
  // into the weights' exponent, and 2^E / V's, by which a group's sum of weights is multiplied again: an
  // addition less for each weight than a product; V's itself, for rows that do not see every group.  Of the tile:
  // E, and the least exponent (kNoFold where a scale is zero, no number, or under 2^-8 of another: weights vanish
  // there that the rows' sums need).
  auto put_scales = [&](int t, const Scales &g) {
    if (wave != 0) return;
    const int i = lane % kGroups;
    const bool absent = first_key + t * S::kKeys + 16 * i >= key_end, number = g.v > 0.f && g.v < INFINITY;
    int most = number && !absent ? exponent_of(g.v) : kNoScale;
    int least = absent ? -kNoFold : number ? most : kNoFold;
#pragma unroll
    for (int j = 1; j < kGroups; j <<= 1) {  // among four lanes, or two
      most = max(most, j == 1 ? swapped<0xb1>(most) : swapped<0x4e>(most));
      least = min(least, j == 1 ? swapped<0xb1>(least) : swapped<0x4e>(least));
    }
    if (least < most - kFoldBits) least = kNoFold;
    const float v = absent ? 1.f : ldexp_fast(g.v, -most);
    float *const sc = scales + (t & 1) * S::kScaleWords;
    if (lane < kGroups) {
      sc[lane] = g.k;
      sc[kGroups + lane] = log2_fast(v);
      sc[2 * kGroups + lane] = absent ? 0.f : __builtin_amdgcn_rcpf(v);
      sc[3 * kGroups + lane] = g.v;
    }
    if (lane == 0) {
      int *const of_tile = reinterpret_cast<int *>(sc + 4 * kGroups);
      of_tile[0] = most;
      of_tile[1] = least;
    }
  };

  // ---- products ----
  f32x16 o[kDimTiles];
#pragma unroll
  for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  // (rows behind a sequence's last are given a bound that nothing reaches: without one they would take their wave into
  // the rare branch in every tile)
  float m = row_ok ? kLowest : -kLowest, l = 0.f;
  int e = kNoScale;
  auto scale_sums = [&](float f) {
#pragma unroll
    for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] *= f;
  };
  // products of the keys of tile t and this wave's rows (and dims)
  auto multiply_k = [&](int t, f32x16 (&z)[kSubs]) {
    const _Float16 *const kb = kt + (t & 1) * S::kTile + dim0 / 16 * 512 + lane * 8;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
      for (int j = 0; j < 16; ++j) z[sub][j] = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub) {
        const h8 k = *reinterpret_cast<const h8 *>(kb + (sub * (D / 16) + i) * 512);
        z[sub] = mfma32(k, qh[i], z[sub]);
        if constexpr (HALVES) z[sub] = mfma32(k, ql[i], z[sub]);
      }
  };
  // two waves' sums over their dims; every wave of the workgroup comes here
  auto meet_scores = [&](f32x16 (&z)[kSubs]) {
    if constexpr (kParts > 1) {
      static_assert(kSubs == 1 && kParts == 2, "memory for 16 scores a lane");
#pragma unroll
      for (int j = 0; j < 16; ++j) meet[(wave * 16 + j) * 64 + lane] = z[0][j];
      __syncthreads();
      // the sum of two is the same in either order: both waves have the same weights
#pragma unroll
      for (int j = 0; j < 16; ++j) z[0][j] += meet[((wave ^ 1) * 16 + j) * 64 + lane];
    }
  };
  // weights of tile t times its values
  auto multiply_v = [&](int t, const h8 (&ph)[kGroups], const h8 (&pl)[kGroups]) {
    const _Float16 *const vb = vt + (t & 1) * S::kTile + part_of * kDimTiles * 512 + lane * 8;
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
#pragma unroll
      for (int i = 0; i < kDimTiles; ++i) {
        const h8 v = *reinterpret_cast<const h8 *>(vb + (u * (D / 32) + i) * 512);
        o[i] = mfma32(v, ph[u], o[i]);
        if constexpr (HALVES) o[i] = mfma32(v, pl[u], o[i]);
      }
  };

  // A tile's scores on their way to weights: log2 of the weights times V's scale over 2^e, and what
  // a group's sum of them is multiplied with.
  float y[kSubs][16], share[kGroups];
  bool summed;  // by row: l has the tile's weights already, from its scores alone
  auto weights = [&](h8 (&ph)[kGroups], h8 (&pl)[kGroups], float &add) {
    float sum[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      float p[8];
      sum[u] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = exp2_fast(y[u >> 1][8 * (u & 1) + j]);
        sum[u] += p[j];
        ph[u][j] = (_Float16)p[j];
        if constexpr (HALVES) pl[u][j] = (_Float16)(p[j] - (float)ph[u][j]);
      }
    }
    float most = sum[0];
    add = sum[0] * share[0];
#pragma unroll
    for (int u = 1; u < kGroups; ++u) {
      most += sum[u];
      add = __builtin_fmaf(sum[u], share[u], add);
    }
    return most;
  };
  // Some row's weights are too large for fp16: its bound moves up to its largest score, the others' stay.
  auto raise = [&](float most) {
    const bool mine = fmaxf(most, __shfl_xor(most, 32)) > kMostSum;
    float top = y[0][0];
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, y[sub][j]);
    top = fmaxf(top, __shfl_xor(top, 32));
    const float by = mine ? fmaxf(top - kBias, 0.f) : 0.f;
    m += by;
    const float f = exp2_fast(-by);
    l *= f;
    scale_sums(f);
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
      for (int j = 0; j < 16; ++j) y[sub][j] -= by;
  };
  auto all_weights = [&](h8 (&ph)[kGroups], h8 (&pl)[kGroups]) {
    float add;
    const float most = weights(ph, pl, add);
    if (__any(most > kMostSum)) {
      rare();
      raise(most);
      weights(ph, pl, add);
    }
    l += summed ? 0.f : add;  // (add is NaN where a scale of V is)
  };
  // y of tile t from its products, before the rare cases below
  float fk[kGroups], lw[kGroups];
  int e_next, least;
  int e_low = kNoScale, e_high = kNoScale;  // of the wave's rows
  bool unset = true;                        // some row has no bound
  bool odd;                                 // y is not all (rare_cases)
  auto tile_scales = [&](int t) {
    const float *const sc = scales + (t & 1) * S::kScaleWords;
    const int *const of_tile = reinterpret_cast<const int *>(sc + 4 * kGroups);
    const int most = __builtin_amdgcn_readfirstlane(of_tile[0]);
    least = __builtin_amdgcn_readfirstlane(of_tile[1]);
    e_next = max(e, most);
    summed = false;
    odd = unset || most > e_low || least < e_high - kFoldBits;
    const float shift = (float)(most - e_next), back = ldexp_fast(1.f, e_next - most);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      fk[i] = sc[i] * factor;
      lw[i] = sc[kGroups + i] + shift;
      share[i] = sc[2 * kGroups + i] * back;
    }
  };
  auto scale_scores = [&](const f32x16 (&z)[kSubs]) {
    const float mb = m - kBias;
    float add[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) add[i] = lw[i] - mb;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
      for (int j = 0; j < 16; ++j) y[sub][j] = __builtin_fmaf(z[sub][j], fk[2 * sub + (j >> 3)], add[2 * sub + (j >> 3)]);
  };
  // What is not in every tile: keys that some row of the wave does not see, a scale of V above all that some row
  // has seen, a row's first keys (its bound is not set), scales that do not fold.  (One branch for all of them, on
  // scalars: a vote over the rows' exponents and bounds in every tile took 8192 tokens from 565 to 578 us.)
  auto rare_cases = [&](int t, const f32x16 (&z)[kSubs]) {
    const int key = first_key + t * S::kKeys;
    const float *const sc = scales + (t & 1) * S::kScaleWords;
    const bool ragged = key + S::kKeys - 1 > pos_lo || (a.window && key <= pos_hi - a.window);
    auto unseen = [&](int pos, int sub, int j) {
      const int at = key + 32 * sub + 8 * (j >> 2) + 4 * half + (j & 3);
      return at > pos || (a.window && at <= pos - a.window);
    };
    if (!ragged && !odd) return;
    rare();
    const int pos = position();
    int low = least;
    if (ragged) {
      // a row's exponents are those of the groups that it sees; the others may have any scale
      auto sees = [&](int i) { return key + 16 * i <= pos && !(a.window && key + 16 * i + 15 <= pos - a.window); };
      auto exponent = [&](float v) { return v > 0.f && v < INFINITY ? exponent_of(v) : kNoScale; };
      e_next = e;
      low = -kNoFold;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int at = exponent(sc[3 * kGroups + i]);
        e_next = sees(i) ? max(e_next, at) : e_next;
        low = sees(i) ? min(low, at == kNoScale ? kNoFold : at) : low;
      }
      asm volatile("" ::: "memory");  // (read again below: four registers less)
      const float mb = m - kBias;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int at = exponent(sc[3 * kGroups + i]);
        const float v = ldexp_fast(sc[3 * kGroups + i], -at);
        lw[i] = log2_fast(v) + (float)(at - e_next);
        share[i] = sees(i) ? ldexp_fast(__builtin_amdgcn_rcpf(v), e_next - at) : 0.f;
#pragma unroll
        for (int j = 8 * (i & 1); j < 8 * (i & 1) + 8; ++j)
          y[i >> 1][j] = unseen(pos, i >> 1, j) ? -INFINITY : __builtin_fmaf(z[i >> 1][j], fk[i], lw[i] - mb);
      }
    }
    if (__any(e_next > e)) {
      scale_sums(ldexp_fast(1.f, e - e_next));
      e = e_next;
    }
    summed = low < e - kFoldBits;
    const bool anew = summed || m == kLowest;
    if (__any(anew)) {
      float top = kLowest;
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          y[sub][j] = unseen(pos, sub, j) ? -INFINITY : z[sub][j] * fk[2 * sub + (j >> 3)];
          top = fmaxf(top, y[sub][j]);
        }
      top = fmaxf(top, __shfl_xor(top, 32));
      const float was = m;
      m = anew ? fmaxf(m, top) : m;
      const float f = exp2_fast(was - m);
      l *= f;
      scale_sums(f);
      const float mb = m - kBias;
      float sum = 0.f;
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          // x: for a row's largest score kBias to the bit, however large (one rounding, as in scale_scores, would
          // leave that score's last bits); rows with a bound keep what they had
          const float x = y[sub][j] - mb, as_was = __builtin_fmaf(z[sub][j], fk[2 * sub + (j >> 3)], lw[2 * sub + (j >> 3)] - mb);
          sum += exp2_fast(x);
          y[sub][j] = x == -INFINITY ? x : anew ? x + lw[2 * sub + (j >> 3)] : as_was;
        }
      l += summed ? sum : 0.f;
    }
    unset = __any(m == kLowest);
    e_low = e_high = __builtin_amdgcn_readfirstlane(e);
    while (const uint64_t below = __ballot(e < e_low)) e_low = __builtin_amdgcn_readlane(e, __builtin_ctzll(below));
    while (const uint64_t above = __ballot(e > e_high)) e_high = __builtin_amdgcn_readlane(e, __builtin_ctzll(above));
  };

  if (n > 0) {
    Codes k_next, v_next;
    Scales s_next;
    Pages pk, pv;
    if constexpr (D == 64) load_queries();  // (beside the fetches its scalar registers do not fit)
    {
      const Pages p0 = look_up(0), p1 = look_up(1);
      pv = look_up(2);
      pk = look_up(3);
      const Codes k0 = fetch(c.k, 0, p0), k1 = fetch(c.k, 1, p1), v0 = fetch(c.v, 0, p0);
      const Scales s0 = fetch_scales(0, p0), s1 = fetch_scales(1, p1);
      v_next = fetch(c.v, 1, p1);
      k_next = fetch(c.k, 2, pv);
      s_next = fetch_scales(2, pv);
      if constexpr (D != 64) load_queries();
      put_k(0, k0);
      put_scales(0, s0);
      put_k(1, k1);
      put_scales(1, s1);
      put_v(0, v0);
    }
    __syncthreads();
    auto stage = [&](int t) {  // beside tile t's values: the next tiles to LDS, others on their way
      put_k(t + 2, k_next);
      put_v(t + 1, v_next);
      put_scales(t + 2, s_next);
      k_next = fetch(c.k, t + 3, pk);
      v_next = fetch(c.v, t + 2, pv);
      s_next = fetch_scales(t + 3, pk);
      pv = pk;
      pk = look_up(t + 4);
    };
    f32x16 z[kSubs];
    multiply_k(0, z);
    meet_scores(z);
    tile_scales(0);
    scale_scores(z);
    rare_cases(0, z);
    __syncthreads();  // K's first buffer is free
    h8 ph[kGroups], pl[kGroups];
    for (int t = 0; t + 1 < n; ++t) {
      // K of t + 1, V of t and the scales of t + 1 are in LDS; K of t + 2, V of t + 1 in registers
      multiply_k(t + 1, z);
      all_weights(ph, pl);
      meet_scores(z);
      stage(t);
      multiply_v(t, ph, pl);
      tile_scales(t + 1);
      scale_scores(z);
      rare_cases(t + 1, z);
      __syncthreads();
    }
    all_weights(ph, pl);
    multiply_v(n - 1, ph, pl);
  }

  l += __shfl_xor(l, 32);
  // the row again: nothing of it but its position was kept
  const int out_row = wr0 + (threadIdx.x & 31), out_tok = position() - q.first;
  if (out_row >= rows) return;
  const int out_head = head * a.group + out_row - out_tok * a.group;
  const int64_t at = (int64_t)(q.row0 + out_tok) * a.n_q + out_head;
  const Finish fin(m, l, e, splits == 1 && a.sinks ? a.sinks[out_head] * kLog2e : -INFINITY);
  const Partials part(ws, b, c, a.n_q, splits);
  if (half == 0 && part_of == 0) {
    if (splits > 1)
      part.lse2[split * part.rows + at] = fin.lse2;
    else if (a.lse)
      a.lse[at] = fin.lse2 * kLn2;
  }
#pragma unroll
  for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = j * (S::kDims / 4) + 8 * i + k, r = d & 31;  // (operand row of the lanes' first half)
        v[j] = l == 0.f ? 0.f : o[d >> 5][4 * (r >> 3) + (r & 3)] * fin.factor;
      }
      const int dim = dim0 + 4 * (8 * i + 4 * half + k);
      if (splits > 1)
        store_values<kF32, 4>(part.out, (split * part.rows + at) * D + dim, v);
      else
        store_row<4>(a.out, a.out_type, at * D + dim, v);
    }
}

template <int D, bool HALVES>
hipError_t launch_dim(const Cache &c, const Batch &b, const Attention &a, int splits, void *ws, hipStream_t s) {
  using S = Shape<D, HALVES>;
  // More LDS than a launch may ask for by itself: allowed once on each device (twice does no harm).
  static std::atomic<uint64_t> allowed{0};
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(tile_kernel<D, HALVES>), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  const int tiles = (int)((int64_t)b.n_tok * a.group / S::kRows + b.n_seq);
  tile_kernel<D, HALVES><<<dim3((uint32_t)tiles * c.n_kv, (uint32_t)splits), S::kThreads, S::kLds, s>>>(c, b, a, splits, ws, tiles);
  return hipGetLastError();
}

}  // namespace

int tile_rows(int d, bool halves) {
  if (d > 256) return Shape<512, false>::kRows;
  return d == 128 && !halves ? Shape<128, false>::kRows : Shape<256, false>::kRows;
}

hipError_t launch_tile(const Cache &c, const Batch &b, const Attention &a, int splits, void *ws, hipStream_t s) {
  const bool halves = a.q.type == kF32 || a.out_type == kF32;
  switch (c.d) {
    case 64: return halves ? launch_dim<64, true>(c, b, a, splits, ws, s) : launch_dim<64, false>(c, b, a, splits, ws, s);
    case 128: return halves ? launch_dim<128, true>(c, b, a, splits, ws, s) : launch_dim<128, false>(c, b, a, splits, ws, s);
    case 192: return halves ? launch_dim<192, true>(c, b, a, splits, ws, s) : launch_dim<192, false>(c, b, a, splits, ws, s);
    case 256: return halves ? launch_dim<256, true>(c, b, a, splits, ws, s) : launch_dim<256, false>(c, b, a, splits, ws, s);
    default: return halves ? hipErrorInvalidValue : launch_dim<512, false>(c, b, a, splits, ws, s);  // attention_plan
  }
}

}  // namespace kv
