// kv8_tile.hip -- attention for many query rows a key/value head (prompts, chunks of them, many
// heads on one): keys and values go through LDS as fp16 tiles that all waves multiply with.
//
// A workgroup takes 32 query rows a wave (tokens x the head's query heads) and a stretch of their
// keys, kKeys at a time (heads of 512: two waves share 32 rows, half of the dims each, and add
// their scores through LDS; a wave could not hold the sums and queries of 512 dims).  Codes come from HBM or L2 as int8, become fp16 once in the workgroup
// and lie in LDS in the order of the matrix operands, so that every operand is one conflict-free
// 16-byte read a lane.  Both products run on v_mfma_f32_32x32x16_f16, transposed (S^T = K Q^T,
// O^T = V^T P^T): a lane then holds 16 of 32 keys of one row, its weights become the second product's
// operand without leaving the lane, and a row's running bound and sum are one register each.
// Two LDS buffers and one barrier a tile: while the waves multiply tile t, tile t + 1 is written to
// the other buffer from registers and tile t + 2 is on its way from memory.
#include "kv8_attn.h"

namespace kv {
namespace {

// Keys of a tile, waves of a workgroup.
template <int D>
struct Shape {
  static constexpr int kKeys = D <= 128 ? 64 : 32;
  static constexpr int kWaves = 4;
  static constexpr int kParts = D > 256 ? 2 : 1;           // waves that share 32 rows
  static constexpr int kDims = D / kParts;                 // dims of a wave
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRows = 32 * kWaves / kParts;
  static constexpr int kGroups = kKeys / 16;               // of 16 keys, each under one scale
  static constexpr int kTile = kKeys * D;                  // fp16 values of a K or V tile
  static constexpr int kChunks = kKeys * D / 16;           // 16-byte pieces of codes of a K or V tile
  static constexpr int kPasses = (kChunks + kThreads - 1) / kThreads;
  static constexpr int kMeet = kParts > 1 ? kWaves * 16 * 64 : 0;  // fp32 scores of the waves
  static constexpr int kLds = 2 * (2 * kTile * 2 + 2 * kGroups * 4) + kMeet * 4;
};

// What a thread carries of a tile on its way: codes, and one of its scales.
template <int D>
struct Staged {
  u32x4 k[Shape<D>::kPasses], v[Shape<D>::kPasses];
  float scale;
};

template <int D, bool HALVES>
__global__ __launch_bounds__(Shape<D>::kThreads, D <= 128 && !HALVES ? 2 : 1) void tile_kernel(
    Cache c, Batch b, Attention a, int splits, void *ws, int tiles) {
  using S = Shape<D>;
  constexpr int kSteps = S::kDims / 16, kDimTiles = S::kDims / 32, kParts = S::kParts;
  extern __shared__ __align__(16) char lds[];
  _Float16 *const kt = reinterpret_cast<_Float16 *>(lds);     // [2][kTile]
  _Float16 *const vt = kt + 2 * S::kTile;                     // [2][kTile]
  float *const scales = reinterpret_cast<float *>(vt + 2 * S::kTile);  // [2][k, v][kGroups]
  float *const meet = scales + 4 * S::kGroups;                         // [wave][16][64]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int part_of = wave % kParts, dim0 = part_of * S::kDims;  // this wave's dims
  const int half = lane >> 5, col = lane & 31;
  // late tiles of a sequence have the most keys: they start first
  const int head = blockIdx.x % c.n_kv, w = tiles - 1 - blockIdx.x / c.n_kv, split = blockIdx.y;

  // the rows
  const Slots slots{S::kRows, a.group, 1};
  const int s = find_sequence(b, slots, w);
  const Span q = span_of(b, c, s);
  const int rows = q.n * a.group, r0 = (int)(w - slots.first(b, s)) * S::kRows;
  if (r0 >= rows) return;
  const int wg_hi = q.first + (min(r0 + S::kRows, rows) - 1) / a.group, wg_lo = q.first + r0 / a.group;
  const int wr0 = r0 + 32 * (wave / kParts);
  const bool wave_ok = wr0 < rows;
  const int tok_hi = (min(wr0 + 32, rows) - 1) / a.group;
  const int row = wr0 + col, tok = min(row / a.group, tok_hi);
  const bool row_ok = row < rows;
  const int q_head = head * a.group + (row_ok ? row - tok * a.group : 0);
  const int pos = row_ok ? q.first + tok : -1;
  const int pos_lo = q.first + wr0 / a.group, pos_hi = wave_ok ? q.first + tok_hi : -1;

  // the keys: tiles [t_begin, t_end) from key0 on
  const int key0 = a.window ? max(wg_lo - a.window + 1, 0) & ~(S::kKeys - 1) : 0;
  const int key_end = wg_hi + 1;
  const int n_tiles = max(key_end - key0 + S::kKeys - 1, 0) / S::kKeys;
  const int per = (n_tiles + splits - 1) / splits;
  const int t_begin = split * per, t_end = min(n_tiles, t_begin + per);

  // query operands: lane (half, col) holds dims 16 i + 8 half + 0 .. 7 of the wave's dims of row col
  h8 qh[kSteps], ql[HALVES ? kSteps : 1];
  const int64_t q_at = (int64_t)(q.row0 + tok) * a.q.token_stride + (int64_t)q_head * a.q.head_stride + 8 * half;
  const float factor = by_type(a.q.type, [&](auto type) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      float v[8];
      load_values<type.value, 8>(a.q.p, q_at + 16 * i, a.q.wide, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, as<uint32_t>(v[j]) & 0x7fffffffu);
    }
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
    const RowScale rs(as<float>(amax), a.scale);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      float v[8];
      load_values<type.value, 8>(a.q.p, q_at + dim0 + 16 * i, a.q.wide, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = ldexp_fast(v[j], -rs.e);
        qh[i][j] = (_Float16)x;
        if constexpr (HALVES) ql[i][j] = (_Float16)(x - (float)qh[i][j]);
      }
    }
    return rs.factor;
  });

  // ---- staging ----
  // piece ch of a tile's K (or V) codes: group ch / D of 16 keys, piece ch % D of its 16 * D bytes
  int pages[2][S::kPasses];  // of this thread's pieces, two tiles ahead; -1: none
  int scale_page[2];
  const int scale_group = tid % S::kGroups;
  const bool scale_mine = tid < 2 * S::kGroups, scale_is_v = tid >= S::kGroups;
  auto look_up = [&](int t, int slot) {
    const int key = key0 + t * S::kKeys;
#pragma unroll
    for (int p = 0; p < S::kPasses; ++p) {
      const int k16 = key + 16 * ((tid + p * S::kThreads) / D);
      pages[slot][p] = t < t_end && k16 < key_end ? page_of(c, b, s, k16) : -1;
    }
    const int k16 = key + 16 * scale_group;
    scale_page[slot] = scale_mine && t < t_end && k16 < key_end ? page_of(c, b, s, k16) : -1;
  };
  auto fetch = [&](int t, int slot, Staged<D> &g) {
    const int key = key0 + t * S::kKeys;
#pragma unroll
    for (int p = 0; p < S::kPasses; ++p) {
      const int ch = tid + p * S::kThreads;
      g.k[p] = g.v[p] = u32x4{0, 0, 0, 0};
      if (pages[slot][p] >= 0 && (S::kChunks % S::kThreads == 0 || ch < S::kChunks)) {
        const int64_t at = code_offset(c, pages[slot][p], head, key + 16 * (ch / D)) + 16 * (ch % D);
        g.k[p] = *reinterpret_cast<const u32x4 *>(c.k + at);
        g.v[p] = *reinterpret_cast<const u32x4 *>(c.v + at);
      }
    }
    g.scale = as<float>(0x7fc00000u);  // keys without a page: NaN where a row sees them
    if (scale_page[slot] >= 0) g.scale = (scale_is_v ? c.vs : c.ks)[scale_offset(c, scale_page[slot], head, key + 16 * scale_group)];
  };
  auto put = [&](int buf, const Staged<D> &g) {
    _Float16 *const kb = kt + buf * S::kTile, *const vb = vt + buf * S::kTile;
#pragma unroll
    for (int p = 0; p < S::kPasses; ++p) {
      const int ch = tid + p * S::kThreads, group = ch / D, piece = ch % D;
      if (S::kChunks % S::kThreads != 0 && ch >= S::kChunks) break;
      // K: 16 dims of one key -> operand (32 keys, 16 dims), halves of 8 dims
      _Float16 *kd = kb + ((group >> 1) * (D / 16) + (piece >> 4)) * 512 + (16 * (group & 1) + (piece & 15)) * 8;
      *reinterpret_cast<h8 *>(kd) = codes_f16(g.k[p][0], g.k[p][1]);
      *reinterpret_cast<h8 *>(kd + 256) = codes_f16(g.k[p][2], g.k[p][3]);
      // V: 4 dims of 4 keys -> operand (32 dims, 16 keys) of this group.  Of the N dims of a wave,
      // operand row n holds dim 4 (n % (N / 4)) + n / (N / 4), so that the dims that adjacent lanes
      // write at once are adjacent rows
      const int quad = piece / (D / 4), d4 = piece % (D / 4);
      _Float16 *vd = vb + group * (D / 32) * 512 + (quad & 1) * 256 + (quad >> 1) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = d4 / (S::kDims / 4) * S::kDims + j * (S::kDims / 4) + d4 % (S::kDims / 4);
        *reinterpret_cast<h4 *>(vd + (n >> 5) * 512 + (n & 31) * 8) = codes_f16(g.v[p][j]);
      }
    }
    if (scale_mine) scales[(buf * 2 + scale_is_v) * S::kGroups + scale_group] = g.scale;
  };

  f32x16 o[kDimTiles];
#pragma unroll
  for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  float m = kLowest, l = 0.f;
  int e = kNoScale;

  Staged<D> g;
  look_up(t_begin, 0);
  look_up(t_begin + 1, 1);
  fetch(t_begin, 0, g);
  if (t_begin < t_end) put(0, g);
  fetch(t_begin + 1, 1, g);
  look_up(t_begin + 2, 0);
  __syncthreads();

  for (int t = t_begin; t < t_end; ++t) {
    const int buf = (t - t_begin) & 1;
    if (t + 1 < t_end) {
      put(buf ^ 1, g);
      fetch(t + 2, 0, g);
      look_up(t + 3, 0);
    }
    const int tile_key = key0 + t * S::kKeys;
#pragma unroll
    for (int sub = 0; sub < S::kKeys / 32; ++sub) {
      const int key = tile_key + 32 * sub;
      const bool seen = key <= pos_hi && !(a.window && key + 31 <= pos_lo - a.window);  // by a row of this wave
      if (kParts == 1 && !seen) continue;
      const _Float16 *const kb = kt + buf * S::kTile + (sub * (D / 16) + dim0 / 16) * 512 + lane * 8;
      f32x16 z;
#pragma unroll
      for (int j = 0; j < 16; ++j) z[j] = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const h8 k = *reinterpret_cast<const h8 *>(kb + i * 512);
        z = mfma32(k, qh[i], z);
        if constexpr (HALVES) z = mfma32(k, ql[i], z);
      }
      if constexpr (kParts > 1) {  // one tile a step, so the barrier behind it also frees this memory
        static_assert(S::kKeys == 32 && kParts == 2, "");
#pragma unroll
        for (int j = 0; j < 16; ++j) meet[(wave * 16 + j) * 64 + lane] = z[j];
        __syncthreads();
        // both waves add in the same order: their weights are the same bits
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = meet[((wave ^ 1) * 16 + j) * 64 + lane];
          z[j] = z[j] + x;
        }
        if (!seen) continue;
      }
      const float *const sc = scales + buf * 2 * S::kGroups + 2 * sub;
      const float f0 = sc[0] * factor, f1 = sc[1] * factor;
      const float v0 = sc[S::kGroups], v1 = sc[S::kGroups + 1];
      const bool ragged = key + 31 > pos_lo || (a.window && key <= pos_hi - a.window);
      float y[16];
      auto weigh = [&](float mb) {  // log2 of the weights under bound mb: scores under 0
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = __builtin_fmaf(z[j], j < 8 ? f0 : f1, -mb);
        if (ragged) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int at = key + 8 * (j >> 2) + 4 * half + (j & 3);
            if (at > pos || (a.window && at <= pos - a.window)) y[j] = -INFINITY;
          }
        }
      };
      auto largest = [&] {
        float top = fmaxf(y[0], y[1]);
#pragma unroll
        for (int j = 2; j < 16; j += 2) top = fmaxf(fmaxf(top, y[j]), y[j + 1]);
        return top;
      };
      weigh(m - kBias);
      if (__any(largest() > kSlack + kBias)) {
        weigh(0.f);
        float top = largest();
        top = fmaxf(top, __shfl_xor(top, 32));
        const float was = m;
        m = fmaxf(m, top);
        const float f = exp2_fast(was - m);
        l *= f;
#pragma unroll
        for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[i][j] *= f;
        // from the rounded scores, as the bound is: scores of 2^28 have no other that is below it
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] -= m - kBias;
      }
      int e2 = kNoScale;
      if (v0 != 0.f && key <= pos_hi) e2 = exponent_of(v0);
      if (v1 != 0.f && key + 16 <= pos_hi) e2 = max(e2, exponent_of(v1));
      e2 = __builtin_amdgcn_readfirstlane(e2);
      if (e2 > e) {
        const float f = ldexp_fast(1.f, e - e2);
        e = e2;
#pragma unroll
        for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[i][j] *= f;
      }
      const float w0 = ldexp_fast(v0, -e), w1 = ldexp_fast(v1, -e);
      h8 ph[2], pl[2];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float p = exp2_fast(y[j]);
        l += p;
        float x = p * (j < 8 ? w0 : w1);
        if (ragged && y[j] == -INFINITY) x = 0.f;  // also where the scale is not finite
        ph[j >> 3][j & 7] = (_Float16)x;
        if constexpr (HALVES) pl[j >> 3][j & 7] = (_Float16)(x - (float)ph[j >> 3][j & 7]);
      }
      const _Float16 *const vb = vt + buf * S::kTile + (2 * sub * (D / 32) + part_of * kDimTiles) * 512 + lane * 8;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < kDimTiles; ++i) {
          const h8 v = *reinterpret_cast<const h8 *>(vb + (u * (D / 32) + i) * 512);
          o[i] = mfma32(v, ph[u], o[i]);
          if constexpr (HALVES) o[i] = mfma32(v, pl[u], o[i]);
        }
    }
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (!row_ok) return;
  const int64_t at = (int64_t)(q.row0 + tok) * a.n_q + q_head;
  const Finish fin(m, l, e, splits == 1 && a.sinks ? a.sinks[q_head] * kLog2e : -INFINITY);
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
        const int n = j * (S::kDims / 4) + 8 * i + k, r = n & 31;  // (operand row of the lanes' first half)
        v[j] = l == 0.f ? 0.f : o[n >> 5][4 * (r >> 3) + (r & 3)] * fin.factor;
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
  using S = Shape<D>;
  static const hipError_t ready = hipFuncSetAttribute(reinterpret_cast<const void *>(tile_kernel<D, HALVES>),
                                                      hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
  if (ready != hipSuccess) return ready;
  const int tiles = (int)((int64_t)b.n_tok * a.group / S::kRows + b.n_seq);
  tile_kernel<D, HALVES><<<dim3((uint32_t)tiles * c.n_kv, (uint32_t)splits), S::kThreads, S::kLds, s>>>(c, b, a, splits, ws, tiles);
  return hipGetLastError();
}

}  // namespace

int tile_rows(int d) { return d > 256 ? Shape<512>::kRows : Shape<256>::kRows; }

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
