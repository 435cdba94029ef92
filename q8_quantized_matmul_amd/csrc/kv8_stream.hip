// kv8_stream.hip -- attention for few query rows a key/value head (single tokens, drafts):
// the cache streams through, straight from HBM into matrix operands.
//
// A workgroup takes 16 query rows that share a key/value head (tokens x the head's query heads) and
// a stretch of their keys; its four waves take 32 keys each in turn and meet at the end.  Per
// step a wave multiplies 32 keys by its 16 rows, S^T = K Q^T, on v_mfma_f32_16x16x32_f16:
// transposed, so that a lane's results are 4 + 4 keys of one row, which is how the second
// product, O^T = V^T P^T, takes its weights: they never leave the lane.  The codes of 16 keys lie as
// that instruction's operand takes them, so every load of a wave is 1024 adjacent bytes (K) or
// four runs of 256 (V) and there is no LDS in the loop.
// What bounds it is HBM: 2 * d bytes a key, 160 VALU instructions a lane for the codes of 32 keys
// of 128 values (8 KB) beside 16 matrix instructions.  Measured, 32 heads of 128 on 8: 64 sequences of up to
// 8192 tokens (667 MB) 133 us, 5.0 TB/s, a copy of 1 GiB reaching 5.1; one of 131072 (269 MB) 57 us and 5
// for the join; one of 2000 6.4 us and 4 to 5.  64 heads of 512 on one, 12 sequences of up to 6000: 52 us, where
// each of the four tiles of 16 rows loads and converts the codes again (178 MB for 45) and, at one wave a SIMD, waits for
// its loads with nothing else to do: the vector ALU is busy for 26 %.  Not taken: the next step's codes fetched
// behind this step's products (8 % slower for 131072 tokens: fewer waves fit); two tiles of rows a wave,
// two waves sharing the dims of a head of 512 (10 % faster there, elsewhere slower).
#include "kv8_attn.h"

namespace kv {
namespace {

constexpr int kRows = 16, kStep = 32, kWaves = 4;

template <int D, bool HALVES>
__global__ __launch_bounds__(256) void stream_kernel(Cache c, Batch b, Attention a, int splits, void *ws) {
  constexpr int kChunks = D / 64;
  __shared__ float join_o[kWaves][64][kRows + 1];
  __shared__ float join_m[kWaves][kRows], join_l[kWaves][kRows];
  __shared__ int join_e[kWaves][kRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, col = lane & 15;
  const int head = blockIdx.x % c.n_kv, w = blockIdx.x / c.n_kv, split = blockIdx.y;

  // the rows
  int s = w, tile = 0;
  if ((int64_t)b.max_new * a.group > kRows) {
    const Slots slots{kRows, a.group, 1};
    s = find_sequence(b, slots, w);
    tile = (int)(w - slots.first(b, s));
  }
  const Span q = span_of(b, c, s);
  const int rows = q.n * a.group, r0 = tile * kRows;
  if (r0 < 0 || r0 >= rows) return;  // below 0: starts that do not ascend from 0
  const int tok_hi = (min(r0 + kRows, rows) - 1) / a.group;
  const int row = r0 + col, tok = min(row / a.group, tok_hi);
  const bool row_ok = row < rows;
  const int q_head = head * a.group + (row_ok ? row - tok * a.group : 0);
  const int pos = row_ok ? q.first + tok : -1;
  const int pos_lo = q.first + r0 / a.group, pos_hi = q.first + tok_hi;

  // the keys: steps [st, st_end) of 32 from key0 on
  const int key0 = a.window ? max(pos_lo - a.window + 1, 0) & ~(kStep - 1) : 0;
  const int key_end = pos_hi + 1;
  const int steps = max(key_end - key0 + kStep - 1, 0) / kStep;
  const int per = ((steps + splits - 1) / splits + kWaves - 1) / kWaves * kWaves;  // whole turns of the waves
  const int st_end = min(steps, (split + 1) * per);
  const int st_begin = split * per + wave;

  // query operands: lane (g, col) holds dims 64 c + 16 g + 0 .. 15 of row col, as K's 16-dim chunks lie
  h8 qh[2 * kChunks], ql[HALVES ? 2 * kChunks : 1];
  float factor;
  {
    float v[kChunks][16], amax = 0.f;
    const int64_t at = (int64_t)(q.row0 + tok) * a.q.token_stride + (int64_t)q_head * a.q.head_stride + 16 * g;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      load_row<16>(a.q, at + 64 * i, v[i]);
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = as<float>(max(as<uint32_t>(amax), as<uint32_t>(v[i][j]) & 0x7fffffffu));
    }
    amax = as<float>(max(as<uint32_t>(amax), (uint32_t)__shfl_xor(as<int>(amax), 16)));
    amax = as<float>(max(as<uint32_t>(amax), (uint32_t)__shfl_xor(as<int>(amax), 32)));
    const RowScale rs(amax, a.scale);
    factor = rs.factor;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float x = ldexp_fast(v[i][j], -rs.e);
        const _Float16 hi = (_Float16)x;
        qh[2 * i + (j >> 3)][j & 7] = hi;
        if constexpr (HALVES) ql[2 * i + (j >> 3)][j & 7] = (_Float16)(x - (float)hi);
      }
  }

  f32x4 o[4 * kChunks];
#pragma unroll
  for (int i = 0; i < 4 * kChunks; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kLowest, l = 0.f;
  int e = kNoScale;

  for (int chunk = st_begin; chunk < st_end; chunk += 32 * kWaves) {
    // pages and scales of this wave's next 32 steps: lane i looks up 16 keys, step i / 2, half i & 1
    int page = 0, exponent = kNoScale;
    float ks = 0.f, vs = 0.f;
    {
      const int st = chunk + (lane >> 1) * kWaves;
      const int key = key0 + st * kStep + 16 * (lane & 1);
      if (st < st_end && key < key_end) {
        page = page_of(c, b, s, key);
        if (page >= 0) {
          const int64_t at = scale_offset(c, page, head, key);
          ks = c.ks[at];
          vs = c.vs[at];
          if (vs != 0.f) exponent = exponent_of(vs);
        } else {
          page = 0;
          ks = vs = as<float>(0x7fc00000u);
        }
      }
    }
    const int n = min((st_end - chunk + kWaves - 1) / kWaves, 32);
    for (int t = 0; t < n; ++t) {
      const int key = key0 + (chunk + t * kWaves) * kStep;
      u32x4 kc[2][kChunks], vc[2][kChunks];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = code_offset(c, __builtin_amdgcn_readlane(page, 2 * t + h), head, key + 16 * h);
        const int8_t *kp = c.k + at + 16 * lane, *vp = c.v + at + g * 4 * D + 16 * col;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          kc[h][i] = *reinterpret_cast<const u32x4 *>(kp + 1024 * i);
          vc[h][i] = *reinterpret_cast<const u32x4 *>(vp + 256 * i);
        }
      }
      float x[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const h8 k0 = codes_f16(kc[h][i][0], kc[h][i][1]), k1 = codes_f16(kc[h][i][2], kc[h][i][3]);
          z = mfma16(k0, qh[2 * i], z);
          z = mfma16(k1, qh[2 * i + 1], z);
          if constexpr (HALVES) {
            z = mfma16(k0, ql[2 * i], z);
            z = mfma16(k1, ql[2 * i + 1], z);
          }
        }
        const float f = as<float>(__builtin_amdgcn_readlane(as<int>(ks), 2 * t + h)) * factor;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[h][i] = z[i] * f;
      }
      // keys that not every row sees
      const bool ragged = key + kStep - 1 > pos_lo || (a.window && key <= pos_hi - a.window);
      if (ragged) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = key + 16 * h + 4 * g + i;
            if (j > pos || (a.window && j <= pos - a.window)) x[h][i] = -INFINITY;
          }
      }
      float top = x[0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i >> 2][i & 3]);
      if (__any(top > m + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float was = m;
        m = top > m + kSlack ? top : m;  // by row: no other row's keys move its bound
        const float f = exp2_fast(was - m);
        l *= f;
#pragma unroll
        for (int i = 0; i < 4 * kChunks; ++i) o[i] *= f;
      }
      int e2 = max(__builtin_amdgcn_readlane(exponent, 2 * t), __builtin_amdgcn_readlane(exponent, 2 * t + 1));
      if (ragged) {  // by row: of the 16 keys that it sees one of
        e2 = kNoScale;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = key + 16 * h;
          if (j <= pos && (!a.window || j + 15 > pos - a.window)) e2 = max(e2, __builtin_amdgcn_readlane(exponent, 2 * t + h));
        }
      }
      if (__any(e2 > e)) {
        e2 = max(e, e2);
        const float f = ldexp_fast(1.f, e - e2);
        e = e2;
#pragma unroll
        for (int i = 0; i < 4 * kChunks; ++i) o[i] *= f;
      }
      h8 ph, pl;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float v = ldexp_fast(as<float>(__builtin_amdgcn_readlane(as<int>(vs), 2 * t + h)), -e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = exp2_fast(x[h][i] - (m - kBias));
          l += p;
          float y = p * v;
          if (ragged && x[h][i] == -INFINITY) y = 0.f;  // also where v is not finite
          ph[4 * h + i] = (_Float16)y;
          if constexpr (HALVES) pl[4 * h + i] = (_Float16)(y - (float)ph[4 * h + i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4 * kChunks; ++i) {
        const h8 v = codes_f16(vc[0][i >> 2][i & 3], vc[1][i >> 2][i & 3]);
        o[i] = mfma16(v, ph, o[i]);
        if constexpr (HALVES) o[i] = mfma16(v, pl, o[i]);
      }
    }
  }

  // the four waves' sums, 64 dims at a time; a thread takes 4 dims of one row
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    join_m[wave][col] = m;
    join_l[wave][col] = l;
    join_e[wave][col] = e;
  }
  __syncthreads();
  const int jr = threadIdx.x >> 4, jd = (threadIdx.x & 15) * 4;
  float jm = kLowest, jl = 0.f, jf[kWaves];
  int je = kNoScale;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    jm = fmaxf(jm, join_m[i][jr]);
    je = max(je, join_e[i][jr]);
  }
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const float f = exp2_fast(join_m[i][jr] - jm);
    jl += join_l[i][jr] * f;
    jf[i] = ldexp_fast(f, join_e[i][jr] - je);
  }
  const int j_row = r0 + jr, j_tok = j_row / a.group, j_head = head * a.group + j_row % a.group;
  const bool j_ok = j_row < rows;
  const int64_t j_at = (int64_t)(q.row0 + j_tok) * a.n_q + j_head;  // row of the outputs
  const float sink2 = splits == 1 && a.sinks && j_ok ? a.sinks[j_head] * kLog2e : -INFINITY;
  const Finish fin(jm, jl, je, sink2);
  const Partials part(ws, b, c, a.n_q, splits);
  if (j_ok && jd == 0) {
    if (splits > 1)
      part.lse2[split * part.rows + j_at] = fin.lse2;
    else if (a.lse)
      a.lse[j_at] = fin.lse2 * kLn2;
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) join_o[wave][16 * g + 4 * k + j][col] = o[4 * i + j][k];
    __syncthreads();
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) sum += join_o[k][jd + j][jr] * jf[k];
      v[j] = jl == 0.f ? 0.f : sum * fin.factor;
    }
    if (j_ok) {
      if (splits > 1)
        store_values<kF32, 4>(part.out, (split * part.rows + j_at) * D + 64 * i + jd, v);
      else
        store_row<4>(a.out, a.out_type, j_at * D + 64 * i + jd, v);
    }
  }
}

// out[row] = sum over splits of out_s * exp2(lse2_s) / (their sum, and the sink's).  A thread takes 4 dims.  Up to
// kFewSplits a workgroup takes as many rows as fit, a thread all splits of its row; above, one row, of which a thread
// has every n-th split (what bounds it is latency: a row's loads are on their way together), and the n
// sums are added in order.  Every split has written every row (zeros where it has no key of it), so weights that
// vanish multiply too: a row that sees a NaN keeps it.
constexpr int kMostSplits = 256, kFewSplits = 8;
__global__ __launch_bounds__(256) void join_kernel(Cache c, Batch b, Attention a, int splits, const void *ws) {
  __shared__ float weight[kMostSplits], wave_top[4], wave_sum[4];
  __shared__ f32x4 sums[256];
  const Partials part(const_cast<void *>(ws), b, c, a.n_q, splits);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lanes = c.d / 4, groups = 256 / lanes, group = tid / lanes, at = tid % lanes * 4;
  const bool few = splits <= kFewSplits;
  const int64_t row = few ? (int64_t)blockIdx.x * groups + group : blockIdx.x;
  const int tok = (int)(row / a.n_q), head = (int)(row - (int64_t)tok * a.n_q);
  bool mine = group < groups && row < part.rows && tok >= start_of(b, 0) && tok < (b.starts ? start_of(b, b.n_seq) : b.n_seq);
  if (!few && !__any(mine)) return;  // one row: the same for all
  const float *const x = part.out + row * c.d + at;
  const int64_t stride = part.rows * c.d;
  float top = -INFINITY, sum = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (few) {
    if (!mine) return;
    float z[kFewSplits];
    f32x4 y[kFewSplits];
#pragma unroll
    for (int s = 0; s < kFewSplits; ++s) {
      z[s] = s < splits ? part.lse2[s * part.rows + row] : -INFINITY;
      if (s < splits) y[s] = *reinterpret_cast<const f32x4 *>(x + s * stride);
      top = fmaxf(top, z[s]);
    }
#pragma unroll
    for (int s = 0; s < kFewSplits; ++s) {
      const float w = z[s] == -INFINITY ? 0.f : exp2_fast(z[s] - top);
      sum += w;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += s < splits ? y[s][j] * w : 0.f;
    }
  } else {
    const float z = tid < splits ? part.lse2[tid * part.rows + row] : -INFINITY;
    top = z;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
    if (lane == 0) wave_top[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
    const float w = z == -INFINITY ? 0.f : exp2_fast(z - top);
    weight[tid] = w;
    sum = w;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) sum += __shfl_xor(sum, i);
    if (lane == 0) wave_sum[wave] = sum;
    __syncthreads();
    sum = (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]);
    if (group < groups) {
#pragma unroll 8
      for (int s = group; s < splits; s += groups) {
        const float f = weight[s];
        const f32x4 y = *reinterpret_cast<const f32x4 *>(x + s * stride);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += y[j] * f;
      }
    }
    sums[tid] = v;
    __syncthreads();
    if (group != 0) return;
    for (int i = 1; i < groups; ++i) {
      const f32x4 y = sums[i * lanes + tid];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += y[j];
    }
  }
  // weights relative to the largest: a sum of them is a sum of kBias more
  const Finish fin(top + kBias, sum, 0, a.sinks ? a.sinks[head] * kLog2e : -INFINITY);
  float out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) out[j] = sum == 0.f ? 0.f : v[j] * fin.factor;
  store_row<4>(a.out, a.out_type, row * c.d + at, out);
  if (at == 0 && a.lse) a.lse[row] = fin.lse2 * kLn2;
}

template <int D>
hipError_t launch_dim(const Cache &c, const Batch &b, const Attention &a, int splits, void *ws, hipStream_t s) {
  const int64_t tiles = (int64_t)b.max_new * a.group > kRows ? (int64_t)b.n_tok * a.group / kRows + b.n_seq : b.n_seq;
  const dim3 grid((uint32_t)(tiles * c.n_kv), (uint32_t)splits);
  if (a.q.type == kF32 || a.out_type == kF32)
    stream_kernel<D, true><<<grid, 256, 0, s>>>(c, b, a, splits, ws);
  else
    stream_kernel<D, false><<<grid, 256, 0, s>>>(c, b, a, splits, ws);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_stream(const Cache &c, const Batch &b, const Attention &a, int splits, void *ws, hipStream_t s) {
  switch (c.d) {
    case 64: return launch_dim<64>(c, b, a, splits, ws, s);
    case 128: return launch_dim<128>(c, b, a, splits, ws, s);
    case 192: return launch_dim<192>(c, b, a, splits, ws, s);
    case 256: return launch_dim<256>(c, b, a, splits, ws, s);
    default: return launch_dim<512>(c, b, a, splits, ws, s);
  }
}

hipError_t launch_join(const Cache &c, const Batch &b, const Attention &a, int splits, const void *ws, hipStream_t s) {
  const uint32_t rows = (uint32_t)b.n_tok * a.n_q, groups = 256 / (c.d / 4);
  join_kernel<<<dim3(splits <= kFewSplits ? (rows + groups - 1) / groups : rows), 256, 0, s>>>(c, b, a, splits, ws);
  return hipGetLastError();
}

}  // namespace kv
