// kv8_device.h -- device helpers of the 8-bit key/value cache: ragged batches,
// page lookups, strided rows of three types, codes to fp16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv8_launch.h"

namespace kv {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <class T, class S>
__device__ __forceinline__ T as(const S &v) {
  return __builtin_bit_cast(T, v);
}

// ---- the batch -----------------------------------------------------------

// A sequence's rows [row0, row0 + n) of the token arrays and its length; row i is at
// position first + i, which may be negative.
struct Span {
  int row0, n, len, first;
};

__device__ __forceinline__ int start_of(const Batch &b, int s) {
  return b.starts ? min(max(b.starts[s], 0), b.n_tok) : s;
}

__device__ __forceinline__ Span span_of(const Batch &b, const Cache &c, int s) {
  Span r;
  r.row0 = start_of(b, s);
  r.n = b.starts ? min(max(start_of(b, s + 1) - r.row0, 0), b.max_new) : 1;
  r.len = min(max(b.lens[s], 0), b.width << c.page_log);
  r.first = r.len - r.n;
  return r;
}

// Work is handed out in units of `unit` rows * mult: sequence s has the slots from
// first_slot(s) on, which leaves each at least as many as it has units (`spare` more than
// whole ones), without a pass over the batch.
struct Slots {
  int unit, mult, spare;
  __device__ __forceinline__ int64_t first(const Batch &b, int s) const {
    return (int64_t)start_of(b, s) * mult / unit + (int64_t)spare * s;
  }
};

// The sequence that slot w belongs to: the last one whose first slot is not behind w.
// Every lane of a wave calls this with the same w; 64 sequences a step.
__device__ __forceinline__ int find_sequence(const Batch &b, const Slots &slots, int64_t w) {
  const int lane = threadIdx.x & 63;
  int lo = 0, span = b.n_seq;
  while (span > 1) {
    const int step = (span + 63) >> 6;
    const int off = lane * step;
    const bool le = off < span && slots.first(b, lo + off) <= w;
    const int n = __popcll(__ballot(le));
    const int skip = max(n - 1, 0) * step;
    lo += skip;
    span = min(step, span - skip);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Page of a position (below len), or -1 where the table holds none of the pool.
__device__ __forceinline__ int page_of(const Cache &c, const Batch &b, int s, int pos) {
  const int id = b.table[(int64_t)s * b.width + (pos >> c.page_log)];
  return (uint32_t)id < (uint32_t)c.n_pages ? id : -1;
}

// Codes of 16 tokens from pos on: a multiple of 16 within its page.  The same offset for K and V.
__device__ __forceinline__ int64_t code_offset(const Cache &c, int page, int head, int pos) {
  return ((((int64_t)page * c.n_kv + head) << c.page_log) + (pos & ((1 << c.page_log) - 1))) * c.d;
}
__device__ __forceinline__ int64_t scale_offset(const Cache &c, int page, int head, int pos) {
  return (((int64_t)page * c.n_kv + head) << (c.page_log - c.block_log)) +
         ((pos & ((1 << c.page_log) - 1)) >> c.block_log);
}

// ---- rows ----------------------------------------------------------------

// N adjacent values (4 or 8 times a power of two) of any of the three types as fp32; wide:
// the address is aligned as the row's start is (16 bytes).
template <int TYPE, int N>
__device__ __forceinline__ void load_values(const void *p, int64_t at, bool wide, float (&v)[N]) {
  if constexpr (TYPE == kF32) {
    const float *x = static_cast<const float *>(p) + at;
    if (wide) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const f32x4 t = reinterpret_cast<const f32x4 *>(x)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = x[i];
    }
  } else {
    const uint16_t *x = static_cast<const uint16_t *>(p) + at;
    uint16_t raw[N];
    if (wide) {
      if constexpr (N >= 8) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          const u32x4 t = reinterpret_cast<const u32x4 *>(x)[i];
#pragma unroll
          for (int j = 0; j < 8; ++j) raw[8 * i + j] = (uint16_t)(t[j >> 1] >> (16 * (j & 1)));
        }
      } else {
        const u32x2 t = *reinterpret_cast<const u32x2 *>(x);
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = (uint16_t)(t[j >> 1] >> (16 * (j & 1)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) raw[i] = x[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = TYPE == kBF16 ? as<float>((uint32_t)raw[i] << 16) : (float)as<_Float16>(raw[i]);
  }
}

// Eight adjacent values as they lie in memory.
template <int TYPE>
struct Eight {
  u32x4 raw[TYPE == kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *p, int64_t at, bool wide) {
    if constexpr (TYPE == kF32) {
      const uint32_t *x = static_cast<const uint32_t *>(p) + at;
      if (wide) {
        raw[0] = reinterpret_cast<const u32x4 *>(x)[0];
        raw[1] = reinterpret_cast<const u32x4 *>(x)[1];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) raw[j >> 2][j & 3] = x[j];
      }
    } else {
      const uint16_t *x = static_cast<const uint16_t *>(p) + at;
      if (wide) {
        raw[0] = *reinterpret_cast<const u32x4 *>(x);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[0][j] = x[2 * j] | (uint32_t)x[2 * j + 1] << 16;
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (TYPE == kF32) return as<float>(raw[j >> 2][j & 3]);
    const uint32_t bits = raw[0][j >> 1] >> (16 * (j & 1));
    return TYPE == kBF16 ? as<float>(bits << 16) : (float)as<_Float16>((uint16_t)bits);
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, as<uint32_t>(get(j)) & 0x7fffffffu);
    return m;
  }
};

// bf16 and fp16 bits, rounded to nearest even.
__device__ __forceinline__ uint32_t bf16_bits(float v) { return as<uint16_t>((__bf16)v); }
__device__ __forceinline__ uint32_t f16_bits(float v) { return as<uint16_t>((_Float16)v); }

// N (a multiple of 4) adjacent values as TYPE, rounded once, at an address aligned to 4 of them.
template <int TYPE, int N>
__device__ __forceinline__ void store_values(void *p, int64_t at, const float (&v)[N]) {
  if constexpr (TYPE == kF32) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at)[i] =
          f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      w[i] = TYPE == kBF16 ? bf16_bits(v[2 * i]) | bf16_bits(v[2 * i + 1]) << 16
                           : f16_bits(v[2 * i]) | f16_bits(v[2 * i + 1]) << 16;
    uint16_t *o = static_cast<uint16_t *>(p) + at;
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i)
        reinterpret_cast<u32x4 *>(o)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) reinterpret_cast<u32x2 *>(o)[i] = u32x2{w[2 * i], w[2 * i + 1]};
    }
  }
}

// ---- codes ---------------------------------------------------------------

// Four int8 codes as fp16, exactly: the byte q + 128 under the exponent of 1024 (0x64)
// reads 1024 + 128 + q, from which 1152 is taken.  Five instructions.
__device__ __forceinline__ h4 codes_f16(uint32_t codes) {
  const uint32_t u = codes ^ 0x80808080u;
  const h2 bias = {(_Float16)1152.f, (_Float16)1152.f};
  const h2 lo = as<h2>(__builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias;
  const h2 hi = as<h2>(__builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias;
  return h4{lo.x, lo.y, hi.x, hi.y};
}
__device__ __forceinline__ h8 codes_f16(uint32_t a, uint32_t b) {
  const h4 x = codes_f16(a), y = codes_f16(b);
  return h8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}

}  // namespace kv
