// mxfp4_mfma.h -- the scaled matrix instructions on MXFP4 operands, and the
// operand loads of the weight-streaming kernels.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with both formats e2m1: lane l holds the 32
// values of one block -- row l % 16 of its operand, k block l / 16 of the
// instruction's four -- in four registers, in the order they have in memory, and
// that block's scale byte in a byte of a fifth register that the instruction
// selects.  So a block is one 16-byte load, and nothing is unpacked.  The result
// D[i][j], i a row of A and j a row of B: lane l holds j = l % 16 and i = 4 *
// (l / 16) + 0..3.  The 32x32x64 form: row l % 32, block l / 32 of two, D with j
// = l % 32 and i = 8 * (r / 4) + 4 * (l / 32) + r % 4 for r = 0..15.
// Products and scales are exact; sums are fp32.
#pragma once

#include "mxfp4_device.h"

namespace mx {

template <int J>  // J: byte of the scale registers
__device__ __forceinline__ f32x4 mfma16(const u32x4 &a, uint32_t sa, const u32x4 &b, uint32_t sb,
                                        f32x4 c) {
  const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, J, (int)sa, J, (int)sb);
}

template <int J>
__device__ __forceinline__ f32x16 mfma32(const u32x4 &a, uint32_t sa, const u32x4 &b, uint32_t sb,
                                         f32x16 c) {
  const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, J, (int)sa, J, (int)sb);
}

// Four consecutive blocks of a row: a lane's operands of four instructions.  A
// step of 16 blocks (512 values) gives lane group l / 16 blocks 4 * (l / 16) +
// 0..3, so that the four lanes of a row read 256 adjacent bytes and the four
// scale bytes are one dword; which k goes to which lane does not matter as long
// as A and B agree.
struct Blocks4 {
  u32x4 c[4];
  uint32_t s;  // scale of block i in byte i
};

constexpr int kStepBlocks = 16;

// Global-memory pointers, also where the base came from memory: a generic load
// would count on the LDS counter too.
typedef __attribute__((address_space(1))) const u32x4 global_u32x4;
typedef __attribute__((address_space(1))) const uint32_t global_u32;
typedef __attribute__((address_space(1))) const uint8_t global_u8;

// Blocks b0..b0+3 of a row of nb blocks; blocks past the row are zero (codes and
// scale: 0 * 2^-127).  WHOLE: nb is a multiple of 4 and scale rows are dword
// aligned, so the four blocks are all inside or all outside.
template <bool WHOLE>
__device__ __forceinline__ void load_blocks(const uint8_t *codes, const uint8_t *scales, int b0,
                                            int nb, Blocks4 &r) {
  if constexpr (WHOLE) {
    if (b0 < nb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.c[i] = ((global_u32x4 *)(codes + (int64_t)b0 * 16))[i];
      r.s = *(global_u32 *)(scales + b0);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.c[i] = u32x4{0, 0, 0, 0};
      r.s = 0;
    }
  } else {
    r.s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.c[i] = u32x4{0, 0, 0, 0};
      if (b0 + i < nb) {
        r.c[i] = ((global_u32x4 *)(codes + (int64_t)b0 * 16))[i];
        r.s |= (uint32_t)((global_u8 *)scales)[b0 + i] << (8 * i);
      }
    }
  }
}

__device__ __forceinline__ f32x4 mfma_blocks4(const Blocks4 &a, const Blocks4 &b, f32x4 c) {
  c = mfma16<0>(a.c[0], a.s, b.c[0], b.s, c);
  c = mfma16<1>(a.c[1], a.s, b.c[1], b.s, c);
  c = mfma16<2>(a.c[2], a.s, b.c[2], b.s, c);
  return mfma16<3>(a.c[3], a.s, b.c[3], b.s, c);
}

// Stores N consecutive fp32 values as the output type, `valid` of them, with one
// store where all are valid and `wide` says the address is aligned to it.
template <int TYPE>
__device__ __forceinline__ void store4(void *out, int64_t elem, const f32x4 &v, int valid, bool wide) {
  if constexpr (TYPE == kF32) {
    float *p = static_cast<float *>(out) + elem;
    if (valid >= 4 && wide) {
      *reinterpret_cast<f32x4 *>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < valid) p[i] = v[i];
    }
  } else {
    uint16_t *p = static_cast<uint16_t *>(out) + elem;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = TYPE == kBF16 ? bf16_bits(v[i]) : f16_bits(v[i]);
    if (valid >= 4 && wide) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *reinterpret_cast<u32x2 *>(p) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < valid) p[i] = (uint16_t)h[i];
    }
  }
}

}  // namespace mx
