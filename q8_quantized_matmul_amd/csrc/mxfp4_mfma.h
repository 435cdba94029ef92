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

// A lane's operands of the four instructions of a step, 16 blocks (512 values) of a
// row.  Instruction i takes blocks 4 i + g from lane group g = l / 16, so that the
// four lanes of a row read 64 adjacent bytes at a time, what the caches serve at
// once (four adjacent blocks to a lane: a layer of 64 tokens 546-559 us, with this
// order 535; loads that bypass the caches 615).  Which k goes to which lane does
// not matter as long as A and B agree.
struct Blocks4 {
  u32x4 c[4];
  uint32_t s;  // scale of block i in byte i
};

constexpr int kStepBlocks = 16;

// The scale bytes of blocks 4 g .. 4 g + 3 in lane group g -- one dword of the row --
// to byte i of lane group g = the scale of block 4 i + g: a 4 x 4 transpose of bytes
// between the lane groups.
__device__ __forceinline__ uint32_t spread_scales(uint32_t d) {
  const uint32_t g = (threadIdx.x >> 4) & 3;
  const auto h = __builtin_amdgcn_permlane32_swap(d, d, false, false);         // groups 0 1 0 1, 2 3 2 3
  const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);  // group 0, 1 everywhere
  const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);  // 2, 3
  const uint32_t sel = g | ((4 + g) << 8);
  return __builtin_amdgcn_perm(lo[1], lo[0], sel | 0x0C0C0000u) |
         __builtin_amdgcn_perm(hi[1], hi[0], (sel << 16) | 0x0C0Cu);
}

// Byte offsets of the lane's blocks b0 + 4 i + g of row `row` of a matrix of nb
// blocks a row, from the matrix (within 32 bits: the caller gives the address of the
// tile it works on, which is uniform, so that an address costs a lane one register).
// Blocks past the end of the row are read from inside it, to keep the loads free of
// branches, and given the scale byte 0; both operands do so, and products of 2^-254
// vanish in fp32.  Scale rows may start at any byte.  SHORT: nb below 4.
template <bool SHORT>
struct Offsets4 {
  uint32_t c[4];
  uint32_t s;
  int past;  // of the dword's four blocks b0 + 4 g .. + 3, those past the end
  __device__ __forceinline__ Offsets4(uint32_t row, int b0, int nb) {
    const int g = (threadIdx.x >> 4) & 3, b = b0 + 4 * g;
    past = min(max(b + 4 - nb, 0), 4);
    s = row * (uint32_t)nb + (SHORT ? 0u : (uint32_t)min(b, nb - 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = (row * (uint32_t)nb + (uint32_t)min(b0 + 4 * i + g, nb - 1)) * 16;
  }
};

// Global-memory pointers, also where the base came from memory: a generic load
// would count on the LDS counter too.
typedef __attribute__((address_space(1))) const u32x4 global_u32x4;
typedef __attribute__((address_space(1))) const uint8_t global_u8;

// The blocks, with their scales still as loaded: finish_blocks when they are used.
template <bool SHORT>
__device__ __forceinline__ void load_blocks(const uint8_t *codes, const uint8_t *scales,
                                            const Offsets4<SHORT> &o, int nb, Blocks4 &r) {
  typedef uint32_t u32_a1 __attribute__((aligned(1)));
  typedef __attribute__((address_space(1))) const u32_a1 global_u32_a1;
  global_u8 *c = (global_u8 *)codes, *s = (global_u8 *)scales;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.c[i] = *(global_u32x4 *)(c + o.c[i]);
  if constexpr (SHORT) {
    r.s = 0;
    for (int i = 0; i < nb; ++i) r.s |= (uint32_t)s[o.s + i] << (8 * i);
  } else {  // near the end the four bytes read end with the row
    r.s = *(global_u32_a1 *)(s + o.s);
  }
}
template <bool SHORT>
__device__ __forceinline__ void finish_blocks(const Offsets4<SHORT> &o, Blocks4 &r) {
  if constexpr (SHORT) r.s = o.past == 4 ? 0u : r.s;
  else r.s = (r.s >> (4 * o.past)) >> (4 * o.past);  // in two steps, so that 32 bits give zero
  r.s = spread_scales(r.s);
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
