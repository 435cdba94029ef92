// mxfp4_quantize.hip -- MXFP4 quantization of rows, and back.
//
// Both are bound by memory: per block of 32 values the quantizer reads 64 or
// 128 bytes and writes 17.  A lane takes eight consecutive values (one or two
// 16-byte loads, one dword of codes), four lanes a block, so a wave's loads and
// code stores are contiguous and the block maximum is two cross-lane moves.
// The codes and scales of consecutive rows are contiguous whatever the row
// stride of x, so the grid runs over groups of eight values of the whole
// matrix; only the address of x needs the row.
//
// The unquantized side passes by the caches (it is touched once, and is most of the
// bytes), so that the codes stay in them for whoever reads them next.  Measured, 2048
// x 32768 bfloat16 quantized and then dequantized, 170 MB each way: 58 us, 67 with all
// accesses cached, 67 with none.  One group a lane: four of them are 57 us there, but
// 5.9 for 4.4 at 64 x 4096, where it is latency that counts.
#include "mxfp4_device.h"

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kGridX = 1u << 20;  // workgroups along x: a launch has 2^32 threads along it at most

template <int TYPE>
__device__ __forceinline__ Eight<TYPE> load_eight(const void *x, int64_t elem, bool aligned16) {
  Eight<TYPE> v;
  constexpr int N = sizeof(v.d) / 4;
  const uint8_t *p = static_cast<const uint8_t *>(x) + elem * (TYPE == kF32 ? 4 : 2);
  if (aligned16) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.d[4 * i + j] = t[j];
    }
  } else if constexpr (TYPE == kF32) {
#pragma unroll
    for (int i = 0; i < N; ++i) v.d[i] = reinterpret_cast<const uint32_t *>(p)[i];
  } else {
    const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) v.d[i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
  }
  return v;
}

// The thread's group of eight values.
__device__ __forceinline__ int64_t group() {
  return ((int64_t)blockIdx.y * kGridX + blockIdx.x) * kThreads + threadIdx.x;
}

// groups: n_rows * in_dim / 8.  A quad of lanes never straddles the end
// (groups is a multiple of 4), nor a row (in_dim / 8 is).
template <int TYPE>
__global__ __launch_bounds__(kThreads) void quantize_kernel(uint32_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales,
                                                            const void *__restrict__ x,
                                                            int64_t x_stride, int64_t groups,
                                                            int64_t groups_per_row,
                                                            bool aligned16) {
  const int64_t g = group();
  if (g >= groups) return;
  const int64_t row = g / groups_per_row;
  const Eight<TYPE> v = load_eight<TYPE>(x, row * x_stride + (g - row * groups_per_row) * 8, aligned16);
  const uint32_t byte = scale_byte(max_quad(amax_bits<TYPE>(v)));
  codes[g] = encode<TYPE>(v, byte);
  if ((g & 3) == 0) scales[g >> 2] = (uint8_t)byte;
}

constexpr uint32_t kNan32 = 0x7FC00000u;

template <int TYPE>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(void *__restrict__ out,
                                                              const uint32_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales,
                                                              int64_t groups) {
  const int64_t g = group();
  if (g >= groups) return;
  const uint32_t c = codes[g], b = scales[g >> 2];
  const float s = scale_value(b);
  f32x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  if (b == 255) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f32x2{__builtin_bit_cast(float, kNan32), __builtin_bit_cast(float, kNan32)};
  }
  if constexpr (TYPE == kF32) {
    f32x4 *o = static_cast<f32x4 *>(out) + 2 * g;
    __builtin_nontemporal_store(f32x4{p[0].x, p[0].y, p[1].x, p[1].y}, o);
    __builtin_nontemporal_store(f32x4{p[2].x, p[2].y, p[3].x, p[3].y}, o + 1);
  } else {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = TYPE == kBF16 ? bf16_bits(p[i].x) | (bf16_bits(p[i].y) << 16)
                           : f16_bits(p[i].x) | (f16_bits(p[i].y) << 16);
    __builtin_nontemporal_store(o, static_cast<u32x4 *>(out) + g);
  }
}

dim3 grid_of(int64_t groups) {
  const int64_t n = (groups + kThreads - 1) / kThreads;
  return n <= kGridX ? dim3((uint32_t)n) : dim3(kGridX, (uint32_t)((n + kGridX - 1) / kGridX));
}

}  // namespace

hipError_t launch_quantize(uint8_t *codes, uint8_t *scales, const void *x, int x_type,
                           int64_t x_stride, int64_t n_rows, int64_t in_dim, hipStream_t s) {
  const int64_t groups = n_rows * (in_dim / 8), per_row = in_dim / 8;
  const int64_t size = x_type == kF32 ? 4 : 2;
  const bool a16 = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (n_rows == 1 || x_stride * size % 16 == 0);
  auto *c = reinterpret_cast<uint32_t *>(codes);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of(groups), dim3(kThreads), 0, s, c, scales, x, x_stride,
                       groups, per_row, a16);
  };
  if (x_type == kF32) go(quantize_kernel<kF32>);
  else if (x_type == kBF16) go(quantize_kernel<kBF16>);
  else go(quantize_kernel<kF16>);
  return hipGetLastError();
}

hipError_t launch_dequantize(void *out, int out_type, const uint8_t *codes, const uint8_t *scales,
                             int64_t n_rows, int64_t in_dim, hipStream_t s) {
  const int64_t groups = n_rows * (in_dim / 8);
  auto *c = reinterpret_cast<const uint32_t *>(codes);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of(groups), dim3(kThreads), 0, s, out, c, scales, groups);
  };
  if (out_type == kF32) go(dequantize_kernel<kF32>);
  else if (out_type == kBF16) go(dequantize_kernel<kBF16>);
  else go(dequantize_kernel<kF16>);
  return hipGetLastError();
}

}  // namespace mx
