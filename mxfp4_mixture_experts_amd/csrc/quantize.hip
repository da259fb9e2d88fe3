// MXFP4 quantisation of bf16 or fp32 tensors, for gfx950: the inverse of
// mxfp4_dequantize.
//
// A block of 32 elements shares the exponent e = floor(log2(max |x|)) - 2, at
// least -127, which brings its largest magnitude into [4, 8); its scale byte is
// e + 127, read off the fp32 exponent field of the maximum.  Each element
// becomes the E2M1 value nearest to x * 2^-e (ties to the even code, magnitudes
// above 6 to 6).  The multiplication by a power of two is exact down to the
// fp32 subnormals, which lie far below the smallest code's rounding border, so
// the one rounding is v_cvt_scalef32_pk_fp4_f32's.  That convert is called with
// scale 1: its own scale argument would be subnormal for e = -127.  A block
// with a NaN or an infinity gets E8M0's NaN, byte 255, and zero codes.
//
// Rows in storage order: 8 elements a lane, four lanes a block, so every load
// and store of a wave is contiguous; bound by HBM.  Columns (the transposed
// form): a lane holds a column's whole block, 32 row loads of 64 columns a wave; the
// waves of a workgroup hold consecutive blocks of the same columns, whose codes meet
// in LDS, so that the stores run along the columns: 512 contiguous bytes of values,
// 128 of codes.  4096 x 2880 bf16 with values: 10.2 us where the tensors stay in the last-
// level cache (5.2 TB/s), 14.3 from HBM (3.7); fp32 16.1 and 16.6 (4.6 TB/s).  (In the cache:
// written by the lanes that made them, 16 bytes a column, 24.6; with two bf16 columns a
// lane in 32-bit loads 11.5; the values' stores not marked as streamed 14.6.)

#include "kernels.h"
#include "common.h"

namespace mxfp4 {
namespace {

constexpr int kQnThreads = 256;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Scale byte of a block whose largest magnitude has fp32 bits m: the exponent
// field less 2 (an element's own exponent reaches 2), 0 for tinier blocks; 255
// for an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if (m >= 0x7f800000u) return 255u;
  const uint32_t ex = m >> 23;
  return ex > 2 ? ex - 2 : 0u;
}

// 2^(127 - byte), the factor that brings a block into the codes' range (byte 0 ..
// 252; with byte 255 the elements are taken as 0 and the factor is not used)
__device__ __forceinline__ float block_factor(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes l ^ 1
  return umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes l ^ 2
}

// eight codes (element 0 in the low nibble of byte 0) of y, already scaled
__device__ __forceinline__ uint32_t codes8(const float (&y)[8]) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.0f, 3);
  return c;
}

// the bf16 values of eight codes under a scale byte (NaN for byte 255)
__device__ __forceinline__ u32x4_t values8(uint32_t c, uint32_t byte) {
  if (byte == 255u) return u32x4_t{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
  const float f = __uint_as_float(byte ? byte << 23 : 0x00400000u);
  return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 3))};
}

// the raw 8 elements of item i and their fp32 bit patterns
template <bool F32>
struct Item {
  u32x4_t v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* x, size_t i) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(x) + i * (F32 ? 2 : 1);
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); j++) v[j] = __builtin_nontemporal_load(p + j);
  }
  __device__ __forceinline__ uint32_t bits(int j) const {
    if (F32) return v[j >> 2][j & 3];
    const uint32_t w = v[0][j >> 1];
    return (j & 1) ? (w & 0xffff0000u) : (w << 16);
  }
};

// items of 8 elements, four to a block; kQnUnroll of them in flight a lane
constexpr int kQnUnroll = 4;

template <bool F32, bool VALUES>
__global__ __launch_bounds__(kQnThreads) void quantize_kernel(const void* __restrict__ x, size_t items,
                                                              uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales,
                                                              u32x4_t* __restrict__ values) {
  const int lane = threadIdx.x & 63;
  const size_t wave = ((size_t)blockIdx.x * kQnThreads + threadIdx.x) >> 6;
  const size_t waves = (size_t)gridDim.x * (kQnThreads / 64);
  for (size_t base = wave * 64 * kQnUnroll; base < items; base += waves * 64 * kQnUnroll) {
    Item<F32> it[kQnUnroll];
#pragma unroll
    for (int u = 0; u < kQnUnroll; u++) {
      const size_t i = base + 64 * u + lane;
      it[u].load(x, i < items ? i : items - 1);  // unconditional loads; stores masked
    }
#pragma unroll
    for (int u = 0; u < kQnUnroll; u++) {
      const size_t i = base + 64 * u + lane;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) m = umax(m, it[u].bits(j) & 0x7fffffffu);
      // items is a multiple of 4: a block's four lanes are valid together
      const uint32_t byte = scale_byte(quad_max(m));
      const float f = block_factor(byte);
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; j++) y[j] = byte == 255u ? 0.f : __uint_as_float(it[u].bits(j)) * f;
      const uint32_t c = codes8(y);
      if (i < items) {
        codes[i] = c;
        if ((lane & 3) == 0) scales[i >> 2] = (uint8_t)byte;
        if (VALUES) __builtin_nontemporal_store(values8(c, byte), values + i);
      }
    }
  }
}

// The transposed form: x [R, C]; output row c holds column c, in blocks along r.
// A wave takes one block of 32 rows of 64 columns.
constexpr int kQtWaves = 8;

template <bool F32, bool VALUES>
__global__ __launch_bounds__(kQtWaves * 64) void quantize_transposed_kernel(const void* __restrict__ x, size_t R,
                                                                            int C, u32x4_t* __restrict__ codes,
                                                                            uint8_t* __restrict__ scales,
                                                                            u32x4_t* __restrict__ values) {
  // a column's 8 blocks of codes, 4 words of padding by which 64 columns' stores meet no bank twice
  __shared__ __attribute__((aligned(16))) uint32_t tile[64][kQtWaves * 4 + 4];
  __shared__ uint8_t bytes[64][kQtWaves];
  const size_t RB = R >> 5;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const size_t rb0 = (size_t)blockIdx.x * kQtWaves;
  const int col0 = blockIdx.y * 64;
  uint32_t raw[32];
  // past the last block or column: the last one's again, not stored
  const size_t at = (rb0 + wave < RB ? rb0 + wave : RB - 1) * 32 * C + (col0 + lane < C ? col0 + lane : C - 1);
#pragma unroll
  for (int r = 0; r < 32; r++) {
    if (F32) raw[r] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(x) + at + (size_t)r * C);
    else raw[r] = (uint32_t)reinterpret_cast<const uint16_t*>(x)[at + (size_t)r * C] << 16;
  }
  uint32_t m = 0;
#pragma unroll
  for (int r = 0; r < 32; r++) m = umax(m, raw[r] & 0x7fffffffu);
  const uint32_t byte = scale_byte(m);
  const float f = block_factor(byte);
  u32x4_t q;
#pragma unroll
  for (int g = 0; g < 4; g++) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = byte == 255u ? 0.f : __uint_as_float(raw[8 * g + j]) * f;
    q[g] = codes8(y);
  }
  *reinterpret_cast<u32x4_t*>(&tile[lane][wave * 4]) = q;
  bytes[lane][wave] = (uint8_t)byte;
  __syncthreads();
  const int blocks = (int)(RB - rb0 < kQtWaves ? RB - rb0 : kQtWaves), cols = min(64, C - col0);
  // thread: a block of a column, 8 blocks of 8 columns a wave
#pragma unroll
  for (int i = threadIdx.x; i < 64 * kQtWaves; i += kQtWaves * 64) {
    const int c = i / kQtWaves, b = i % kQtWaves;
    if (c < cols && b < blocks) {
      const size_t o = (size_t)(col0 + c) * RB + rb0 + b;
      codes[o] = *reinterpret_cast<const u32x4_t*>(&tile[c][b * 4]);
      scales[o] = bytes[c][b];
    }
  }
  if (VALUES) {
    // thread: 8 values of a column, 2 columns' 32 a wave
#pragma unroll 2
    for (int i = threadIdx.x; i < 64 * kQtWaves * 4; i += kQtWaves * 64) {
      const int c = i / (kQtWaves * 4), w = i % (kQtWaves * 4);
      if (c < cols && w < blocks * 4)
        __builtin_nontemporal_store(values8(tile[c][w], bytes[c][w >> 2]),
                                    values + ((size_t)(col0 + c) * RB + rb0) * 4 + w);
    }
  }
}

}  // namespace

hipError_t launch_quantize(const void* x, bool f32, size_t nblocks, uint8_t* blocks, uint8_t* scales,
                           uint16_t* values, hipStream_t stream) {
  const size_t items = nblocks * 4;
  const size_t per_wg = (size_t)kQnThreads * kQnUnroll;
  const size_t want = (items + per_wg - 1) / per_wg;
  const unsigned grid = (unsigned)(want < 8192 ? want : 8192);  // 32 workgroups per CU, then grid-stride
  auto kern = f32 ? (values ? quantize_kernel<true, true> : quantize_kernel<true, false>)
                  : (values ? quantize_kernel<false, true> : quantize_kernel<false, false>);
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kQnThreads), 0, stream, x, items, reinterpret_cast<uint32_t*>(blocks),
                     scales, reinterpret_cast<u32x4_t*>(values));
  return hipGetLastError();
}

hipError_t launch_quantize_transposed(const void* x, bool f32, long long R, int C, uint8_t* blocks, uint8_t* scales,
                                      uint16_t* values, hipStream_t stream) {
  const size_t RB = (size_t)R >> 5;
  const dim3 grid((unsigned)((RB + kQtWaves - 1) / kQtWaves), (unsigned)((C + 63) / 64));
  auto launch = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(kQtWaves * 64), 0, stream, x, (size_t)R, C,
                       reinterpret_cast<u32x4_t*>(blocks), scales, reinterpret_cast<u32x4_t*>(values));
  };
  if (f32) launch(values ? quantize_transposed_kernel<true, true> : quantize_transposed_kernel<true, false>);
  else launch(values ? quantize_transposed_kernel<false, true> : quantize_transposed_kernel<false, false>);
  return hipGetLastError();
}

}  // namespace mxfp4
