// Rows of any length and element alignment, eight elements at a time: the
// loads and stores shared by the norm and the balance kernels.
#pragma once
#include "common.h"

namespace mxfp4 {

// 16 bytes at the alignment of their elements: gfx950 reads and writes global
// memory at any byte address, so rows of odd widths keep the 128-bit accesses.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));

// two fp32 -> two bf16 (round to nearest even), packed
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const bf16x2_v v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(float f, uint16_t* p) { *p = to_bf16(f); }
__device__ __forceinline__ void from_f32(float f, float* p) { *p = f; }
// f as the element type stores it
__device__ __forceinline__ float rounded(float f, const uint16_t*) { return bf16_bits_to_f32(to_bf16(f)); }
__device__ __forceinline__ float rounded(float f, const float*) { return f; }

__device__ __forceinline__ void unpack8(const u32x4_a2 d, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __uint_as_float(d[i] << 16);
    v[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void load8_full(const uint16_t* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const u32x4_a2*>(p), v);
}
__device__ __forceinline__ void load8_full(const float* p, float (&v)[8]) {
  const f32x4_a4 a = *reinterpret_cast<const f32x4_a4*>(p), b = *reinterpret_cast<const f32x4_a4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
}

// eight elements from p, of which the first `valid` exist; `fill` in the others
template <typename E>
__device__ __forceinline__ void load8(const E* p, int valid, float (&v)[8], float fill = 0.f) {
  if (valid >= 8) {
    load8_full(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = i < valid ? to_f32(p[i]) : fill;
  }
}

__device__ __forceinline__ void store8_full(uint16_t* p, const float (&v)[8]) {
  u32x4_a2 d;
#pragma unroll
  for (int i = 0; i < 4; i++) d[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4_a2*>(p) = d;
}
__device__ __forceinline__ void store8_full(float* p, const float (&v)[8]) {
  f32x4_a4 a, b;
#pragma unroll
  for (int i = 0; i < 4; i++) a[i] = v[i], b[i] = v[4 + i];
  *reinterpret_cast<f32x4_a4*>(p) = a;
  *reinterpret_cast<f32x4_a4*>(p + 4) = b;
}

template <typename E>
__device__ __forceinline__ void store8(E* p, int valid, const float (&v)[8]) {
  if (valid >= 8) {
    store8_full(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < valid) from_f32(v[i], p + i);
  }
}

}  // namespace mxfp4
