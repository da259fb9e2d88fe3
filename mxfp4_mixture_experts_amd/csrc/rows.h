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

// Eight elements as loaded.  Fetching and widening are separate, so that all of
// a thread's loads are under way before the first result is waited for (a
// conversion beside each load would wait for it there).
template <typename E>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4_t d;
};
template <>
struct Raw8<float> {
  f32x4_t a, b;
};

__device__ __forceinline__ void fetch8_full(const uint16_t* p, Raw8<uint16_t>& r) {
  r.d = *reinterpret_cast<const u32x4_a2*>(p);
}
__device__ __forceinline__ void fetch8_full(const float* p, Raw8<float>& r) {
  r.a = *reinterpret_cast<const f32x4_a4*>(p);
  r.b = *reinterpret_cast<const f32x4_a4*>(p + 4);
}
// the first `valid` of the eight elements at p; 0 in the others
__device__ __forceinline__ void fetch8_part(const uint16_t* p, int valid, Raw8<uint16_t>& r) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t lo = 2 * i < valid ? p[2 * i] : 0u, hi = 2 * i + 1 < valid ? p[2 * i + 1] : 0u;
    r.d[i] = lo | (hi << 16);
  }
}
__device__ __forceinline__ void fetch8_part(const float* p, int valid, Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    r.a[i] = i < valid ? p[i] : 0.f;
    r.b[i] = 4 + i < valid ? p[4 + i] : 0.f;
  }
}
template <typename E>
__device__ __forceinline__ void fetch8(const E* p, int valid, Raw8<E>& r) {
  if (valid >= 8)
    fetch8_full(p, r);
  else if (valid > 0)
    fetch8_part(p, valid, r);
  else
    r = Raw8<E>{};
}

__device__ __forceinline__ void widen8(const Raw8<uint16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __uint_as_float(r.d[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.d[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = r.a[i], v[4 + i] = r.b[i];
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
  } else if (valid > 0) {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < valid) from_f32(v[i], p + i);
  }
}

// Totals over groups of L neighbouring lanes (a power of two); every lane of a
// group receives its total, and adding in this order gives every lane the same
// bits.  Register moves only (DPP within 16 lanes, gfx950's row swaps across
// them): about 8 cycles a step, where a lane exchange through the LDS takes over
// a hundred.  Lanes of other groups may be inactive.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int L, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  if constexpr (L >= 2) v = op(v, dpp<0xB1>(v));    // quad_perm [1, 0, 3, 2]
  if constexpr (L >= 4) v = op(v, dpp<0x4E>(v));    // quad_perm [2, 3, 0, 1]
  if constexpr (L >= 8) v = op(v, dpp<0x141>(v));   // the other quad of eight lanes (mirrored)
  if constexpr (L >= 16) v = op(v, dpp<0x140>(v));  // the other half of sixteen (mirrored)
  if constexpr (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace mxfp4
