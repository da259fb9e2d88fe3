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
// r moved down by n elements (0 <= n < 8), zeros behind
__device__ __forceinline__ void shift_down(Raw8<uint16_t>& r, int n) {
  if (n & 4) r.d = u32x4_t{r.d[2], r.d[3], 0u, 0u};
  if (n & 2) r.d = u32x4_t{r.d[1], r.d[2], r.d[3], 0u};
  if (n & 1) {
    r.d[0] = __builtin_amdgcn_alignbit(r.d[1], r.d[0], 16);
    r.d[1] = __builtin_amdgcn_alignbit(r.d[2], r.d[1], 16);
    r.d[2] = __builtin_amdgcn_alignbit(r.d[3], r.d[2], 16);
    r.d[3] >>= 16;
  }
}
__device__ __forceinline__ void shift_down(Raw8<float>& r, int n) {
  if (n & 4) r.a = r.b, r.b = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (n & 2) r.a = f32x4_t{r.a[2], r.a[3], r.b[0], r.b[1]}, r.b = f32x4_t{r.b[2], r.b[3], 0.f, 0.f};
  if (n & 1) r.a = f32x4_t{r.a[1], r.a[2], r.a[3], r.b[0]}, r.b = f32x4_t{r.b[1], r.b[2], r.b[3], 0.f};
}
__device__ __forceinline__ void set8(Raw8<uint16_t>& r, int i, uint16_t v) {
  r.d[i >> 1] |= (uint32_t)v << (16 * (i & 1));
}
__device__ __forceinline__ void set8(Raw8<float>& r, int i, float v) {
  if (i < 4)
    r.a[i] = v;
  else
    r.b[i - 4] = v;
}

// Elements i .. i + 7 of a row of N (0 where i >= N).  A row's last, partial
// chunk is fetched as the row's last eight elements, so it is the same single
// load; settle8 moves it into place.  The two are apart because the move has to
// wait for the load.  tiny: the row has fewer than eight elements, read one by
// one; a launch-wide value, so that the choice is a scalar branch (as a lane's
// own choice it makes each wide load wait for the element loads).
template <typename E>
__device__ __forceinline__ void fetch8(const E* row, int i, int N, bool tiny, Raw8<E>& r) {
  r = Raw8<E>{};
  if (tiny) {
#pragma unroll
    for (int j = 0; j < 7; j++)
      if (i == 0 && j < N) set8(r, j, row[j]);
  } else if (i < N) {
    fetch8_full(row + min(i, N - 8), r);
  }
}
// whether a row of N has a partial last chunk that settle8 has to move
__device__ __forceinline__ bool ragged(int N) { return N > 8 && (N & 7) != 0; }
template <typename E>
__device__ __forceinline__ void settle8(int i, int N, Raw8<E>& r) {
  if (i < N && i + 8 > N) shift_down(r, i + 8 - N);
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

// STREAM: marked non-temporal
template <bool STREAM>
__device__ __forceinline__ void store8_full(uint16_t* p, const float (&v)[8]) {
  u32x4_t d;
#pragma unroll
  for (int i = 0; i < 4; i++) d[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if constexpr (STREAM)
    __builtin_nontemporal_store(d, reinterpret_cast<u32x4_a2*>(p));
  else
    *reinterpret_cast<u32x4_a2*>(p) = d;
}
template <bool STREAM>
__device__ __forceinline__ void store8_full(float* p, const float (&v)[8]) {
  f32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; i++) a[i] = v[i], b[i] = v[4 + i];
  if constexpr (STREAM) {
    __builtin_nontemporal_store(a, reinterpret_cast<f32x4_a4*>(p));
    __builtin_nontemporal_store(b, reinterpret_cast<f32x4_a4*>(p + 4));
  } else {
    *reinterpret_cast<f32x4_a4*>(p) = a;
    *reinterpret_cast<f32x4_a4*>(p + 4) = b;
  }
}

typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef float f32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));

// the first n (under 8) elements, as pieces of four, two and one
__device__ __forceinline__ void store8_part(uint16_t* p, int n, const float (&v)[8]) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; i++) d[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if (n & 4) {
    *reinterpret_cast<u32x2_a2*>(p) = u32x2_a2{d[0], d[1]};
    d[0] = d[2], d[1] = d[3];
    p += 4;
  }
  if (n & 2) {
    *reinterpret_cast<u32_a2*>(p) = d[0];
    d[0] = d[1];
    p += 2;
  }
  if (n & 1) *p = (uint16_t)d[0];
}
__device__ __forceinline__ void store8_part(float* p, int n, const float (&v)[8]) {
  float d[4] = {v[0], v[1], v[2], v[3]};
  if (n & 4) {
    *reinterpret_cast<f32x4_a4*>(p) = f32x4_a4{d[0], d[1], d[2], d[3]};
    d[0] = v[4], d[1] = v[5], d[2] = v[6];
    p += 4;
  }
  if (n & 2) {
    *reinterpret_cast<f32x2_a4*>(p) = f32x2_a4{d[0], d[1]};
    d[0] = d[2];
    p += 2;
  }
  if (n & 1) *p = d[0];
}

// elements i .. i + 7 of a row of N, those that it has; stream: whole chunks
// marked non-temporal
template <typename E>
__device__ __forceinline__ void store8(E* row, int i, int N, const float (&v)[8], bool stream = false) {
  if (i + 8 <= N) {
    if (stream) {
      // the empty statements keep the two branches' stores from being moved out
      // of them as one, which drops the mark
      asm volatile("");
      store8_full<true>(row + i, v);
      asm volatile("");
    } else {
      store8_full<false>(row + i, v);
    }
  } else if (i < N) {
    store8_part(row + i, N - i, v);
  }
}

// Totals over groups of L neighbouring lanes (a power of two); every lane of a
// group receives its total, and adding in this order gives every lane the same
// bits.  Register moves only (DPP within 16 lanes, gfx950's row swaps across
// them): about 8 cycles a step, where a lane exchange through the LDS takes over
// a hundred.  Lanes of other groups may be inactive.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits(int v) { return (uint32_t)v; }
__device__ __forceinline__ void from_bits(uint32_t b, float& v) { v = __uint_as_float(b); }
__device__ __forceinline__ void from_bits(uint32_t b, int& v) { v = (int)b; }

template <int L, typename V, typename Op>
__device__ __forceinline__ V group_reduce(V v, Op op) {
  if constexpr (L >= 2) v = op(v, dpp<0xB1>(v));    // quad_perm [1, 0, 3, 2]
  if constexpr (L >= 4) v = op(v, dpp<0x4E>(v));    // quad_perm [2, 3, 0, 1]
  if constexpr (L >= 8) v = op(v, dpp<0x141>(v));   // the other quad of eight lanes (mirrored)
  if constexpr (L >= 16) v = op(v, dpp<0x140>(v));  // the other half of sixteen (mirrored)
  V x, y;
  if constexpr (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
    from_bits(p[0], x);
    from_bits(p[1], y);
    v = op(x, y);
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
    from_bits(p[0], x);
    from_bits(p[1], y);
    v = op(x, y);
  }
  return v;
}
template <int L, typename V>
__device__ __forceinline__ V group_sum(V v) {
  return group_reduce<L>(v, [](V a, V b) { return a + b; });
}
// the sum of the four lanes of a wave that have the same place among 16
__device__ __forceinline__ float rows_sum(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
// The maximum, compared as integers in the floats' order: an integer maximum
// takes its moved operand in the same instruction, a float one first quiets it.
template <int L>
__device__ __forceinline__ float group_max(float v) {
  int key = __float_as_int(v);
  key ^= (key >> 31) & 0x7fffffff;
  key = group_reduce<L>(key, [](int a, int b) { return a > b ? a : b; });
  return __int_as_float(key ^ ((key >> 31) & 0x7fffffff));
}
// the same for a group size known at the call only (uniform, at most 32)
__device__ __forceinline__ float group_sum_up_to_32(float v, int L) {
  if (L >= 2) v += dpp<0xB1>(v);
  if (L >= 4) v += dpp<0x4E>(v);
  if (L >= 8) v += dpp<0x141>(v);
  if (L >= 16) v += dpp<0x140>(v);
  if (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

}  // namespace mxfp4
