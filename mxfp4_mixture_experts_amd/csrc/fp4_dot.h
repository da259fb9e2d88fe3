// MXFP4 weights times bf16 inputs by dot products, shared by the kernels that
// stream weight rows for a few tokens.
#pragma once
#include "common.h"

namespace mxfp4 {

typedef __bf16 bf16x2_d __attribute__((ext_vector_type(2)));

// 2^(s - 127) as an fp32 value; s = 0 is the subnormal 2^-127
__device__ __forceinline__ float e8m0_value(uint32_t s) { return __uint_as_float(s ? (s << 23) : 0x00400000u); }

// eight products of bf16 pairs, summed in fp32 in element order
__device__ __forceinline__ float dot8(const uint4 w, const uint4 x, float a) {
  const uint32_t wv[4] = {w.x, w.y, w.z, w.w}, xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; i++)
    a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_d, wv[i]), __builtin_bit_cast(bf16x2_d, xv[i]), a,
                                        false);
  return a;
}

// One MXFP4 block's 32 products with 32 staged bf16 inputs, added to a: the
// block's four code words w (8 codes each) become exact bf16 weights through
// v_cvt_scalef32_pk_bf16_fp4 with the E8M0 factor sf, and v_dot2_f32_bf16
// multiplies them by the inputs x0 .. x3 (8 each) and sums in fp32, in element
// order.  keep = 0 zeroes the block (a block past K).
__device__ __forceinline__ float block_dot(const uint4 w, uint32_t keep, float sf, const uint4 x0, const uint4 x1,
                                           const uint4 x2, const uint4 x3, float a) {
  const uint32_t wd[4] = {w.x & keep, w.y & keep, w.z & keep, w.w & keep};
  const uint4 xv[4] = {x0, x1, x2, x3};
#pragma unroll
  for (int d = 0; d < 4; d++) {
    a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wd[d], sf, 0),
                                        __builtin_bit_cast(bf16x2_d, xv[d].x), a, false);
    a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wd[d], sf, 1),
                                        __builtin_bit_cast(bf16x2_d, xv[d].y), a, false);
    a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wd[d], sf, 2),
                                        __builtin_bit_cast(bf16x2_d, xv[d].z), a, false);
    a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wd[d], sf, 3),
                                        __builtin_bit_cast(bf16x2_d, xv[d].w), a, false);
  }
  return a;
}

}  // namespace mxfp4
