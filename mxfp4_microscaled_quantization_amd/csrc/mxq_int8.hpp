// The 8-bit rule shared by the row quantizer, the fused product and the quantized
// query/key norm: symmetric codes with one binary32 scale for a group of values,
//   s = fl32(amax / 127),  inv = fl32(127 / amax),  q = RNE(fl32(x * inv)) in [-127, 127],
// both quotients correctly rounded.  amax below 2^-118 (an all-zero group too) gives s = 0
// and codes 0: from there down s or inv would leave the normal range, and the values are
// nothing next to any output.  A group with an infinity or a NaN gets s = NaN and codes 0.
#pragma once

#include "mxq_device.hpp"

namespace mxq {

struct Int8Scale {
  float s;         // dequantization scale
  float inv;       // multiplier of the values; 0 where the codes are 0
  unsigned keep;   // all ones, or 0 where the codes are 0
};

// amax_bits: binary32 pattern of max |x| (sign clear), compared as an integer, so that an
// infinity or a NaN wins over every finite value.
__device__ __forceinline__ Int8Scale int8_scale(unsigned amax_bits) {
  Int8Scale r;
  if (amax_bits >= 0x7F800000u) {
    r.s = __uint_as_float(0x7FC00000u);
    r.inv = 0.0f;
    r.keep = 0u;
  } else if (amax_bits < 0x04800000u) {   // 2^-118
    r.s = 0.0f;
    r.inv = 0.0f;
    r.keep = 0u;
  } else {
    const float amax = __uint_as_float(amax_bits);
    r.s = amax / 127.0f;
    r.inv = 127.0f / amax;
    r.keep = ~0u;
  }
  return r;
}

// RNE(fl32(x * inv)) of four values as four bytes.  Adding 1.5 * 2^23 leaves the integer
// nearest to the (already rounded) product, ties to even, in the low bits of the sum; the
// product and the sum must not contract into one rounding.
__device__ __forceinline__ unsigned int8_pack4(float x0, float x1, float x2, float x3, float inv) {
#pragma clang fp contract(off)
  constexpr float kMagic = 12582912.0f;
  const float p0 = x0 * inv, p1 = x1 * inv, p2 = x2 * inv, p3 = x3 * inv;
  const unsigned b0 = __float_as_uint(p0 + kMagic), b1 = __float_as_uint(p1 + kMagic);
  const unsigned b2 = __float_as_uint(p2 + kMagic), b3 = __float_as_uint(p3 + kMagic);
  // v_perm_b32: bytes 0-3 are the second operand's, 4-7 the first's
  const unsigned lo = __builtin_amdgcn_perm(b1, b0, 0x0C0C0400u);
  const unsigned hi = __builtin_amdgcn_perm(b3, b2, 0x04000C0Cu);
  return lo | hi;
}

// max |x| of the two bf16 in a word, as bf16 patterns in both halves
__device__ __forceinline__ v2h abs_bf16x2(int pair) { return __builtin_bit_cast(v2h, (unsigned)pair & 0x7FFF7FFFu); }

// Max over each 8 or 16 lanes, or the 64 lanes of a wave, in every lane: DPP inside a row of
// 16, then two lane swaps across rows.
__device__ __forceinline__ unsigned row8_max_u32(unsigned v) {
  v = quad_max_u32(v);
  return max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
}
__device__ __forceinline__ unsigned row16_max_u32(unsigned v) {
  v = row8_max_u32(v);
  v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // row_mirror
  return v;
}
__device__ __forceinline__ unsigned wave_max_u32(unsigned v) {
  v = row16_max_u32(v);
  v = max(v, (unsigned)__shfl_xor((int)v, 16));
  v = max(v, (unsigned)__shfl_xor((int)v, 32));
  return v;
}

}  // namespace mxq
