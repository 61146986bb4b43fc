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

// 8 elements of a row as loaded: 16 bytes of bf16, or twice 16 bytes of binary32
template <bool F32> struct Unit {
  v4i d[F32 ? 2 : 1];
};

// STREAM: loads past the caches, for inputs that do not fit them (see launch_quantize_int8)
template <bool F32, bool STREAM>
__device__ __forceinline__ Unit<F32> load_unit(const void* x, int64_t elem) {
  auto get = [](const v4i* p) { return STREAM ? __builtin_nontemporal_load(p) : *p; };
  Unit<F32> u;
  if constexpr (F32) {
    const v4i* p = reinterpret_cast<const v4i*>(static_cast<const float*>(x) + elem);
    u.d[0] = get(p);
    u.d[1] = get(p + 1);
  } else {
    u.d[0] = get(reinterpret_cast<const v4i*>(static_cast<const uint16_t*>(x) + elem));
  }
  return u;
}

template <bool F32>
__device__ __forceinline__ Unit<F32> zero_unit() {
  Unit<F32> u;
  u.d[0] = v4i{0, 0, 0, 0};
  if constexpr (F32) u.d[1] = v4i{0, 0, 0, 0};
  return u;
}

// max |x| of a unit as a binary32 pattern
template <bool F32>
__device__ __forceinline__ unsigned unit_max(const Unit<F32>& u) {
  if constexpr (F32) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((unsigned)u.d[0][i] & 0x7FFFFFFFu, (unsigned)u.d[1][i] & 0x7FFFFFFFu));
    return m;
  } else {
    v2h m = abs_bf16x2(u.d[0][0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, abs_bf16x2(u.d[0][i]));
    return max((unsigned)m[0], (unsigned)m[1]) << 16;
  }
}

template <bool F32>
__device__ __forceinline__ v2u unit_codes(const Unit<F32>& u, const Int8Scale& sc) {
  v2u o;
  if constexpr (F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o[h] = int8_pack4(__int_as_float(u.d[h][0]), __int_as_float(u.d[h][1]), __int_as_float(u.d[h][2]),
                        __int_as_float(u.d[h][3]), sc.inv) & sc.keep;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o[h] = int8_pack4(bf16_lo_f32(u.d[0][2 * h]), bf16_hi_f32(u.d[0][2 * h]), bf16_lo_f32(u.d[0][2 * h + 1]),
                        bf16_hi_f32(u.d[0][2 * h + 1]), sc.inv) & sc.keep;
  }
  return o;
}

}  // namespace mxq
