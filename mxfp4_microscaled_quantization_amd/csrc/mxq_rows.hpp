// Helpers of the kernels that take a row of a matrix as units of 8 elements (layer_norm.hip,
// activation.hip): a unit as 8 binary32 values and back, and sums over the lanes of a wave.
#pragma once

#include <type_traits>

#include "mxq_int8.hpp"

namespace mxq {

template <bool F32>
__device__ __forceinline__ void widen_unit(const Unit<F32>& u, float (&v)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __int_as_float(u.d[0][e]);
      v[4 + e] = __int_as_float(u.d[1][e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf16_lo_f32(u.d[0][e]);
      v[2 * e + 1] = bf16_hi_f32(u.d[0][e]);
    }
  }
}

// Hides from the compiler that a unit is what it was: it is then widened again where it is used, instead of
// being held widened from one pass to the next.
template <bool F32>
__device__ __forceinline__ void forget_unit(Unit<F32>& u) {
  asm volatile("" : "+v"(u.d[0]));
  if constexpr (F32) asm volatile("" : "+v"(u.d[1]));
}

// Rounds once, to nearest even, where the output is bf16.  PAST: stored past the caches.
template <bool F32, bool PAST>
__device__ __forceinline__ void store_unit(void* y, int64_t elem, const float (&v)[8]) {
  auto put = [](v4i* p, v4i d) {
    if constexpr (PAST)
      __builtin_nontemporal_store(d, p);
    else
      *p = d;
  };
  if constexpr (F32) {
    v4i* p = reinterpret_cast<v4i*>(static_cast<float*>(y) + elem);
    put(p, v4i{__float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3])});
    put(p + 1, v4i{__float_as_int(v[4]), __float_as_int(v[5]), __float_as_int(v[6]), __float_as_int(v[7])});
  } else {
    put(reinterpret_cast<v4i*>(static_cast<uint16_t*>(y) + elem),
        v4i{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]), (int)pack_bf16x2(v[4], v[5]),
            (int)pack_bf16x2(v[6], v[7])});
  }
}

// store_unit, where `quad` says that the 4 lanes of this one's quad hold 4 consecutive units and are all here (they agree
// on it).  In binary32 a lane's unit is two pieces of 16 bytes, and each of two plain stores past the caches would leave
// every second piece for the other: the quad's pieces change places, and each store writes 64 bytes in a run (layer norm's
// gradient, 75600 x 5120: 1749 MB written of 1548, 924 us; so 878).
template <bool F32, bool PAST>
__device__ __forceinline__ void store_out(void* y, int64_t elem, const float (&v)[8], bool quad) {
  if constexpr (F32 && PAST) {
    if (quad) {
      const int l = (int)threadIdx.x & 3;
      v4i first, second;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int lo = __float_as_int(v[e]), hi = __float_as_int(v[4 + e]);
        // of lanes 0 0 1 1, and of lanes 2 2 3 3
        const int lo0 = __builtin_amdgcn_update_dpp(0, lo, 0x50, 0xF, 0xF, true), hi0 = __builtin_amdgcn_update_dpp(0, hi, 0x50, 0xF, 0xF, true);
        const int lo1 = __builtin_amdgcn_update_dpp(0, lo, 0xFA, 0xF, 0xF, true), hi1 = __builtin_amdgcn_update_dpp(0, hi, 0xFA, 0xF, 0xF, true);
        first[e] = l & 1 ? hi0 : lo0;
        second[e] = l & 1 ? hi1 : lo1;
      }
      v4i* p = reinterpret_cast<v4i*>(static_cast<float*>(y) + elem - l * 4);
      __builtin_nontemporal_store(first, p);
      __builtin_nontemporal_store(second, p + 4);
      return;
    }
  }
  store_unit<F32, PAST>(y, elem, v);
}

// The 8 codes of a unit as values fl32(code * scale): the product is rounded by itself, also where a sum follows.
__device__ __forceinline__ void widen_codes(v2u c, float s, float (&v)[8]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * h + e] = (float)(int8_t)(c[h] >> (8 * e)) * s;
}

__device__ __forceinline__ v2u pack_codes(const float (&v)[8], const Int8Scale& sc) {
  return v2u{int8_pack4(v[0], v[1], v[2], v[3], sc.inv) & sc.keep, int8_pack4(v[4], v[5], v[6], v[7], sc.inv) & sc.keep};
}

// Largest |v| as a binary32 pattern: a NaN wins over an infinity, which wins over finite values.
__device__ __forceinline__ unsigned max_abs8(const float (&v)[8]) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return m;
}

// Sum over each row of 16 lanes, the same bits in every lane.
__device__ __forceinline__ float row16_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});    // lane ^ 1
  v += dpp(v, std::integral_constant<int, 0x4E>{});    // lane ^ 2
  v += dpp(v, std::integral_constant<int, 0x141>{});   // row_half_mirror: the other quad of 8
  v += dpp(v, std::integral_constant<int, 0x140>{});   // row_mirror: the other 8 of 16
  return v;
}

// Lane i of the lower half gets a[i] + a[i + 32], lane i of the upper one b[i] + b[i - 32].
__device__ __forceinline__ float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The same with rows of 16 lanes: rows 0 and 2 get a of their own and of the next row, rows 1 and 3 b of the row before
// and of their own.
__device__ __forceinline__ float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over each group of G lanes (8 to 64), the same bits in every lane of it.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  static_assert(G >= 8, "whole halves of rows");
  if constexpr (G >= 64) v = fold32(v, v);
  if constexpr (G >= 32) v = fold16(v, v);
  if constexpr (G >= 16) return row16_sum(v);
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});
  v += dpp(v, std::integral_constant<int, 0x4E>{});
  return v + dpp(v, std::integral_constant<int, 0x141>{});
}
__device__ __forceinline__ float wave_sum(float v) { return group_sum<64>(v); }

// Sums over the wave of two values: a's in the lower half's lanes, b's in the upper half's.
__device__ __forceinline__ float wave_sum2(float a, float b) {
  const float t = fold32(a, b);
  return row16_sum(fold16(t, t));
}
// Of four: a's in row 0 of 16 lanes, c's in row 1, b's in row 2, d's in row 3.
__device__ __forceinline__ float wave_sum4(float a, float b, float c, float d) { return row16_sum(fold16(fold32(a, b), fold32(c, d))); }

// Lane `lane` of v, as a scalar.
__device__ __forceinline__ float of_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Max over each group of G lanes, in every lane.
template <int G>
__device__ __forceinline__ unsigned group_max(unsigned v) {
  v = G >= 16 ? row16_max_u32(v) : row8_max_u32(v);
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
  }
  if constexpr (G >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(r[0], r[1]);
  }
  return v;
}

// Sum of a unit's elements onto s.  Two bf16 in one instruction, which flushes subnormal numbers.
template <bool F32>
__device__ __forceinline__ float sum_unit(const Unit<F32>& u, float s) {
  if constexpr (F32) {
    float v[8];
    widen_unit<true>(u, v);
    return s + (((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7])));
  } else {
    const bf16x2 one = __builtin_bit_cast(bf16x2, 0x3F803F80u);
#pragma unroll
    for (int k = 0; k < 4; ++k) s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u.d[0][k]), one, s, false);
    return s;
  }
}

// a * b as a binary32 value, the same wherever it is used: not contracted into one of the sums that it is a part of.
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// s / n, rounded correctly but for rare last bits, from inv = fl32(1 / n); exact where n divides s.
__device__ __forceinline__ float quotient(float s, float n, float inv) {
  const float q = s * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, n, s), inv, q);
}

}  // namespace mxq
