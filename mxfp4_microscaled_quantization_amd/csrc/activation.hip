// The feed-forward layer's activation between its two products, to the input's type or to 8-bit
// codes (the second product's operand), with an 8-bit checkpoint of its input for the backward
// pass, and the gradient from that checkpoint.
//
//   gelu_tanh(u) = u * s(2 sqrt(2 / pi) (u + 0.044715 u^3)),  silu(u) = u * s(u),
//   s(z) = 1 / (1 + exp(-z));
//   du = dy * f'(v),  f'(v) = s + v s (1 - s) dz/du  at v = fl32(code * scale)
// The checkpoint holds u clamped to +-L (4 for gelu_tanh, 8 for silu) by the rule of
// mxq_int8.hpp: beyond L the derivative is within 4e-4 (gelu_tanh) or 3e-3 (silu) of its
// limits 0 and 1, so that an outlier does not coarsen the step, which is at most L / 127,
// for the values whose derivative does vary.
//
// Both are bound by HBM, with the vector units close behind (about 20 operations for each
// element, two of them transcendental).  The forward pass holds a row in registers between its
// maxima and its codes, as the row quantizer does; the backward pass is a plain element kernel.
// 75600 x 13824 bf16, gelu_tanh: 687 us (6.1 TB/s), with a checkpoint 891 (5.9), to codes 560 (5.6, the vector units
// never idle), to codes with a checkpoint 735 (5.7), backward 885 (5.9); a 1 GiB copy reaches 5.0 TB/s.  silu, which
// has fewer operations, to codes 546.
#include <type_traits>

#include "mxq_internal.hpp"
#include "mxq_rows.hpp"

namespace mxq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluB = -2.0f * 0.7978845608028654f * kLog2e;   // exp(-z) = 2^(u (A u^2 + B))
constexpr float kGeluA = kGeluB * 0.044715f;
constexpr float kGeluDz = 2.0f * 0.7978845608028654f;            // dz/du = Dz + Dz2 u^2
constexpr float kGeluDz2 = kGeluDz * 3.0f * 0.044715f;

template <int ACT>
__device__ __forceinline__ constexpr float checkpoint_limit() { return ACT == ACT_GELU_TANH ? 4.0f : 8.0f; }

// exp(-z); infinities at its ends make s(z) 0 or 1
template <int ACT>
__device__ __forceinline__ float exp_minus_z(float u) {
  if constexpr (ACT == ACT_GELU_TANH)
    return __builtin_amdgcn_exp2f(u * __builtin_fmaf(u * u, kGeluA, kGeluB));
  else
    return __builtin_amdgcn_exp2f(u * -kLog2e);
}

template <int ACT>
__device__ __forceinline__ float act(float u) {
  return u * __builtin_amdgcn_rcpf(1.0f + exp_minus_z<ACT>(u));
}

// f' = s + u s (1 - s) z', with 1 - s = e s: no difference of nearly equal numbers.  For |u| up to 2^14 (slope_scale).
template <int ACT>
__device__ __forceinline__ float act_slope(float u) {
  // e stays finite, so that the limit far below is 0 within 2^45 2^-100: u z' s (1 - s) grows as u^3 at most
  const float e = fminf(exp_minus_z<ACT>(u), 0x1p100f), s = __builtin_amdgcn_rcpf(1.0f + e);
  const float t = ACT == ACT_GELU_TANH ? u * __builtin_fmaf(u * u, kGeluDz2, kGeluDz) : u;
  return __builtin_fmaf(t * (e * s), s, s);
}

// The scale of a row of codes for its slopes: clamped to +-128, where a code other than 0 is past the end of the slope's way to
// its limits (at 128 already for the nearest code), and u, up to 2^14, is where act_slope is good.  NaN where it is not finite.
__device__ __forceinline__ float slope_scale(float s) {
  return fabsf(s) < __builtin_inff() ? __builtin_amdgcn_fmed3f(s, -128.0f, 128.0f) : __uint_as_float(0x7FC00000u);
}

// Largest |v| by a floating maximum, which passes over a NaN.  The values are finite where u is (|f(u)| <= |u|), and a row
// whose u is not is told by u's own maximum.
__device__ __forceinline__ float max8(float m, const float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) m = fmaxf(fmaxf(m, fabsf(v[e])), fabsf(v[e + 1]));
  return m;
}

// The scale of the checkpoint of a row whose largest |u| has the pattern `top`: an infinity is clamped like any large
// value, a NaN makes the scale NaN.
template <int ACT>
__device__ __forceinline__ Int8Scale checkpoint_scale(unsigned top) {
  return int8_scale(top > 0x7F800000u ? top : min(top, __float_as_uint(checkpoint_limit<ACT>())));
}

template <bool F32, int ACT>
__device__ __forceinline__ v2u checkpoint_codes(const Unit<F32>& u, const Int8Scale& sc) {
  constexpr float kLimit = checkpoint_limit<ACT>();
  float v[8];
  widen_unit<F32>(u, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_fmed3f(v[e], -kLimit, kLimit);
  return pack_codes(v, sc);
}

// W waves for a row, C units of 8 elements in each thread; W == 1: four rows in a workgroup.
template <bool F32, bool STREAM, bool QUANT, int ACT, int W, int C>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void activation_kernel(ActParams p) {
  constexpr int T = 64 * W, RPB = W < 4 ? 4 / W : 1;
  static_assert(W == 1 || W >= 4, "a workgroup holds whole rows");
  __shared__ unsigned tops[2][2][W];
  const uint32_t tid = threadIdx.x % T, sub = threadIdx.x / T, lane = threadIdx.x & 63, wave = tid >> 6;
  int par = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < p.rows; row += (int64_t)gridDim.x * RPB, par ^= 1) {
    Unit<F32> u[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      u[c] = i < p.units ? load_unit<F32, STREAM>(p.u, row * p.ld_u + (int64_t)i * 8) : zero_unit<F32>();
    }
    unsigned top_u = 0, top_y = 0;
    float most = 0.0f;
    float y[QUANT ? C : 1][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      float(&o)[8] = y[QUANT ? c : 0];
      if (i < p.units) {   // a wave past the row has nothing to compute
        widen_unit<F32>(u[c], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = act<ACT>(o[e]);
        if constexpr (QUANT)
          most = max8(most, o);
        else
          store_out<F32, STREAM>(p.y, row * p.ld_y + (int64_t)i * 8, o, (i | 3) < p.units);
      }
      top_u = max(top_u, unit_max<F32>(u[c]));
    }
    if (QUANT || p.kept) {
      top_y = __float_as_uint(most);
      if constexpr (QUANT) top_y = group_max<64>(top_y);
      top_u = group_max<64>(top_u);
      if constexpr (W > 1) {
        // two slots in turn: a wave may reach the next row's store while another still reads
        if (lane == 0) {
          tops[par][0][wave] = top_y;
          tops[par][1][wave] = top_u;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < W; ++k) {
          top_y = max(top_y, tops[par][0][k]);
          top_u = max(top_u, tops[par][1][k]);
        }
      }
    }
    if constexpr (QUANT) {
      const Int8Scale sc = int8_scale(top_u < 0x7F800000u ? top_y : top_u);
      if (tid == 0) p.scales[row] = sc.s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        if (i < p.units)
          __builtin_nontemporal_store(pack_codes(y[c], sc),
                                      reinterpret_cast<v2u*>(static_cast<int8_t*>(p.y) + row * p.ld_y + (int64_t)i * 8));
      }
    }
    if (p.kept) {
      const Int8Scale sc = checkpoint_scale<ACT>(top_u);
      if (tid == 0) p.kept_scales[row] = sc.s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        if (i < p.units)
          __builtin_nontemporal_store(checkpoint_codes<F32, ACT>(u[c], sc), reinterpret_cast<v2u*>(p.kept + row * p.ld_kept + (int64_t)i * 8));
      }
    }
  }
}

// Rows of up to G units, 64 / G of them in a wave: lane l of a group has unit l, R rows of each group in flight.
template <bool F32, bool STREAM, bool QUANT, int ACT, int G>
__global__ __launch_bounds__(256) void activation_short_kernel(ActParams p) {
  constexpr int PER = 256 / G, R = 4;   // rows of the workgroup at once, passes in flight
  const uint32_t l = threadIdx.x % G;
  const bool own = l < p.units;
  for (int64_t r0 = (int64_t)blockIdx.x * (PER * R) + threadIdx.x / G; r0 < p.rows; r0 += (int64_t)gridDim.x * (PER * R)) {
    Unit<F32> u[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t row = r0 + k * PER;
      u[k] = own && row < p.rows ? load_unit<F32, STREAM>(p.u, row * p.ld_u + (int64_t)l * 8) : zero_unit<F32>();
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t row = r0 + k * PER;
      const bool in = own && row < p.rows;
      const unsigned top_u = group_max<G>(unit_max<F32>(u[k]));
      float o[8];
      widen_unit<F32>(u[k], o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = act<ACT>(o[e]);
      if constexpr (QUANT) {
        const unsigned top_y = group_max<G>(__float_as_uint(max8(0.0f, o)));
        const Int8Scale sc = int8_scale(top_u < 0x7F800000u ? top_y : top_u);
        if (l == 0 && row < p.rows) p.scales[row] = sc.s;
        if (in)
          __builtin_nontemporal_store(pack_codes(o, sc), reinterpret_cast<v2u*>(static_cast<int8_t*>(p.y) + row * p.ld_y + (int64_t)l * 8));
      } else if (in) {
        store_out<F32, STREAM>(p.y, row * p.ld_y + (int64_t)l * 8, o, (l | 3) < p.units);
      }
      if (p.kept) {
        const Int8Scale sc = checkpoint_scale<ACT>(top_u);
        if (l == 0 && row < p.rows) p.kept_scales[row] = sc.s;
        if (in)
          __builtin_nontemporal_store(checkpoint_codes<F32, ACT>(u[k], sc), reinterpret_cast<v2u*>(p.kept + row * p.ld_kept + (int64_t)l * 8));
      }
    }
  }
}

constexpr int kActGradThreads = 256;
constexpr int kActGradUnroll = 4;

template <bool F32, int ACT>
__global__ __launch_bounds__(kActGradThreads) void activation_backward_kernel(ActGradParams p) {
  const uint64_t stride = (uint64_t)gridDim.x * kActGradThreads * kActGradUnroll;
  for (uint64_t g0 = (uint64_t)blockIdx.x * kActGradThreads * kActGradUnroll + threadIdx.x; g0 < p.total; g0 += stride) {
    Unit<F32> d[kActGradUnroll];
    v2u c[kActGradUnroll];
    float s[kActGradUnroll];
    uint32_t row[kActGradUnroll], col[kActGradUnroll];
    bool ok[kActGradUnroll];
#pragma unroll
    for (int k = 0; k < kActGradUnroll; ++k) {
      const uint64_t g64 = g0 + (uint64_t)k * kActGradThreads;
      ok[k] = g64 < p.total;
      const uint32_t g = ok[k] ? (uint32_t)g64 : 0u;
      row[k] = g / p.units;
      col[k] = (g - row[k] * p.units) * 8u;
      d[k] = load_unit<F32, true>(p.dy, row[k] * p.ld_dy + col[k]);
      c[k] = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(p.kept + row[k] * p.ld_kept + col[k]));
      s[k] = p.kept_scales[row[k]];
    }
#pragma unroll
    for (int k = 0; k < kActGradUnroll; ++k) {
      float v[8], o[8];
      widen_codes(c[k], slope_scale(s[k]), v);
      widen_unit<F32>(d[k], o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= act_slope<ACT>(v[e]);
      // whole quads of units in each row (60000 x 1040, of 130 units: 106 us, quad by quad 111)
      if (ok[k]) store_out<F32, true>(p.dx, row[k] * p.ld_dx + col[k], o, p.units % 4 == 0);
    }
  }
}

}  // namespace

hipError_t launch_activation(const ActParams& p, bool f32, bool quant, ActKind act, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  auto go = [&](auto kernel, int threads, int rows_per_block) {
    const int64_t blocks = (p.rows + rows_per_block - 1) / rows_per_block;
    const int64_t cap = (int64_t)1 << 20;   // blocks * threads stays below 2^32
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(threads), 0, stream, p);
  };
  auto pick = [&](auto f_tag, auto s_tag, auto q_tag, auto a_tag) {
    constexpr bool F = decltype(f_tag)::value, S = decltype(s_tag)::value, Q = decltype(q_tag)::value;
    constexpr int A = decltype(a_tag)::value;
    auto longest = [&] {
      if (p.units <= 1024 * 4)
        go(activation_kernel<F, S, Q, A, 16, 4>, 1024, 1);
      else
        go(activation_kernel<F, S, Q, A, 16, 8>, 1024, 1);
    };
    // The waves of a row, us at 13824 columns and more rows than the GPU holds unless said otherwise.  Up to 32 units several
    // rows share a wave (150000 x 256 bf16 to codes 24, a wave for each row 39).  A row's codes wait in registers for its
    // scales, which every wave has to work out: few waves of longer threads (75600 rows bf16 557, over 16 waves 872; 40000 x
    // 2048 38, over 4 waves 46).  A result that is stored at once has nothing to wait for: more waves, in binary32 of one
    // unit a thread as far as that goes (30000 x 4096 174, over 4 waves 185), in bf16, whose codes beside the result
    // are packed for each wave, of three from 4096 to 6144 columns and from 8192 to 12288 (20000 x 4112 with codes 73, of two 88;
    // plain 55 and 55) and of two or one elsewhere (40000 x 2048 52, over one wave 60; 20000 x 6160 86, of four 90).
    if (p.units <= 8)
      go(activation_short_kernel<F, S, Q, A, 8>, 256, 32 * 4);
    else if (p.units <= 16)
      go(activation_short_kernel<F, S, Q, A, 16>, 256, 16 * 4);
    else if (p.units <= 32)
      go(activation_short_kernel<F, S, Q, A, 32>, 256, 8 * 4);
    else if (p.units <= 64)
      go(activation_kernel<F, S, Q, A, 1, 1>, 256, 4);
    else if (p.units <= 128)
      go(activation_kernel<F, S, Q, A, 1, 2>, 256, 4);
    else if (p.units <= 192)
      go(activation_kernel<F, S, Q, A, 1, 3>, 256, 4);
    else if constexpr (Q) {
      if (p.units <= 256)
        go(activation_kernel<F, S, Q, A, 1, 4>, 256, 4);
      else if (p.units <= 256 * 2)
        go(activation_kernel<F, S, Q, A, 4, 2>, 256, 1);
      else if (p.units <= 256 * 3)
        go(activation_kernel<F, S, Q, A, 4, 3>, 256, 1);
      else if (p.units <= 256 * 4)
        go(activation_kernel<F, S, Q, A, 4, 4>, 256, 1);
      else if (p.units <= 512 * 3)
        go(activation_kernel<F, S, Q, A, 8, 3>, 512, 1);
      else if (p.units <= 512 * 4)
        go(activation_kernel<F, S, Q, A, 8, 4>, 512, 1);
      else
        longest();
    } else if constexpr (F) {
      if (p.units <= 256)
        go(activation_kernel<F, S, Q, A, 4, 1>, 256, 1);
      else if (p.units <= 512)
        go(activation_kernel<F, S, Q, A, 8, 1>, 512, 1);
      else if (p.units <= 512 * 2)
        go(activation_kernel<F, S, Q, A, 8, 2>, 512, 1);
      else if (p.units <= 1024 * 2)
        go(activation_kernel<F, S, Q, A, 16, 2>, 1024, 1);
      else
        longest();
    } else {
      if (p.units <= 256)
        go(activation_kernel<F, S, Q, A, 4, 1>, 256, 1);
      else if (p.units <= 256 * 2)
        go(activation_kernel<F, S, Q, A, 4, 2>, 256, 1);
      else if (p.units <= 256 * 3)
        go(activation_kernel<F, S, Q, A, 4, 3>, 256, 1);
      else if (p.units <= 512 * 2)
        go(activation_kernel<F, S, Q, A, 8, 2>, 512, 1);
      else if (p.units <= 512 * 3)
        go(activation_kernel<F, S, Q, A, 8, 3>, 512, 1);
      else if (p.units <= 1024 * 2)
        go(activation_kernel<F, S, Q, A, 16, 2>, 1024, 1);
      else
        longest();
    }
  };
  // see launch_quantize_int8
  const bool stream_loads = p.rows * (int64_t)p.units * 8 * (f32 ? 4 : 2) > ((int64_t)256 << 20);
  using T = std::true_type;
  using N = std::false_type;
  auto a = [&](auto f, auto s, auto q) {
    if (act == ACT_GELU_TANH)
      pick(f, s, q, std::integral_constant<int, ACT_GELU_TANH>{});
    else
      pick(f, s, q, std::integral_constant<int, ACT_SILU>{});
  };
  auto q = [&](auto f, auto s) { quant ? a(f, s, T{}) : a(f, s, N{}); };
  auto s = [&](auto f) { stream_loads ? q(f, T{}) : q(f, N{}); };
  f32 ? s(T{}) : s(N{});
  return hipGetLastError();
}

hipError_t launch_activation_backward(const ActGradParams& p, bool f32, ActKind act, hipStream_t stream) {
  if (p.total == 0) return hipSuccess;
  const int64_t per = (int64_t)kActGradThreads * kActGradUnroll, cap = (int64_t)1 << 20;
  const int64_t blocks = ((int64_t)p.total + per - 1) / per;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(kActGradThreads), 0, stream, p);
  };
  if (act == ACT_GELU_TANH)
    f32 ? go(activation_backward_kernel<true, ACT_GELU_TANH>) : go(activation_backward_kernel<false, ACT_GELU_TANH>);
  else
    f32 ? go(activation_backward_kernel<true, ACT_SILU>) : go(activation_backward_kernel<false, ACT_SILU>);
  return hipGetLastError();
}

}  // namespace mxq
