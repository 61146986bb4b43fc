// Root-mean-square norm of every query and key head with the position rotation in the same
// pass, for the output of a QKV projection; the result in the input's type, or as 8-bit
// codes with one scale for each token and head (mxq_int8.hpp).
//
// For a head x of D elements, all in binary32, rounded once at the end:
//   r = 1 / sqrt(sum x^2 / D + eps),  y = (x * r) * w
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first R elements,
// (2i, 2i+1) interleaved or (i, i + R/2) by halves, with cos / sin of row position[token].
//
// HBM-bound: every element is read and written once.  G lanes own a head (8 elements
// each; the smallest power of two that covers D), so a wave holds 64 / G heads of one token
// at a time and U such sets in flight; the reduction is DPP and lane swaps inside the G
// lanes.  A lane's 8 elements are 4 whole pairs: consecutive ones when interleaved, 4 from
// each half otherwise, so that no partner has to be fetched from another lane.  cos and sin
// are loaded once for a token and kept over its heads.
#include <type_traits>

#include "mxq_int8.hpp"
#include "mxq_internal.hpp"

namespace mxq {
namespace {

constexpr int kQkWaves = 4;   // waves per workgroup, one token each

template <int G>
__device__ __forceinline__ float group_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});    // lane ^ 1
  v += dpp(v, std::integral_constant<int, 0x4E>{});    // lane ^ 2
  v += dpp(v, std::integral_constant<int, 0x141>{});   // row_half_mirror: the other quad of 8
  if constexpr (G >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});   // row_mirror: the other 8 of 16
  if constexpr (G >= 32) v += __shfl_xor(v, 16);
  if constexpr (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

template <int G>
__device__ __forceinline__ unsigned group_max(unsigned v) {
  v = quad_max_u32(v);
  v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
  if constexpr (G >= 16) v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
  if constexpr (G >= 32) v = max(v, (unsigned)__shfl_xor((int)v, 16));
  if constexpr (G >= 64) v = max(v, (unsigned)__shfl_xor((int)v, 32));
  return v;
}

// 4 elements of a row at element offset e, as binary32
template <bool F32>
__device__ __forceinline__ v4f load4(const void* x, int64_t e) {
  if constexpr (F32) {
    return *reinterpret_cast<const v4f*>(static_cast<const float*>(x) + e);
  } else {
    const v2u d = *reinterpret_cast<const v2u*>(static_cast<const uint16_t*>(x) + e);
    return v4f{bf16_lo_f32((int)d[0]), bf16_hi_f32((int)d[0]), bf16_lo_f32((int)d[1]), bf16_hi_f32((int)d[1])};
  }
}

// F32: type of x and of the unquantized output; QUANT: 8-bit codes and scales instead;
// HALVES: pairs (i, i + R/2); U: sets of 64 / G heads in flight.
template <int G, bool F32, bool QUANT, bool HALVES, int U>
__global__ __launch_bounds__(64 * kQkWaves) void qk_norm_rope_kernel(QkNormParams p) {
  constexpr int HPS = 64 / G;   // heads per set
  const int lane = threadIdx.x & 63, l = lane % G, sub = lane / G;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int heads = p.q.heads + p.k.heads;
  const bool own = 8 * l < p.head_dim, turned = 8 * l < p.rot_dim;
  // element offsets of this lane's two runs of 4
  const int e0 = HALVES && turned ? 4 * l : 8 * l, e1 = HALVES && turned ? p.rot_dim / 2 + 4 * l : 8 * l + 4;

  auto weights = [&](const void* w, v4f(&o)[2]) {
    o[0] = o[1] = v4f{1.0f, 1.0f, 1.0f, 1.0f};
    if (w && own) {
      o[0] = p.w_f32 ? load4<true>(w, e0) : load4<false>(w, e0);
      o[1] = p.w_f32 ? load4<true>(w, e1) : load4<false>(w, e1);
    }
  };
  v4f wq[2], wk[2];
  weights(p.q.w, wq);
  weights(p.k.w, wk);

  for (int64_t t = (int64_t)blockIdx.x * kQkWaves + wave; t < p.tokens; t += (int64_t)gridDim.x * kQkWaves) {
    v4f c = {1.0f, 1.0f, 1.0f, 1.0f}, s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (turned) {
      const int64_t pos = p.positions ? p.positions[t] : t;
      if (pos >= 0 && pos < p.table_rows) {
        c = *reinterpret_cast<const v4f*>(p.cos + pos * p.ld_table + 4 * l);
        s = *reinterpret_cast<const v4f*>(p.sin + pos * p.ld_table + 4 * l);
      } else {
        const float nan = __uint_as_float(0x7FC00000u);
        c = s = v4f{nan, nan, nan, nan};
      }
    }
    for (int h0 = blockIdx.y * (HPS * U); h0 < heads; h0 += gridDim.y * (HPS * U)) {
      v4f x[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * HPS + sub;
        const bool is_q = h < p.q.heads;
        const void* xs = is_q ? p.q.x : p.k.x;
        const int64_t at = is_q ? t * p.q.ld_x + h * p.q.hs_x : t * p.k.ld_x + (h - p.q.heads) * p.k.hs_x;
        x[u][0] = x[u][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (own && h < heads) {
          x[u][0] = load4<F32>(xs, at + e0);
          x[u][1] = load4<F32>(xs, at + e1);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * HPS + sub;
        const bool is_q = h < p.q.heads;
        void* out = is_q ? p.q.out : p.k.out;
        const int64_t at = is_q ? t * p.q.ld_o + h * p.q.hs_o : t * p.k.ld_o + (h - p.q.heads) * p.k.hs_o;
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss += x[u][0][e] * x[u][0][e] + x[u][1][e] * x[u][1][e];
        const float r = rsqrtf(group_sum<G>(ss) * p.inv_dim + p.eps);
        float y[2][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[b][e] = x[u][b][e] * r * (is_q ? wq[b][e] : wk[b][e]);
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& a = HALVES ? y[0][i] : y[i >> 1][2 * (i & 1)];
            float& b = HALVES ? y[1][i] : y[i >> 1][2 * (i & 1) + 1];
            const float a0 = a, b0 = b;
            a = a0 * c[i] - b0 * s[i];
            b = b0 * c[i] + a0 * s[i];
          }
        }
        if constexpr (QUANT) {
          unsigned m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m = max(m, max(__float_as_uint(y[0][e]) & 0x7FFFFFFFu, __float_as_uint(y[1][e]) & 0x7FFFFFFFu));
          const Int8Scale sc = int8_scale(group_max<G>(m));
          if (h < heads) {
            if (l == 0) {
              if (is_q)
                p.q.scales[t * p.q.ld_s + h] = sc.s;
              else
                p.k.scales[t * p.k.ld_s + (h - p.q.heads)] = sc.s;
            }
            if (own) {
              int8_t* o = static_cast<int8_t*>(out) + at;
              const unsigned lo = int8_pack4(y[0][0], y[0][1], y[0][2], y[0][3], sc.inv) & sc.keep;
              const unsigned hi = int8_pack4(y[1][0], y[1][1], y[1][2], y[1][3], sc.inv) & sc.keep;
              if constexpr (HALVES) {
                *reinterpret_cast<unsigned*>(o + e0) = lo;
                *reinterpret_cast<unsigned*>(o + e1) = hi;
              } else {
                *reinterpret_cast<v2u*>(o + e0) = v2u{lo, hi};
              }
            }
          }
        } else if (own && h < heads) {
          if constexpr (F32) {
            float* o = static_cast<float*>(out) + at;
            *reinterpret_cast<v4f*>(o + e0) = v4f{y[0][0], y[0][1], y[0][2], y[0][3]};
            *reinterpret_cast<v4f*>(o + e1) = v4f{y[1][0], y[1][1], y[1][2], y[1][3]};
          } else {
            uint16_t* o = static_cast<uint16_t*>(out) + at;
            const v2u lo = {pack_bf16x2(y[0][0], y[0][1]), pack_bf16x2(y[0][2], y[0][3])};
            const v2u hi = {pack_bf16x2(y[1][0], y[1][1]), pack_bf16x2(y[1][2], y[1][3])};
            if constexpr (HALVES) {
              *reinterpret_cast<v2u*>(o + e0) = lo;
              *reinterpret_cast<v2u*>(o + e1) = hi;
            } else {
              *reinterpret_cast<v4u*>(o + e0) = v4u{lo[0], lo[1], hi[0], hi[1]};
            }
          }
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormParams& p, bool f32, bool quant, bool halves, hipStream_t stream) {
  const int heads = p.q.heads + p.k.heads;
  if (p.tokens == 0 || heads == 0) return hipSuccess;
  auto go = [&](auto g_tag, auto f_tag, auto q_tag, auto h_tag, auto u_tag) {
    constexpr int G = decltype(g_tag)::value, U = decltype(u_tag)::value, SET = 64 / G * U;
    int64_t gx = (p.tokens + kQkWaves - 1) / kQkWaves;
    const int chunks = (heads + SET - 1) / SET;
    if (gx > ((int64_t)1 << 20)) gx = (int64_t)1 << 20;
    // a few tokens: their heads over several workgroups; else one wave takes a whole token
    const int gy = U == 1 ? (chunks < 65535 ? chunks : 65535) : 1;
    hipLaunchKernelGGL((qk_norm_rope_kernel<G, decltype(f_tag)::value, decltype(q_tag)::value, decltype(h_tag)::value, U>),
                       dim3((unsigned)gx, (unsigned)gy), dim3(64 * kQkWaves), 0, stream, p);
  };
  using T = std::true_type;
  using F = std::false_type;
  auto u = [&](auto g, auto f, auto q, auto h) {
    if (p.tokens < 512)
      go(g, f, q, h, std::integral_constant<int, 1>{});
    else
      go(g, f, q, h, std::integral_constant<int, 4>{});
  };
  auto h = [&](auto g, auto f, auto q) { halves ? u(g, f, q, T{}) : u(g, f, q, F{}); };
  auto q = [&](auto g, auto f) { quant ? h(g, f, T{}) : h(g, f, F{}); };
  auto f = [&](auto g) { f32 ? q(g, T{}) : q(g, F{}); };
  if (p.head_dim <= 64)
    f(std::integral_constant<int, 8>{});
  else if (p.head_dim <= 128)
    f(std::integral_constant<int, 16>{});
  else if (p.head_dim <= 256)
    f(std::integral_constant<int, 32>{});
  else
    f(std::integral_constant<int, 64>{});
  return hipGetLastError();
}

}  // namespace mxq
