// Root-mean-square norm of every query and key head with the position rotation in the same
// pass, for the output of a QKV projection; the result in the input's type, or as 8-bit
// codes with one scale for each token and head (mxq_int8.hpp).
//
// For a head x of D elements, all in binary32, rounded once at the end:
//   r = 1 / sqrt(sum x^2 / D + eps),  y = (x * r) * w
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first R elements,
// (2i, 2i+1) interleaved or (i, i + R/2) by halves, with cos / sin of row position[token].
//
// HBM-bound: every element is read and written once, so what counts is that a wave spends
// few instructions on each.  G lanes own a head (8 elements each; the smallest power of two
// that covers D); a wave takes one token's queries or its keys, 64 / G heads at a time and
// U such sets in flight, with the token's cos and sin and the weights in registers and its
// heads addressed through buffer resources by one scalar offset.  The reduction is DPP and
// lane swaps inside the G lanes.  A lane's 8 elements are 4 whole pairs: consecutive ones
// when interleaved, 4 from each half otherwise, so no partner comes from another lane.  Tokens of
// few heads would leave most of such a wave empty: there a wave takes pairs (token, head).
// Measured, 75600 tokens x (40 + 40) heads x 128 in bf16: 0.555 ms in either style, 5.6 TB/s (0.61 ms
// with 64-bit addresses for each lane and queries and keys in one loop), to 8-bit codes 0.42 ms
// interleaved and 0.43 by halves, 5.4 to 5.6 TB/s.  In binary32 by halves 1.13 ms, 5.5 TB/s, to codes
// 0.70 ms; interleaved to codes 0.72 ms, but to binary32 1.75 ms, 3.5 TB/s: a lane's two runs of 16
// bytes then lie side by side, so that each store instruction writes every other 16 bytes past the
// caches, and the memory is written 1.6 times.  57344 x (24 + 24) x 128 bf16 to codes 0.194 ms, 5.4
// TB/s; 32768 x (32 + 8) x 128 by halves 0.117 ms, 5.7 TB/s, to codes 0.099.
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

constexpr uint32_t kOutsideHead = 0x80000000u;   // a byte offset past every resource here
constexpr int kNt = 2;                           // non-temporal: every element is used once

__device__ __forceinline__ v4f widen4(v2u d) {
  return v4f{bf16_lo_f32((int)d[0]), bf16_hi_f32((int)d[0]), bf16_lo_f32((int)d[1]), bf16_hi_f32((int)d[1])};
}

// A lane's two runs of 4 elements of a head, at byte offsets o0 and o1 (o1 follows o0 when
// APART is false).
template <bool F32, bool APART>
__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, uint32_t base, v4f (&x)[2]) {
  if constexpr (F32) {
    x[0] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, o0, base, kNt));
    x[1] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, o1, base, kNt));
  } else if constexpr (APART) {
    x[0] = widen4(__builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(r, o0, base, kNt)));
    x[1] = widen4(__builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(r, o1, base, kNt)));
  } else {
    const v4u d = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(r, o0, base, kNt));
    x[0] = widen4(v2u{d[0], d[1]});
    x[1] = widen4(v2u{d[2], d[3]});
  }
}

// Element offsets of a lane's two runs of 4 in its head.
template <bool HALVES>
__device__ __forceinline__ uint32_t run0(int l, bool turned) { return HALVES && turned ? 4 * l : 8 * l; }
template <bool HALVES>
__device__ __forceinline__ uint32_t run1(const QkNormParams& p, int l, bool turned) {
  return HALVES && turned ? p.rot_dim / 2 + 4 * l : 8 * l + 4;
}

__device__ __forceinline__ void load_weights(const QkNormParams& p, const void* w, bool own, uint32_t e0, uint32_t e1, v4f (&o)[2]) {
  o[0] = o[1] = v4f{1.0f, 1.0f, 1.0f, 1.0f};
  if (w && own) {
    if (p.w_f32) {
      o[0] = *reinterpret_cast<const v4f*>(static_cast<const float*>(w) + e0);
      o[1] = *reinterpret_cast<const v4f*>(static_cast<const float*>(w) + e1);
    } else {
      o[0] = widen4(*reinterpret_cast<const v2u*>(static_cast<const uint16_t*>(w) + e0));
      o[1] = widen4(*reinterpret_cast<const v2u*>(static_cast<const uint16_t*>(w) + e1));
    }
  }
}

// cos and sin of a lane's 4 pairs at position pos.
__device__ __forceinline__ void load_turn(const QkNormParams& p, int64_t pos, int l, v4f& c, v4f& s) {
  if (pos >= 0 && pos < p.table_rows) {
    c = *reinterpret_cast<const v4f*>(p.cos + pos * p.ld_table + 4 * l);
    s = *reinterpret_cast<const v4f*>(p.sin + pos * p.ld_table + 4 * l);
  } else {
    const float nan = __uint_as_float(0x7FC00000u);
    c = s = v4f{nan, nan, nan, nan};
  }
}

// A head's norm and rotation, over the G lanes that hold it.
template <int G, bool HALVES>
__device__ __forceinline__ void norm_and_turn(const QkNormParams& p, const v4f (&x)[2], const v4f (&w)[2], v4f c, v4f s, bool turned, float (&y)[2][4]) {
  float ss = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) ss = __builtin_fmaf(x[1][e], x[1][e], __builtin_fmaf(x[0][e], x[0][e], ss));
  const float r = rsqrtf(__builtin_fmaf(group_sum<G>(ss), p.inv_dim, p.eps));
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[b][e] = x[b][e] * r * w[b][e];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float& a = HALVES ? y[0][i] : y[i >> 1][2 * (i & 1)];
      float& b = HALVES ? y[1][i] : y[i >> 1][2 * (i & 1) + 1];
      const float a0 = a, b0 = b;
      a = __builtin_fmaf(a0, c[i], -(b0 * s[i]));
      b = __builtin_fmaf(a0, s[i], b0 * c[i]);
    }
  }
}

// The scale of a head's codes, over its G lanes.
template <int G>
__device__ __forceinline__ Int8Scale head_scale(const float (&y)[2][4]) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    m = max(m, max(__float_as_uint(y[0][e]) & 0x7FFFFFFFu, __float_as_uint(y[1][e]) & 0x7FFFFFFFu));
  return int8_scale(group_max<G>(m));
}

__device__ __forceinline__ v2u pack4(const float (&y)[4]) { return v2u{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])}; }

// F32: type of x and of the unquantized output; QUANT: 8-bit codes and scales instead;
// HALVES: pairs (i, i + R/2); U: sets of 64 / G heads in flight.
template <int G, bool F32, bool QUANT, bool HALVES, int U>
__global__ __launch_bounds__(64 * kQkWaves) void qk_norm_rope_kernel(QkNormParams p) {
  constexpr int HPS = 64 / G;                                  // heads per set
  constexpr uint32_t IB = F32 ? 4 : 2, OB = QUANT ? 1 : IB;    // bytes of an element in and out
  const int lane = threadIdx.x & 63, l = lane % G, sub = lane / G;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const bool own = 8 * l < p.head_dim, turned = 8 * l < p.rot_dim;
  const uint32_t e0 = run0<HALVES>(l, turned), e1 = run1<HALVES>(p, l, turned);
  // blockIdx.y: the side (queries, then keys), and which of its runs of heads
  const bool keys = blockIdx.y >= (unsigned)p.runs_q;
  const QkSide d = keys ? p.k : p.q;
  const int run = keys ? (int)blockIdx.y - p.runs_q : (int)blockIdx.y, runs = keys ? (int)gridDim.y - p.runs_q : p.runs_q;
  v4f w[2];
  load_weights(p, d.w, own, e0, e1, w);

  for (int64_t t = (int64_t)blockIdx.x * kQkWaves + wave; t < p.tokens; t += (int64_t)gridDim.x * kQkWaves) {
    v4f c = {1.0f, 1.0f, 1.0f, 1.0f}, s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (turned) load_turn(p, p.positions ? p.positions[t] : t, l, c, s);
    // Input and output are buffer resources over the token's heads: the addresses of a set
    // are one scalar offset, loads of heads past the last give zeros and their stores are
    // dropped.
    const uint32_t hs_in = (uint32_t)d.hs_x * IB, hs_out = (uint32_t)d.hs_o * OB;
    const __amdgpu_buffer_rsrc_t in = make_rsrc(static_cast<const char*>(d.x) + t * d.ld_x * IB,
                                                (uint32_t)(d.heads - 1) * hs_in + p.head_dim * IB);
    const __amdgpu_buffer_rsrc_t out = make_rsrc(static_cast<const char*>(d.out) + t * d.ld_o * OB,
                                                 (uint32_t)(d.heads - 1) * hs_out + p.head_dim * OB);
    const uint32_t i0 = own ? sub * hs_in + e0 * IB : kOutsideHead, i1 = own ? sub * hs_in + e1 * IB : kOutsideHead;
    const uint32_t o0 = own ? sub * hs_out + e0 * OB : kOutsideHead, o1 = own ? sub * hs_out + e1 * OB : kOutsideHead;
    for (int h0 = run * (HPS * U); h0 < d.heads; h0 += runs * (HPS * U)) {
      v4f x[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) load8<F32, HALVES>(in, i0, i1, (uint32_t)(h0 + u * HPS) * hs_in, x[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // added to the lane offsets: a 16-byte store with a scalar offset may be followed at
        // once by a write to its data registers (the compiler keeps them apart only in the
        // other form), and was seen to store the new values
        const uint32_t base = (uint32_t)(h0 + u * HPS) * hs_out;
        float y[2][4];
        norm_and_turn<G, HALVES>(p, x[u], w, c, s, turned, y);
        if constexpr (QUANT) {
          const Int8Scale sc = head_scale<G>(y);
          const int h = h0 + u * HPS + sub;
          if (l == 0 && h < d.heads) d.scales[t * d.ld_s + h] = sc.s;
          const unsigned lo = int8_pack4(y[0][0], y[0][1], y[0][2], y[0][3], sc.inv) & sc.keep;
          const unsigned hi = int8_pack4(y[1][0], y[1][1], y[1][2], y[1][3], sc.inv) & sc.keep;
          if constexpr (HALVES) {
            __builtin_amdgcn_raw_buffer_store_b32(lo, out, o0 + base, 0, kNt);
            __builtin_amdgcn_raw_buffer_store_b32(hi, out, o1 + base, 0, kNt);
          } else {
            __builtin_amdgcn_raw_buffer_store_b64(v2u{lo, hi}, out, o0 + base, 0, kNt);
          }
        } else if constexpr (F32) {
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(v4u, v4f{y[0][0], y[0][1], y[0][2], y[0][3]}), out, o0 + base, 0, kNt);
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(v4u, v4f{y[1][0], y[1][1], y[1][2], y[1][3]}), out, o1 + base, 0, kNt);
        } else {
          const v2u lo = pack4(y[0]), hi = pack4(y[1]);
          if constexpr (HALVES) {
            __builtin_amdgcn_raw_buffer_store_b64(lo, out, o0 + base, 0, kNt);
            __builtin_amdgcn_raw_buffer_store_b64(hi, out, o1 + base, 0, kNt);
          } else {
            __builtin_amdgcn_raw_buffer_store_b128(v4u{lo[0], lo[1], hi[0], hi[1]}, out, o0 + base, 0, kNt);
          }
        }
      }
    }
  }
}

// Few heads for each token: a wave takes 64 / G * U consecutive (token, head) pairs of a side, whichever
// tokens they belong to, with addresses of its own in every lane.
template <int G, bool F32, bool QUANT, bool HALVES, int U>
__global__ __launch_bounds__(64 * kQkWaves) void qk_norm_rope_pairs_kernel(QkNormParams p) {
  constexpr int HPS = 64 / G;
  constexpr uint32_t IB = F32 ? 4 : 2, OB = QUANT ? 1 : IB;
  const int lane = threadIdx.x & 63, l = lane % G, sub = lane / G, wave = threadIdx.x >> 6;
  const bool own = 8 * l < p.head_dim, turned = 8 * l < p.rot_dim;
  const uint32_t e0 = run0<HALVES>(l, turned), e1 = run1<HALVES>(p, l, turned);
  const bool keys = blockIdx.x >= (unsigned)p.runs_q;
  const QkSide d = keys ? p.k : p.q;
  const uint32_t pairs = (uint32_t)p.tokens * (uint32_t)d.heads;
  const uint32_t first = ((keys ? blockIdx.x - p.runs_q : blockIdx.x) * kQkWaves + wave) * (HPS * U) + sub;
  uint32_t t[U], h[U];
  int64_t pos[U];
  bool in[U];
  v4f x[U][2], c[U], s[U], w[2];
  load_weights(p, d.w, own, e0, e1, w);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + u * HPS;
    in[u] = i < pairs;
    t[u] = in[u] ? i / (uint32_t)d.heads : 0u;
    h[u] = in[u] ? i - t[u] * (uint32_t)d.heads : 0u;
    pos[u] = turned && p.positions ? p.positions[t[u]] : t[u];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const char* src = static_cast<const char*>(d.x) + (t[u] * d.ld_x + h[u] * d.hs_x) * IB;
    x[u][0] = x[u][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (own) {
      if constexpr (F32) {
        x[u][0] = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(src + e0 * IB));
        x[u][1] = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(src + e1 * IB));
      } else if constexpr (HALVES) {
        x[u][0] = widen4(__builtin_nontemporal_load(reinterpret_cast<const v2u*>(src + e0 * IB)));
        x[u][1] = widen4(__builtin_nontemporal_load(reinterpret_cast<const v2u*>(src + e1 * IB)));
      } else {
        const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(src + e0 * IB));
        x[u][0] = widen4(v2u{v[0], v[1]});
        x[u][1] = widen4(v2u{v[2], v[3]});
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    c[u] = v4f{1.0f, 1.0f, 1.0f, 1.0f};
    s[u] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (turned) load_turn(p, pos[u], l, c[u], s[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float y[2][4];
    norm_and_turn<G, HALVES>(p, x[u], w, c[u], s[u], turned, y);
    char* dst = static_cast<char*>(d.out) + (t[u] * d.ld_o + h[u] * d.hs_o) * OB;
    if constexpr (QUANT) {
      const Int8Scale sc = head_scale<G>(y);
      if (l == 0 && in[u]) d.scales[t[u] * d.ld_s + h[u]] = sc.s;
      const unsigned lo = int8_pack4(y[0][0], y[0][1], y[0][2], y[0][3], sc.inv) & sc.keep;
      const unsigned hi = int8_pack4(y[1][0], y[1][1], y[1][2], y[1][3], sc.inv) & sc.keep;
      if (own && in[u]) {
        if constexpr (HALVES) {
          *reinterpret_cast<unsigned*>(dst + e0) = lo;
          *reinterpret_cast<unsigned*>(dst + e1) = hi;
        } else {
          *reinterpret_cast<v2u*>(dst + e0) = v2u{lo, hi};
        }
      }
    } else if (own && in[u]) {
      if constexpr (F32) {
        *reinterpret_cast<v4f*>(dst + e0 * OB) = v4f{y[0][0], y[0][1], y[0][2], y[0][3]};
        *reinterpret_cast<v4f*>(dst + e1 * OB) = v4f{y[1][0], y[1][1], y[1][2], y[1][3]};
      } else {
        const v2u lo = pack4(y[0]), hi = pack4(y[1]);
        if constexpr (HALVES) {
          *reinterpret_cast<v2u*>(dst + e0 * OB) = lo;
          *reinterpret_cast<v2u*>(dst + e1 * OB) = hi;
        } else {
          *reinterpret_cast<v4u*>(dst + e0 * OB) = v4u{lo[0], lo[1], hi[0], hi[1]};
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormParams& args, bool f32, bool quant, bool halves, hipStream_t stream) {
  if (args.tokens == 0 || args.q.heads + args.k.heads == 0) return hipSuccess;
  auto go = [&](auto g_tag, auto f_tag, auto q_tag, auto h_tag, auto u_tag) {
    constexpr int G = decltype(g_tag)::value, U = decltype(u_tag)::value, SET = 64 / G * U;
    QkNormParams p = args;
    const int64_t waves = (p.tokens + kQkWaves - 1) / kQkWaves, cap = (int64_t)1 << 20;
    // U == 1, a few tokens: every set of heads is a wave's; else a wave runs over all sets
    auto runs = [&](int heads) {
      const int sets = (heads + SET - 1) / SET;
      return heads == 0 ? 0 : U > 1 ? 1 : sets < 32767 ? sets : 32767;
    };
    p.runs_q = runs(p.q.heads);
    const dim3 grid((unsigned)(waves < cap ? waves : cap), (unsigned)(p.runs_q + runs(p.k.heads)));
    hipLaunchKernelGGL((qk_norm_rope_kernel<G, decltype(f_tag)::value, decltype(q_tag)::value, decltype(h_tag)::value, U>),
                       grid, dim3(64 * kQkWaves), 0, stream, p);
  };
  auto go_pairs = [&](auto g_tag, auto f_tag, auto q_tag, auto h_tag) {
    constexpr int G = decltype(g_tag)::value, U = 4, PER = 64 / G * U * kQkWaves;
    QkNormParams p = args;
    auto blocks = [&](int heads) { return (unsigned)((p.tokens * heads + PER - 1) / PER); };
    p.runs_q = (int)blocks(p.q.heads);
    hipLaunchKernelGGL((qk_norm_rope_pairs_kernel<G, decltype(f_tag)::value, decltype(q_tag)::value, decltype(h_tag)::value, U>),
                       dim3(p.runs_q + blocks(p.k.heads)), dim3(64 * kQkWaves), 0, stream, p);
  };
  using T = std::true_type;
  using F = std::false_type;
  // Below 512 tokens the sets are spread over the GPU (4 + 4 heads of 128, 600 tokens: the
  // same time either way); above, two sets in flight for each wave (one: 0.70 ms for
  // 75600 x (40 + 40) x 128; four: 0.55 ms too, but 0.20 for 0.185 ms where 24 heads leave
  // half of them idle at the end).  Where the queries and keys of a token are no more than two
  // sets, (token, head) pairs: 30000 tokens x (2 + 2) heads x 128 28 -> 16 us, (1 + 1) 23 -> 9,
  // (4 + 4) 32 -> 30, but (8 + 8) 41 and 56 (from the memory-side cache; not from it, 25000 x (1 + 1)
  // takes 9.3 us, 30000 x (2 + 2) 18, (4 + 4) 32, (8 + 8) 43).
  auto u = [&](auto g, auto f, auto q, auto h) {
    const int heads = args.q.heads + args.k.heads;
    if (args.tokens < 512)
      go(g, f, q, h, std::integral_constant<int, 1>{});
    else if (heads * decltype(g)::value <= 128 && args.tokens < ((int64_t)1 << 26))   // 2^31 threads, 2^30 pairs
      go_pairs(g, f, q, h);
    else
      go(g, f, q, h, std::integral_constant<int, 2>{});
  };
  auto h = [&](auto g, auto f, auto q) { halves ? u(g, f, q, T{}) : u(g, f, q, F{}); };
  auto q = [&](auto g, auto f) { quant ? h(g, f, T{}) : h(g, f, F{}); };
  auto f = [&](auto g) { f32 ? q(g, T{}) : q(g, F{}); };
  if (args.head_dim <= 64)
    f(std::integral_constant<int, 8>{});
  else if (args.head_dim <= 128)
    f(std::integral_constant<int, 16>{});
  else if (args.head_dim <= 256)
    f(std::integral_constant<int, 32>{});
  else
    f(std::integral_constant<int, 64>{});
  return hipGetLastError();
}

}  // namespace mxq
