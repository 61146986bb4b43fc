// Layer norm of rows, to the input's type or to 8-bit codes (mxq_int8.hpp), and its gradient.
//
// Forward, for a row x of C elements, in binary32:
//   mean = sum x / C;  rstd = 1 / sqrt( sum (x - mean)^2 / C + eps );  y = (x - mean) * rstd * w + b
// Every wave of a row takes the mean of its own elements and the squares of their deviations
// from it (DPP and lane swaps); the waves' means, counts and squares are then joined through LDS
// behind one barrier, sum_k m2_k + n_k (m_k - mean)^2, which is a sum of squares again: nothing cancels.
// What a mean loses in its rounding is taken from the deviations.  A row is read once and
// stays in registers as it was loaded.  Bound by HBM: 75600 x 5120 bf16 274 us (5.65 TB/s; a 1 GiB copy reaches 5.0),
// with the kept codes 348 (5.6), binary32 565 (5.5), 30000 x 13824 bf16 339 (4.9), binary32 592 (5.6).  To codes the
// vector units are never idle either, and time goes with the clock: 228 to 238 us (4.9 to 5.1 TB/s) at 2.4 GHz, 300 in the first
// passes after a pause, at 2.0.
//
// Backward, with xh = (x - mean) * rstd and g = dy * w:
//   dx = rstd * (g - sum g / C - xh * sum (g xh) / C),  dw = sum_rows dy xh,  db = sum_rows dy
// x is the kept input, or its 8-bit codes and row scales.  A thread owns 8 U columns for all
// the rows that its workgroup takes, so that dw and db stay in its registers; the workgroups'
// sums are joined by a second kernel in a fixed order.  Bound by HBM: 75600 x 5120 bf16 401 us (5.8 TB/s), from codes
// 327 (5.9), binary32 880 (5.3), 30000 x 13824 bf16 437 (5.7); rows of a thousand elements wait for their sums (60000 x 1040 84 us, 4.5 TB/s).
#include <type_traits>

#include "mxq_internal.hpp"
#include "mxq_rows.hpp"

namespace mxq {
namespace {

// 8 weights or biases from column 8 i, or `none`.
__device__ __forceinline__ void load_vector8(const void* w, int f32, uint32_t i, float none, float (&o)[8]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = none;
  } else if (f32) {
    widen_unit<true>(load_unit<true, false>(w, (int64_t)i * 8), o);
  } else {
    widen_unit<false>(load_unit<false, false>(w, (int64_t)i * 8), o);
  }
}

// Whether a row has 8-bit codes: not where its squares overflow or, without eps, vanish, nor where it has a NaN.
__device__ __forceinline__ bool finite_stats(float var, float rstd) {
  return var < __builtin_inff() && rstd < __builtin_inff();
}

// The sums of a wave over its elements of a row, as they are joined: with m the rounded mean of its elements and
// d = x - m, e = sum d / n takes back what m lost in its rounding, and m2 = sum (d - e)^2.
struct WaveSums {
  float m, e, m2;
};

// The sums of a row whose squares came out past binary32, once more over G lanes, `in(c)` telling which units are there.  Of large equal
// values the sum overflows, or their rounded mean is off by a last digit whose square does: here the sum is taken of
// values times 2^-11 (G lanes have up to 2^11 of them), the mean kept finite, and the squares taken of what is left once e is off too:
// 0 for equal values.  Deviations that do have such squares, an infinity or a NaN come out as they did.
template <bool F32, int C, int G, class In>
__device__ __forceinline__ WaveSums large_sums(Unit<F32> (&u)[C], float n, float inv_n, In in) {
  static_assert(C * G <= 256, "2^11 values");
  auto sum = [&](auto value) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      forget_unit<F32>(u[c]);
      if (in(c)) {
        float v[8];
        widen_unit<F32>(u[c], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += value(v[k]);
      }
    }
    return group_sum<G>(s);
  };
  constexpr float kTop = 0x1.fffffep127f;
  const float m = __builtin_amdgcn_fmed3f(sum([](float x) { return x * 0x1p-11f; }) * inv_n * 0x1p11f, -kTop, kTop);
  const float e = quotient(sum([&](float x) { return x - m; }), n, inv_n);
  return WaveSums{m, e, sum([&](float x) { const float d = (x - m) - e; return d * d; })};
}

// A row over the whole workgroup of 4 or 8 waves (a multiple of the 4 SIMDs), or (ONE) over a wave, four rows in a workgroup and nothing
// synchronized; C units of 8 elements in each thread.  A workgroup takes many rows: it keeps its columns'
// weights, and loads its next row while it works on one.
template <bool F32, bool QUANT, int C, bool ONE, int MOST = 256>
__global__ __launch_bounds__(MOST) void layer_norm_kernel(NormParams p) {
  // two slots in turn: a wave may reach the next row's store while another still reads
  __shared__ WaveSums sums[2][16];
  __shared__ unsigned tops[2][2][16];
  const uint32_t lane = threadIdx.x & 63;
  // scalar, so that a row's address is too
  const uint32_t wave_id = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t tid = ONE ? lane : threadIdx.x, T = ONE ? 64u : blockDim.x, wave = ONE ? 0u : wave_id;
  const uint32_t rows_here = ONE ? 4 : 1;
  if constexpr (!ONE) {   // slots of waves that are not there
    if (threadIdx.x < 32) {
      sums[threadIdx.x >> 4][threadIdx.x & 15] = WaveSums{0.0f, 0.0f, 0.0f};
      tops[threadIdx.x >> 4][0][threadIdx.x & 15] = tops[threadIdx.x >> 4][1][threadIdx.x & 15] = 0u;
    }
    __syncthreads();
  }
  // elements of wave k
  auto count = [&](uint32_t k) {
    uint32_t n = 0;
#pragma unroll
    for (uint32_t c = 0; c < C; ++c) {
      const uint32_t first = c * T + 64 * k;
      n += k < T / 64 && first < p.units ? min(p.units - first, 64u) : 0u;
    }
    return (float)(8 * n);
  };
  const float n = count(wave), n_of = count(lane & 15);   // of this wave, and of wave lane & 15
  const float inv_n = n > 0.0f ? 1.0f / n : 0.0f;
  auto load_row = [&](int64_t row, Unit<F32>(&u)[C]) {
    const char* x = static_cast<const char*>(p.x) + row * p.ld_x * (F32 ? 4 : 2);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      if (i < p.units) u[c] = p.past ? load_unit<F32, true>(x, i * 8) : load_unit<F32, false>(x, i * 8);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * rows_here;
  int64_t row = (int64_t)blockIdx.x * rows_here + (ONE ? wave_id : 0u);
  Unit<F32> u[C], next[C];
#pragma unroll
  for (int c = 0; c < C; ++c) u[c] = next[c] = zero_unit<F32>();   // threads past the row
  if (row < p.rows) load_row(row, u);
  // With 4 units the registers are short.  In bf16 the weights are read for each row, from the caches (30000 x 13824 to
  // codes 297 us, held 328); in binary32 they are held, and codes are formed from results computed again (378 us, read 457).
  constexpr bool HELD = C < 4 || F32, HOLD = C < 4 || !F32;
  float w[HELD ? C : 1][8], b[HELD ? C : 1][8];
  auto load_weights = [&](int c) {
    const uint32_t i = c * T + tid;
    load_vector8(i < p.units ? p.w : nullptr, p.w_f32, i, 1.0f, w[HELD ? c : 0]);
    load_vector8(i < p.units ? p.b : nullptr, p.w_f32, i, 0.0f, b[HELD ? c : 0]);
  };
  bool odd = false;   // an infinity or a NaN among them
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!HELD && !QUANT) break;
    load_weights(c);
    odd |= max(max_abs8(w[HELD ? c : 0]), max_abs8(b[HELD ? c : 0])) >= 0x7F800000u;
  }
  for (int par = 0; row < p.rows; row += stride, par ^= 1) {
    if (row + stride < p.rows) load_row(row + stride, next);
    // the row stays as it was loaded, and is widened again in each pass
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) s = sum_unit<F32>(u[c], s);
    float m = rounded_product(wave_sum(s), inv_n);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c * T + tid < p.units) {
        float v[8];
        widen_unit<F32>(u[c], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = v[e] - m;
          s1 += d;
          s2 = __builtin_fmaf(d, d, s2);
        }
      }
    }
    const float pair = wave_sum2(s1, s2);
    s1 = of_lane(pair, 0);
    s2 = of_lane(pair, 32);
    // quotients, not products with a rounded 1 / n: a row of equal values then has deviations of exactly 0
    float e = quotient(s1, n, inv_n), q = __builtin_fmaf(-s1, e, s2);
    if (!(q < __builtin_inff())) {   // the whole wave
      const WaveSums k = large_sums<F32, C, 64>(u, n, inv_n, [&](int c) { return c * T + tid < p.units; });
      m = k.m;
      e = k.e;
      q = k.m2;
    }
    unsigned top = 0;
    if (p.kept) {
#pragma unroll
      for (int c = 0; c < C; ++c) top = max(top, unit_max<F32>(u[c]));
      top = group_max<64>(top);
    }
    // m2: the row's sum of squared deviations; the mean in two parts, rounded and what that lost
    float m2 = q, mean = m + e, rest = (m - mean) + e;
    if constexpr (!ONE) {
      if (lane == 0) {
        sums[par][wave] = WaveSums{m, e, q};
        tops[par][0][wave] = top;
      }
      __syncthreads();
      // lane k of each 16 has wave k's, relative to the first wave's mean, so that a mean far from zero costs nothing
      const WaveSums k = sums[par][lane & 15];
      const float r0 = sums[par][0].m, delta = (k.m - r0) + k.e;
      const float a = quotient(group_sum<16>(n_of * delta), p.cols, p.inv_cols), t = delta - a;
      m2 = group_sum<16>(__builtin_fmaf(n_of * t, t, k.m2));
      if (p.kept) top = row16_max_u32(tops[par][0][lane & 15]);
      mean = r0 + a;
      rest = (r0 - mean) + a;
    }
    if (p.kept) {
      const Int8Scale sc = int8_scale(top);
      int8_t* kept = p.kept + row * p.ld_kept;
      if (tid == 0) p.kept_scales[row] = sc.s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        if (i < p.units) __builtin_nontemporal_store(unit_codes<F32>(u[c], sc), reinterpret_cast<v2u*>(kept + i * 8));
      }
    }
    // not a fmaxf alone, which would turn a NaN into 0
    const float var = m2 == m2 ? fmaxf(m2, 0.0f) * p.inv_cols : m2, rstd = rsqrtf(var + p.eps);
    if (tid == 0 && p.mean) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    // (x - mean - rest) * rstd * w + b
    const float shift = -rest * rstd;
    auto result = [&](int c, float(&o)[8]) {
      forget_unit<F32>(u[c]);
      widen_unit<F32>(u[c], o);
      if constexpr (!HELD) load_weights(c);
      const float(&wc)[8] = w[HELD ? c : 0], (&bc)[8] = b[HELD ? c : 0];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = __builtin_fmaf(__builtin_fmaf(o[k] - mean, rstd, shift), wc[k], bc[k]);
    };
    char* y = static_cast<char*>(p.y) + row * p.ld_y * (QUANT ? 1 : F32 ? 4 : 2);
    if constexpr (!QUANT) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        if (i < p.units) {
          float o[8];
          result(c, o);
          if (p.past)
            store_out<F32, true>(y, i * 8, o, (i | 3) < p.units);
          else
            store_unit<F32, false>(y, i * 8, o);
        }
      }
    } else {
      // the largest magnitude by a floating maximum, which passes over a NaN: there is one only where a weight or
      // bias is not finite, or the statistics are not
      float o[HOLD ? C : 1][8], most = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float(&v)[8] = o[HOLD ? c : 0];
        result(c, v);
        if (c * T + tid < p.units)
#pragma unroll
          for (int k = 0; k < 8; k += 2) most = fmaxf(fmaxf(most, fabsf(v[k])), fabsf(v[k + 1]));
      }
      unsigned top_y = group_max<64>(odd || !finite_stats(var, rstd) ? 0x7FC00000u : __float_as_uint(most));
      if constexpr (!ONE) {
        if (lane == 0) tops[par][1][wave] = top_y;
        __syncthreads();
        top_y = row16_max_u32(tops[par][1][lane & 15]);
      }
      const Int8Scale sc = int8_scale(top_y);
      if (tid == 0) p.scales[row] = sc.s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        if constexpr (!HOLD) result(c, o[0]);
        if (i < p.units) __builtin_nontemporal_store(pack_codes(o[HOLD ? c : 0], sc), reinterpret_cast<v2u*>(y + i * 8));
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) u[c] = next[c];
  }
}

// Rows of up to G units, 64 / G of them in a wave: lane l of a group has unit l, R rows of each
// group in flight, the weights in registers.  Registers for 4 waves on a SIMD: the compiler then spreads the rows in flight over them
// (300000 x 128 fp32 with kept codes 65 us, for 5 waves 69; bf16 33 either way).
template <bool F32, bool QUANT, int G>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 4))) void layer_norm_short_kernel(NormParams p) {
  constexpr int PER = 256 / G, R = 4;   // rows of the workgroup at once, passes in flight
  const uint32_t l = threadIdx.x % G;
  const bool own = l < p.units;
  float w[8], b[8];
  load_vector8(own ? p.w : nullptr, p.w_f32, l, 1.0f, w);
  load_vector8(own ? p.b : nullptr, p.w_f32, l, 0.0f, b);
  for (int64_t r0 = (int64_t)blockIdx.x * (PER * R) + threadIdx.x / G; r0 < p.rows; r0 += (int64_t)gridDim.x * (PER * R)) {
    Unit<F32> u[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t row = r0 + k * PER;
      u[k] = own && row < p.rows ? (p.past ? load_unit<F32, true>(p.x, row * p.ld_x + (int64_t)l * 8) : load_unit<F32, false>(p.x, row * p.ld_x + (int64_t)l * 8)) : zero_unit<F32>();
    }
    auto put = [&](int k, float mean, float rest, float m2) {
      const int64_t row = r0 + k * PER;
      const bool there = row < p.rows;
      float v[8];
      widen_unit<F32>(u[k], v);
      const float var = m2 == m2 ? fmaxf(m2, 0.0f) * p.inv_cols : m2, rstd = rsqrtf(var + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(__builtin_fmaf(v[e] - mean, rstd, -rest * rstd), w[e], b[e]);
      if (l == 0 && there && p.mean) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
      if (p.kept) {
        const Int8Scale sc = int8_scale(group_max<G>(unit_max<F32>(u[k])));
        if (l == 0 && there) p.kept_scales[row] = sc.s;
        if (own && there)
          __builtin_nontemporal_store(unit_codes<F32>(u[k], sc), reinterpret_cast<v2u*>(p.kept + row * p.ld_kept + (int64_t)l * 8));
      }
      if constexpr (QUANT) {
        const Int8Scale sc = int8_scale(group_max<G>(!finite_stats(var, rstd) ? 0x7FC00000u : own ? max_abs8(v) : 0u));
        if (l == 0 && there) p.scales[row] = sc.s;
        if (own && there)
          __builtin_nontemporal_store(pack_codes(v, sc), reinterpret_cast<v2u*>(static_cast<int8_t*>(p.y) + row * p.ld_y + (int64_t)l * 8));
      } else if (own && there) {
        if (p.past)
          store_out<F32, true>(p.y, row * p.ld_y + (int64_t)l * 8, v, (l | 3) < p.units);
        else
          store_unit<F32, false>(p.y, row * p.ld_y + (int64_t)l * 8, v);
      }
    };
    // rows for large_sums, of any group: they are written again, so that the others wait for no branch of theirs
    unsigned large = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float v[8];
      widen_unit<F32>(u[k], v);
      const float m = rounded_product(group_sum<G>(sum_unit<F32>(u[k], 0.0f)), p.inv_cols);
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = own ? v[e] - m : 0.0f;
        s1 += d;
        s2 = __builtin_fmaf(d, d, s2);
      }
      s1 = group_sum<G>(s1);
      s2 = group_sum<G>(s2);
      const float e0 = quotient(s1, p.cols, p.inv_cols), m2 = __builtin_fmaf(-s1, e0, s2);
      const float mean = m + e0;
      put(k, mean, (m - mean) + e0, m2);
      large |= m2 < __builtin_inff() ? 0u : 1u << k;
    }
    if (large) {
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (large >> k & 1) {
          Unit<F32> one[1] = {u[k]};
          const WaveSums t = large_sums<F32, 1, G>(one, p.cols, p.inv_cols, [&](int) { return own; });
          const float mean = t.m + t.e;
          put(k, mean, (t.m - mean) + t.e, t.m2);
        }
    }
  }
}

// One row (of dy's type, or codes) as loaded.
template <bool F32, bool CODES> struct Kept { Unit<F32> u; };
template <bool F32> struct Kept<F32, true> { v2u u; };

// Threads of a workgroup: one for each unit of a row up to kNormThreads, U units for each beyond;
// R rows at once.  AFFINE: with weights or their sums.
template <bool F32, bool CODES, bool AFFINE, int U, int R>
__global__ __launch_bounds__(kNormThreads) void layer_norm_backward_kernel(NormGradParams p) {
  static_assert(R == 1 || R == 2, "the four rows of a wave's lanes hold the sums");
  // two slots in turn: a wave may reach the next rows' store while another still reads
  __shared__ float red[2][4][16];
  const uint32_t tid = threadIdx.x, T = blockDim.x, lane = tid & 63;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
  // slots of waves that are not there stay zero
  for (uint32_t i = tid; i < 2 * 4 * 16; i += T) (&red[0][0][0])[i] = 0.0f;
  float w[U][8], dw[U][8], db[U][8];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const uint32_t i = c * T + tid;
    load_vector8(AFFINE && i < p.units ? p.w : nullptr, p.w_f32, i, 1.0f, w[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = db[c][e] = 0.0f;
  }
  __syncthreads();
  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < p.rows; r0 += (int64_t)gridDim.x * R, par ^= 1) {
    Unit<F32> dy[R][U];
    Kept<F32, CODES> x[R][U];
    float mean[R], rstd[R], scale[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = min(r0 + r, p.rows - 1);
      const char* dy_row = static_cast<const char*>(p.dy) + row * p.ld_dy * (F32 ? 4 : 2);
      const char* x_row = static_cast<const char*>(p.x) + row * p.ld_x * (CODES ? 1 : F32 ? 4 : 2);
#pragma unroll
      for (int c = 0; c < U; ++c) {
        const uint32_t i = min(c * T + tid, p.units - 1);   // threads past the row: its last unit, not used
        dy[r][c] = load_unit<F32, true>(dy_row, i * 8);
        if constexpr (CODES)
          x[r][c].u = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(x_row + i * 8));
        else
          x[r][c].u = load_unit<F32, true>(x_row, i * 8);
      }
      mean[r] = p.mean[row];
      rstd[r] = p.rstd[row];
      scale[r] = CODES ? p.x_scales[row] : 1.0f;
    }
    float g[R][U][8], xh[R][U][8], s1[2] = {0.0f, 0.0f}, s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool there = r0 + r < p.rows;
#pragma unroll
      for (int c = 0; c < U; ++c) {
        float d[8];
        widen_unit<F32>(dy[r][c], d);
        if constexpr (CODES)
          widen_codes(x[r][c].u, scale[r], xh[r][c]);
        else
          widen_unit<F32>(x[r][c].u, xh[r][c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xh[r][c][e] = (xh[r][c][e] - mean[r]) * rstd[r];
          g[r][c][e] = AFFINE ? d[e] * w[c][e] : d[e];
        }
        if (there && c * T + tid < p.units) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s1[r] += g[r][c][e];
            s2[r] = __builtin_fmaf(g[r][c][e], xh[r][c][e], s2[r]);
            if constexpr (AFFINE) {
              dw[c][e] = __builtin_fmaf(d[e], xh[r][c][e], dw[c][e]);
              db[c][e] += d[e];
            }
          }
        }
      }
    }
    // row 0 of the wave's lanes: g's sum of the first matrix row, 1: of the second, 2 and 3: those of g xh
    const float sums = R == 2 ? wave_sum4(s1[0], s2[0], s1[1], s2[1]) : wave_sum2(s1[0], s2[0]);
    if ((lane & 15) == 0) red[par][lane >> 4][wave] = sums;
    __syncthreads();
    const float total = row16_sum(red[par][lane >> 4][lane & 15]) * p.inv_cols;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float c1 = of_lane(total, 16 * r), c2 = of_lane(total, 32 + 16 * r);
      if (r0 + r >= p.rows) break;
      char* dx_row = static_cast<char*>(p.dx) + (r0 + r) * p.ld_dx * (F32 ? 4 : 2);
#pragma unroll
      for (int c = 0; c < U; ++c) {
        const uint32_t i = c * T + tid;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd[r] * (g[r][c][e] - __builtin_fmaf(xh[r][c][e], c2, c1));
        if (i < p.units) store_out<F32, true>(dx_row, i * 8, o, (i | 3) < p.units);
      }
    }
  }
  if (AFFINE && p.dw) {
    float* part = p.part + (int64_t)blockIdx.x * 2 * p.units * 8;
#pragma unroll
    for (int c = 0; c < U; ++c) {
      const uint32_t i = c * T + tid;
      if (i < p.units) {
        store_unit<true, false>(gridDim.x > 1 ? part : p.dw, (int64_t)i * 8, dw[c]);
        store_unit<true, false>(gridDim.x > 1 ? part + (int64_t)p.units * 8 : p.db, (int64_t)i * 8, db[c]);
      }
    }
  }
}

// Rows of up to G units, 64 / G of them in a wave, R rows of each group in flight: lane l of a group has unit l
// of all rows that its workgroup takes.
template <bool F32, bool CODES, bool AFFINE, int G>
__global__ __launch_bounds__(256) void layer_norm_backward_short_kernel(NormGradParams p) {
  constexpr int PER = 256 / G, R = 2;   // rows of the workgroup at once, passes in flight
  __shared__ float red[4][2][G * 8];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = threadIdx.x % G;
  const bool own = l < p.units;
  float w[8], dw[8], db[8];
  load_vector8(AFFINE && own ? p.w : nullptr, p.w_f32, l, 1.0f, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
  for (int64_t r0 = (int64_t)blockIdx.x * (PER * R) + threadIdx.x / G; r0 < p.rows; r0 += (int64_t)gridDim.x * (PER * R)) {
    Unit<F32> dy[R];
    Kept<F32, CODES> x[R];
    float mean[R], rstd[R], scale[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = min(r0 + r * PER, p.rows - 1), col = (int64_t)min(l, p.units - 1) * 8;
      dy[r] = load_unit<F32, true>(p.dy, row * p.ld_dy + col);
      if constexpr (CODES)
        x[r].u = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(static_cast<const int8_t*>(p.x) + row * p.ld_x + col));
      else
        x[r].u = load_unit<F32, true>(p.x, row * p.ld_x + col);
      mean[r] = p.mean[row];
      rstd[r] = p.rstd[row];
      scale[r] = CODES ? p.x_scales[row] : 1.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r * PER;
      const bool in = own && row < p.rows;
      float d[8], xh[8], s1 = 0.0f, s2 = 0.0f;
      widen_unit<F32>(dy[r], d);
      if constexpr (CODES)
        widen_codes(x[r].u, scale[r], xh);
      else
        widen_unit<F32>(x[r].u, xh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = in ? d[e] : 0.0f;
        xh[e] = in ? (xh[e] - mean[r]) * rstd[r] : 0.0f;
        if constexpr (AFFINE) {
          dw[e] = __builtin_fmaf(d[e], xh[e], dw[e]);
          db[e] += d[e];
          d[e] *= w[e];
        }
        s1 += d[e];
        s2 = __builtin_fmaf(d[e], xh[e], s2);
      }
      const float c1 = group_sum<G>(s1) * p.inv_cols, c2 = group_sum<G>(s2) * p.inv_cols;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = rstd[r] * (d[e] - __builtin_fmaf(xh[e], c2, c1));
      if (in) store_out<F32, true>(p.dx, row * p.ld_dx + (int64_t)l * 8, d, (l | 3) < p.units);
    }
  }
  if (AFFINE && p.dw) {
    // lanes of one l in a wave, then the waves
    auto over_groups = [](float v) {
      if constexpr (G == 8) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, true));   // row_ror by 8
      if constexpr (G <= 16) v = fold16(v, v);
      if constexpr (G <= 32) v = fold32(v, v);
      return v;
    };
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float sw = over_groups(dw[e]), sb = over_groups(db[e]);
      if (lane < G) {
        red[wave][0][l * 8 + e] = sw;
        red[wave][1][l * 8 + e] = sb;
      }
    }
    __syncthreads();
    const uint32_t n = p.units * 8;
    float* part = p.part + (int64_t)blockIdx.x * 2 * n;
    for (uint32_t i = threadIdx.x; i < 2 * n; i += 256) {
      const uint32_t k = i >= n, c = i - k * n;
      const float v = (red[0][k][c] + red[1][k][c]) + (red[2][k][c] + red[3][k][c]);
      if (gridDim.x > 1)
        part[i] = v;
      else
        (k ? p.db : p.dw)[c] = v;
    }
  }
}

// Sums of `parts` rows of 2 n floats, the first n to dw and the rest to db: 64 columns for each workgroup,
// 16 runs of rows joined in LDS.  The order is fixed.
__global__ __launch_bounds__(1024) void layer_norm_sums_kernel(const float* part, int parts, uint32_t n, float* dw, float* db) {
  __shared__ float red[16][64];
  const uint32_t lane = threadIdx.x & 63, run = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  // 8 rows in flight for each thread: with few columns there are few workgroups, and only latency counts (1536 x 2080:
  // 4 in flight 9.8 us)
  float s[8] = {};
  if (col < 2 * n) {
    int r = run;
    for (; r + 16 * 7 < parts; r += 16 * 8)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += part[(int64_t)(r + 16 * k) * 2 * n + col];
    for (; r < parts; r += 16) s[0] += part[(int64_t)r * 2 * n + col];
  }
  red[run][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  if (run == 0 && col < 2 * n) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += red[k][lane];
    if (col < n)
      dw[col] = t;
    else
      db[col - n] = t;
  }
}

// The gradient's launch.  Several rows share a wave up to 64 units (80000 x 512 bf16 49 us, a workgroup of one wave 65).
// Workgroups leave 2 C floats each, so that there are no more of them than the GPU runs at once,
// and each has 8 rows or more where there are enough rows (4099 x 2064 binary32: 512 workgroups 26 us, 1024 33, 256 30;
// 75600 x 5120 bf16 from codes: 512 328 us, 1024 392).
struct GradLaunch {
  int lanes;      // of a row in the short kernel, or 0
  int threads;
  int64_t groups;
};
GradLaunch grad_launch(int64_t rows, int64_t cols) {
  const int64_t units = cols / 8;
  GradLaunch g;
  g.lanes = units <= 8 ? 8 : units <= 16 ? 16 : units <= 32 ? 32 : units <= 64 ? 64 : 0;
  g.threads = g.lanes ? 256 : units > kNormThreads ? kNormThreads : (int)((units + 63) / 64 * 64);
  const int64_t each = g.lanes ? 256 / g.lanes * 2 : 1, sets = (rows + each - 1) / each;
  const int64_t full = 256 * (1280 / g.threads), some = rows / 8 > 64 ? rows / 8 : 64;
  g.groups = sets < full ? sets : full;
  if (g.groups > some) g.groups = some;
  return g;
}

// Whether a workgroup takes two rows at once, with one barrier for both: where a row has few waves (60000 x 1040 bf16 from
// codes: 75 us for 80), where the GPU holds but one workgroup on a CU (30000 x 8192: 226 us for 243), and for binary32
// (75600 x 5120: 877 us for 918).  Not for the rows between, of which more fit the registers one by one (75600 x
// 5120 bf16 from codes: 371 us for 328).
bool two_rows(int64_t rows, int threads, bool f32) {
  return rows >= 1024 && (f32 || threads <= 256 || threads > 768);
}

}  // namespace

hipError_t launch_layer_norm(const NormParams& args, bool f32, bool quant, hipStream_t stream) {
  if (args.rows == 0) return hipSuccess;
  NormParams p = args;
  // see launch_quantize_int8
  p.past = p.rows * (int64_t)p.units * 8 * (f32 ? 4 : 2) > ((int64_t)256 << 20);
  // About 6 rows in turn for a workgroup where there are enough.  Their weights cost it a reading of the caches
  // once, but workgroups that stay for all rows are slower than ones that come and go: 75600 x 5120 bf16 with 1 row
  // each 354 us, 2 295, 5 276, 6 274, 9 284, 18 296, 74 295.
  auto go = [&](auto kernel, int threads, int rows_per_block, int64_t most) {
    const int64_t sets = (p.rows + rows_per_block - 1) / rows_per_block;
    const int64_t few = 256 * (2048 / threads), many = sets / 6;
    const int64_t blocks = sets < few ? sets : many < few ? few : many;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3((unsigned)threads), 0, stream, p);
  };
  auto pick = [&](auto f_tag, auto q_tag) {
    constexpr bool F = decltype(f_tag)::value, Q = decltype(q_tag)::value;
    const int64_t most = (int64_t)1 << 20;   // blocks * threads stays below 2^32
    // us, to bf16 and to codes.  Several rows in a wave up to 32 units (150000 x 256 26 and 28, a wave for each row 33 and
    // 45; 80000 x 272, one row in a wave, 21 and 28), one wave for a row up to 192 (40000 x 1536 38 and 31, a workgroup
    // 42 and 57), then a workgroup of 4 waves up to 768 units, of 8 beyond (20000 x 5120 78 and 60, of 8 waves 80 and
    // 78), so that a thread holds 4 units at most.
    if (p.units <= 8)
      go(layer_norm_short_kernel<F, Q, 8>, 256, 32 * 4, most);
    else if (p.units <= 16)
      go(layer_norm_short_kernel<F, Q, 16>, 256, 16 * 4, most);
    else if (p.units <= 32)
      go(layer_norm_short_kernel<F, Q, 32>, 256, 8 * 4, most);
    else if (p.units <= 64)
      go(layer_norm_kernel<F, Q, 1, true>, 256, 4, most);
    else if (p.units <= 64 * 2)
      go(layer_norm_kernel<F, Q, 2, true>, 256, 4, most);
    else if (p.units <= 64 * 3)
      go(layer_norm_kernel<F, Q, 3, true>, 256, 4, most);
    else if (p.units <= 256)
      go(layer_norm_kernel<F, Q, 1, false>, 256, 1, most);
    else if (p.units <= 256 * 2)
      go(layer_norm_kernel<F, Q, 2, false>, 256, 1, most);
    else if (p.units <= 256 * 3)
      go(layer_norm_kernel<F, Q, 3, false>, 256, 1, most);
    else if (p.units <= 512 * 2)
      go(layer_norm_kernel<F, Q, 2, false, 512>, 512, 1, most);
    else if (p.units <= 512 * 3)
      go(layer_norm_kernel<F, Q, 3, false, 512>, 512, 1, most);
    else
      go(layer_norm_kernel<F, Q, 4, false, 512>, 512, 1, most);
  };
  using T = std::true_type;
  using N = std::false_type;
  auto q = [&](auto f) { quant ? pick(f, T{}) : pick(f, N{}); };
  f32 ? q(T{}) : q(N{});
  return hipGetLastError();
}

size_t layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  const int64_t groups = grad_launch(rows, cols).groups;
  return groups > 1 ? (size_t)groups * 2 * (size_t)cols * sizeof(float) : 0;
}

hipError_t launch_layer_norm_backward(const NormGradParams& p, bool f32, bool codes, hipStream_t stream) {
  const int64_t cols = (int64_t)p.units * 8;
  const bool sums = p.dw != nullptr, affine = sums || p.w;
  if (p.rows == 0) {
    if (!sums) return hipSuccess;
    hipLaunchKernelGGL(layer_norm_sums_kernel, dim3((unsigned)((2 * cols + 63) / 64)), dim3(1024), 0, stream, p.part, 0, (uint32_t)cols, p.dw, p.db);
    return hipGetLastError();
  }
  const GradLaunch g = grad_launch(p.rows, cols);
  const unsigned groups = (unsigned)g.groups;
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(groups), dim3((unsigned)g.threads), 0, stream, p); };
  using T = std::true_type;
  using N = std::false_type;
  auto u = [&](auto f, auto c, auto a) {
    constexpr bool F = decltype(f)::value, K = decltype(c)::value, A = decltype(a)::value;
    if (g.lanes == 8)
      go(layer_norm_backward_short_kernel<F, K, A, 8>);
    else if (g.lanes == 16)
      go(layer_norm_backward_short_kernel<F, K, A, 16>);
    else if (g.lanes == 32)
      go(layer_norm_backward_short_kernel<F, K, A, 32>);
    else if (g.lanes == 64)
      go(layer_norm_backward_short_kernel<F, K, A, 64>);
    else if (p.units > kNormThreads)
      go(layer_norm_backward_kernel<F, K, A, 2, 1>);
    else if (two_rows(p.rows, g.threads, F))
      go(layer_norm_backward_kernel<F, K, A, 1, 2>);
    else
      go(layer_norm_backward_kernel<F, K, A, 1, 1>);
  };
  auto a = [&](auto f, auto c) { affine ? u(f, c, T{}) : u(f, c, N{}); };
  auto c = [&](auto f) { codes ? a(f, T{}) : a(f, N{}); };
  f32 ? c(T{}) : c(N{});
  if (sums && groups > 1)
    hipLaunchKernelGGL(layer_norm_sums_kernel, dim3((unsigned)((2 * cols + 63) / 64)), dim3(1024), 0, stream, p.part,
                       (int)groups, (uint32_t)cols, p.dw, p.db);
  return hipGetLastError();
}

}  // namespace mxq
