// Layer norm of rows, to the input's type or to 8-bit codes (mxq_int8.hpp), and its gradient.
//
// Forward, for a row x of C elements, in binary32:
//   m0 = sum x / C;  d = x - m0;  e = sum d / C;  mean = m0 + e
//   var = sum d^2 / C - e^2;  rstd = 1 / sqrt(var + eps);  y = (d - e) * rstd * w + b
// e takes back what m0 lost in its rounding (a row of equal values gives y = b), and since
// |e| is about 2^-24 |m0| the subtraction in var loses nothing.  A row is read once and stays in
// registers; the sums are joined by DPP and lane swaps inside a wave and through LDS across
// the W waves of a row.  Bound by HBM.
//
// Backward, with xh = (x - mean) * rstd and g = dy * w:
//   dx = rstd * (g - sum g / C - xh * sum (g xh) / C),  dw = sum_rows dy xh,  db = sum_rows dy
// x is the kept input, or its 8-bit codes and row scales.  A thread owns 8 U columns for all
// the rows that its workgroup takes, so that dw and db stay in its registers; the workgroups'
// sums are joined by a second kernel in a fixed order.
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

// W waves for a row, C units of 8 elements in each thread; W == 1: four rows in a workgroup, and
// nothing is synchronized.
template <bool F32, bool STREAM, bool QUANT, int W, int C>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void layer_norm_kernel(NormParams p) {
  constexpr int T = 64 * W, RPB = W < 4 ? 4 / W : 1;
  static_assert(W == 1 || W >= 4, "a workgroup holds whole rows");
  // written and read between different barriers of a row, so that one copy of each is enough
  __shared__ float sums[3][W];
  __shared__ unsigned tops[2][W];
  const uint32_t tid = threadIdx.x % T, sub = threadIdx.x / T, lane = threadIdx.x & 63, wave = tid >> 6;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < p.rows; row += (int64_t)gridDim.x * RPB) {
    float v[C][8];
    unsigned top = 0;
    float s = 0.0f;
    {
      Unit<F32> u[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        u[c] = i < p.units ? load_unit<F32, STREAM>(p.x, row * p.ld_x + (int64_t)i * 8) : zero_unit<F32>();
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        widen_unit<F32>(u[c], v[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[c][e];
      }
    }
    s = wave_sum(s);
    if (p.kept) {
#pragma unroll
      for (int c = 0; c < C; ++c) top = max(top, max_abs8(v[c]));
      top = wave_max_u32(top);
    }
    if constexpr (W > 1) {
      if (lane == 0) {
        sums[0][wave] = s;
        tops[0][wave] = top;
      }
      __syncthreads();
      s = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        s += sums[0][k];
        top = max(top, tops[0][k]);
      }
    }
    if (p.kept) {
      const Int8Scale sc = int8_scale(top);
      if (tid == 0) p.kept_scales[row] = sc.s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        if (i < p.units)
          __builtin_nontemporal_store(pack_codes(v[c], sc), reinterpret_cast<v2u*>(p.kept + row * p.ld_kept + (int64_t)i * 8));
      }
    }
    const float m0 = s * p.inv_cols;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if ((uint32_t)(c * T) + tid < p.units) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[c][e] -= m0;
          s1 += v[c][e];
          s2 = __builtin_fmaf(v[c][e], v[c][e], s2);
        }
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (W > 1) {
      if (lane == 0) {
        sums[1][wave] = s1;
        sums[2][wave] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        s1 += sums[1][k];
        s2 += sums[2][k];
      }
    }
    const float e0 = s1 * p.inv_cols, var = fmaxf(__builtin_fmaf(-e0, e0, s2 * p.inv_cols), 0.0f);
    // not a fmaxf that would turn a NaN into 0
    const float rstd = s2 == s2 ? rsqrtf(var + p.eps) : s2;
    if (tid == 0 && p.mean) {
      p.mean[row] = m0 + e0;
      p.rstd[row] = rstd;
    }
    top = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      if (i < p.units) {
        float w[8], b[8];
        load_vector8(p.w, p.w_f32, i, 1.0f, w);
        load_vector8(p.b, p.w_f32, i, 0.0f, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = __builtin_fmaf((v[c][e] - e0) * rstd, w[e], b[e]);
        if constexpr (QUANT)
          top = max(top, max_abs8(v[c]));
        else
          store_unit<F32, STREAM>(p.y, row * p.ld_y + (int64_t)i * 8, v[c]);
      }
    }
    if constexpr (QUANT) {
      top = wave_max_u32(top);
      if constexpr (W > 1) {
        if (lane == 0) tops[1][wave] = top;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < W; ++k) top = max(top, tops[1][k]);
      }
      const Int8Scale sc = int8_scale(top);
      if (tid == 0) p.scales[row] = sc.s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t i = c * T + tid;
        if (i < p.units)
          __builtin_nontemporal_store(pack_codes(v[c], sc),
                                      reinterpret_cast<v2u*>(static_cast<int8_t*>(p.y) + row * p.ld_y + (int64_t)i * 8));
      }
    }
  }
}

// One row (of dy's type, or codes) as loaded.
template <bool F32, bool CODES> struct Kept { Unit<F32> u; };
template <bool F32> struct Kept<F32, true> { v2u u; };

// Threads of a workgroup: one for each unit of a row up to kNormThreads, U units for each beyond;
// R rows at once.  AFFINE: with weights, and their sums.
template <bool F32, bool CODES, bool AFFINE, int U, int R>
__global__ __launch_bounds__(kNormThreads) void layer_norm_backward_kernel(NormGradParams p) {
  __shared__ float red[2][R][2][16];
  const uint32_t tid = threadIdx.x, T = blockDim.x, lane = tid & 63, wave = tid >> 6, waves = T >> 6;
  // slots of waves that are not there stay zero
  for (uint32_t i = tid; i < 2 * R * 2 * 16; i += T) (&red[0][0][0][0])[i] = 0.0f;
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
#pragma unroll
      for (int c = 0; c < U; ++c) {
        const uint32_t i = c * T + tid;
        const int64_t col = (int64_t)min(i, p.units - 1) * 8;   // threads past the row: its last unit, not used
        dy[r][c] = load_unit<F32, true>(p.dy, row * p.ld_dy + col);
        if constexpr (CODES)
          x[r][c].u = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(static_cast<const int8_t*>(p.x) + row * p.ld_x + col));
        else
          x[r][c].u = load_unit<F32, true>(p.x, row * p.ld_x + col);
      }
      mean[r] = p.mean[row];
      rstd[r] = p.rstd[row];
      scale[r] = CODES ? p.x_scales[row] : 1.0f;
    }
    float g[R][U][8], xh[R][U][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s1 = 0.0f, s2 = 0.0f;
      const bool there = r0 + r < p.rows;
#pragma unroll
      for (int c = 0; c < U; ++c) {
        float d[8];
        widen_unit<F32>(dy[r][c], d);
        if constexpr (CODES)
          widen_codes(x[r][c].u, scale[r], xh[r][c]);
        else
          widen_unit<F32>(x[r][c].u, xh[r][c]);
        const bool in = there && (uint32_t)(c * T) + tid < p.units;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xh[r][c][e] = (xh[r][c][e] - mean[r]) * rstd[r];
          g[r][c][e] = AFFINE ? d[e] * w[c][e] : d[e];
        }
        if (in) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s1 += g[r][c][e];
            s2 = __builtin_fmaf(g[r][c][e], xh[r][c][e], s2);
            if constexpr (AFFINE) {
              dw[c][e] = __builtin_fmaf(d[e], xh[r][c][e], dw[c][e]);
              db[c][e] += d[e];
            }
          }
        }
      }
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if (lane == 0) {
        red[par][r][0][wave] = s1;
        red[par][r][1][wave] = s2;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float c1 = row16_sum(red[par][r][0][lane & 15]) * p.inv_cols;
      const float c2 = row16_sum(red[par][r][1][lane & 15]) * p.inv_cols;
#pragma unroll
      for (int c = 0; c < U; ++c) {
        const uint32_t i = c * T + tid;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd[r] * (g[r][c][e] - __builtin_fmaf(xh[r][c][e], c2, c1));
        if (r0 + r < p.rows && i < p.units) store_unit<F32, true>(p.dx, (r0 + r) * p.ld_dx + (int64_t)i * 8, o);
      }
    }
  }
  if constexpr (AFFINE) {
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

// Sums of `parts` rows of 2 n floats, the first n to dw and the rest to db: 64 columns for each workgroup,
// 16 runs of rows joined in LDS.  The order is fixed.
__global__ __launch_bounds__(1024) void layer_norm_sums_kernel(const float* part, int parts, uint32_t n, float* dw, float* db) {
  __shared__ float red[16][64];
  const uint32_t lane = threadIdx.x & 63, run = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < 2 * n) {
    int r = run;
    for (; r + 48 < parts; r += 64)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += part[(int64_t)(r + 16 * k) * 2 * n + col];
    for (; r < parts; r += 16) s[0] += part[(int64_t)r * 2 * n + col];
  }
  red[run][lane] = (s[0] + s[1]) + (s[2] + s[3]);
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

// Rows at once in a workgroup of the gradient, and workgroups.
int grad_rows(int64_t rows) { return rows < 1024 ? 1 : 2; }
int64_t grad_threads(int64_t units) { return units > kNormThreads ? kNormThreads : (units + 63) / 64 * 64; }
int64_t grad_groups(int64_t rows, int64_t cols) {
  const int64_t per_cu = 1024 / grad_threads(cols / 8) + 1, cap = 256 * (per_cu < 8 ? per_cu : 8);
  const int64_t sets = (rows + grad_rows(rows) - 1) / grad_rows(rows);
  return sets < cap ? sets : cap;
}

}  // namespace

hipError_t launch_layer_norm(const NormParams& p, bool f32, bool quant, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  auto go = [&](auto kernel, int threads, int rows_per_block) {
    const int64_t blocks = (p.rows + rows_per_block - 1) / rows_per_block;
    const int64_t cap = (int64_t)1 << 20;   // blocks * threads stays below 2^32
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(threads), 0, stream, p);
  };
  auto pick = [&](auto f_tag, auto s_tag, auto q_tag) {
    constexpr bool F = decltype(f_tag)::value, S = decltype(s_tag)::value, Q = decltype(q_tag)::value;
    if (p.units <= 64)
      go(layer_norm_kernel<F, S, Q, 1, 1>, 256, 4);
    else if (p.units <= 128)
      go(layer_norm_kernel<F, S, Q, 1, 2>, 256, 4);
    else if (p.units <= 256)
      go(layer_norm_kernel<F, S, Q, 1, 4>, 256, 4);
    else if (p.units <= 256 * 2)
      go(layer_norm_kernel<F, S, Q, 4, 2>, 256, 1);
    else if (p.units <= 256 * 3)
      go(layer_norm_kernel<F, S, Q, 4, 3>, 256, 1);
    else if (p.units <= 512 * 2)
      go(layer_norm_kernel<F, S, Q, 8, 2>, 512, 1);
    else
      go(layer_norm_kernel<F, S, Q, 8, 4>, 512, 1);
  };
  // see launch_quantize_int8
  const bool stream_loads = p.rows * (int64_t)p.units * 8 * (f32 ? 4 : 2) > ((int64_t)256 << 20);
  using T = std::true_type;
  using N = std::false_type;
  auto q = [&](auto f, auto s) { quant ? pick(f, s, T{}) : pick(f, s, N{}); };
  auto s = [&](auto f) { stream_loads ? q(f, T{}) : q(f, N{}); };
  f32 ? s(T{}) : s(N{});
  return hipGetLastError();
}

size_t layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  const int64_t groups = grad_groups(rows, cols);
  return groups > 1 ? (size_t)groups * 2 * (size_t)cols * sizeof(float) : 0;
}

hipError_t launch_layer_norm_backward(const NormGradParams& p, bool f32, bool codes, hipStream_t stream) {
  const int64_t cols = (int64_t)p.units * 8;
  const bool affine = p.dw != nullptr;
  if (p.rows == 0) {
    if (!affine) return hipSuccess;
    hipLaunchKernelGGL(layer_norm_sums_kernel, dim3((unsigned)((2 * cols + 63) / 64)), dim3(1024), 0, stream, p.part, 0, (uint32_t)cols, p.dw, p.db);
    return hipGetLastError();
  }
  const unsigned groups = (unsigned)grad_groups(p.rows, cols), threads = (unsigned)grad_threads(p.units);
  auto go = [&](auto f, auto c, auto a, auto u) {
    constexpr bool F = decltype(f)::value, K = decltype(c)::value, A = decltype(a)::value;
    constexpr int U = decltype(u)::value;
    if constexpr (U == 1) {
      if (grad_rows(p.rows) == 2) {
        hipLaunchKernelGGL((layer_norm_backward_kernel<F, K, A, U, 2>), dim3(groups), dim3(threads), 0, stream, p);
        return;
      }
    }
    hipLaunchKernelGGL((layer_norm_backward_kernel<F, K, A, U, 1>), dim3(groups), dim3(threads), 0, stream, p);
  };
  using T = std::true_type;
  using N = std::false_type;
  auto u = [&](auto f, auto c, auto a) {
    if (p.units <= kNormThreads)
      go(f, c, a, std::integral_constant<int, 1>{});
    else
      go(f, c, a, std::integral_constant<int, 2>{});
  };
  auto a = [&](auto f, auto c) { affine ? u(f, c, T{}) : u(f, c, N{}); };
  auto c = [&](auto f) { codes ? a(f, T{}) : a(f, N{}); };
  f32 ? c(T{}) : c(N{});
  if (affine && groups > 1)
    hipLaunchKernelGGL(layer_norm_sums_kernel, dim3((unsigned)((2 * cols + 63) / 64)), dim3(1024), 0, stream, p.part,
                       (int)groups, (uint32_t)cols, p.dw, p.db);
  return hipGetLastError();
}

}  // namespace mxq
