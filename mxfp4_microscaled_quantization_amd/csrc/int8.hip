// 8-bit row quantization (one scale for each row: a token of the activations, an output
// channel of the weights) and its dequantization.  The rule is in mxq_int8.hpp.
//
// Both are bandwidth-bound element kernels.  The quantizer needs a row's maximum before
// its first code, so a row is held in registers between the two: T = 64 W threads take
// one row, C units of 8 elements each, all loads first, one reduction (DPP inside a wave,
// LDS across the W waves), then the codes.  Rows past T * 8 * C elements of the largest
// variant are read twice; rows of up to 32 units (heads) share a wave.
// Measured: 75600 x 13824 bf16 0.516 ms (6.1 TB/s; a row over 4 waves x 8 units 0.52, over
// 16 x 2 0.57) and binary32 0.888 ms (5.9 TB/s), 75600 x 5120 bf16 0.184 ms (6.3 TB/s) and
// binary32 0.326 ms (5.9 TB/s), 300000 x 128 bf16 0.022 ms (5.2 TB/s; 0.0185 from the memory-side
// cache, a wave for each row 0.058); dequantization of 75600 x 13824 0.567 ms (5.5 TB/s), of
// 300000 x 128 0.0228 ms (5.1 TB/s; 0.018 from the memory-side cache).
#include <type_traits>

#include "mxq_int8.hpp"
#include "mxq_internal.hpp"

namespace mxq {
namespace {

constexpr int kDqI8Threads = 1024;
constexpr int kDqI8Unroll = 4;

// W waves per row; C units per thread held in registers.  Workgroups of max(W, 4) waves:
// with W == 1 each of the four waves has a row of its own and nothing is synchronized.
template <bool F32, bool STREAM, int W, int C>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void int8_quantize_kernel(
    const void* __restrict__ x, int64_t rows, uint32_t units, int64_t ld_x, int8_t* __restrict__ codes,
    int64_t ld_codes, float* __restrict__ scales) {
  constexpr int T = 64 * W, RPB = W < 4 ? 4 / W : 1;
  static_assert(W == 1 || W >= 4, "a workgroup holds whole rows");
  __shared__ unsigned red[2][W];
  const uint32_t tid = threadIdx.x % T, sub = threadIdx.x / T, lane = threadIdx.x & 63, wave = tid >> 6;
  int par = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < rows; row += (int64_t)gridDim.x * RPB, par ^= 1) {
    Unit<F32> u[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      u[c] = i < units ? load_unit<F32, STREAM>(x, row * ld_x + (int64_t)i * 8) : zero_unit<F32>();
    }
    unsigned m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) m = max(m, unit_max<F32>(u[c]));
    m = wave_max_u32(m);
    if constexpr (W > 1) {
      // two slots in turn: a wave may reach the next row's store while another still reads
      if (lane == 0) red[par][wave] = m;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < W; ++k) m = max(m, red[par][k]);
    }
    const Int8Scale sc = int8_scale(m);
    if (tid == 0) scales[row] = sc.s;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      if (i < units)
        __builtin_nontemporal_store(unit_codes<F32>(u[c], sc),
                                    reinterpret_cast<v2u*>(codes + row * ld_codes + (int64_t)i * 8));
    }
  }
}

// Rows of up to G units, 64 / G of them in a wave: lane l of a group has unit l, R rows of
// each group in flight.
template <bool F32, bool STREAM, int G>
__global__ __launch_bounds__(256) void int8_quantize_short_kernel(const void* __restrict__ x, int64_t rows,
                                                                  uint32_t units, int64_t ld_x,
                                                                  int8_t* __restrict__ codes, int64_t ld_codes,
                                                                  float* __restrict__ scales) {
  constexpr int PER = 256 / G, R = 4;   // rows of the workgroup at once, passes in flight
  const uint32_t l = threadIdx.x % G;
  const bool own = l < units;
  for (int64_t r0 = (int64_t)blockIdx.x * (PER * R) + threadIdx.x / G; r0 < rows; r0 += (int64_t)gridDim.x * (PER * R)) {
    Unit<F32> u[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t row = r0 + k * PER;
      u[k] = own && row < rows ? load_unit<F32, STREAM>(x, row * ld_x + (int64_t)l * 8) : zero_unit<F32>();
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t row = r0 + k * PER;
      unsigned m = unit_max<F32>(u[k]);
      m = G == 8 ? row8_max_u32(m) : row16_max_u32(m);
      if constexpr (G == 32) m = max(m, (unsigned)__shfl_xor((int)m, 16));
      const Int8Scale sc = int8_scale(m);
      if (row < rows) {
        if (l == 0) scales[row] = sc.s;
        if (own)
          __builtin_nontemporal_store(unit_codes<F32>(u[k], sc), reinterpret_cast<v2u*>(codes + row * ld_codes + (int64_t)l * 8));
      }
    }
  }
}

// Rows longer than the registers of 16 waves hold: the second reading comes from the caches.
template <bool F32>
__global__ __launch_bounds__(1024) void int8_quantize_long_kernel(const void* __restrict__ x, int64_t rows,
                                                                  uint32_t units, int64_t ld_x,
                                                                  int8_t* __restrict__ codes, int64_t ld_codes,
                                                                  float* __restrict__ scales) {
  __shared__ unsigned red[2][16];
  const uint32_t tid = threadIdx.x;
  int par = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, par ^= 1) {
    unsigned m = 0;
    for (uint32_t i = tid; i < units; i += 1024) m = max(m, unit_max<F32>(load_unit<F32, false>(x, row * ld_x + (int64_t)i * 8)));
    m = wave_max_u32(m);
    if ((tid & 63) == 0) red[par][tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) m = max(m, red[par][k]);
    const Int8Scale sc = int8_scale(m);
    if (tid == 0) scales[row] = sc.s;
    for (uint32_t i = tid; i < units; i += 1024)
      *reinterpret_cast<v2u*>(codes + row * ld_codes + (int64_t)i * 8) =
          unit_codes<F32>(load_unit<F32, false>(x, row * ld_x + (int64_t)i * 8), sc);
  }
}

// y = bf16_RNE(fl32(q * s_r)): a code is exact in binary32, one multiply, one rounding to
// bf16.  8 codes per lane and unit.
__global__ __launch_bounds__(kDqI8Threads) void int8_dequantize_kernel(const int8_t* __restrict__ codes,
                                                                       int64_t ld_codes,
                                                                       const float* __restrict__ scales,
                                                                       uint16_t* __restrict__ y, int64_t ld_y,
                                                                       uint32_t units_per_row, uint32_t total_units) {
  const uint64_t stride = (uint64_t)gridDim.x * kDqI8Threads * kDqI8Unroll;
  for (uint64_t g0 = (uint64_t)blockIdx.x * kDqI8Threads * kDqI8Unroll + threadIdx.x; g0 < total_units; g0 += stride) {
    v2u c[kDqI8Unroll];
    float s[kDqI8Unroll];
    int64_t yo[kDqI8Unroll];
    bool ok[kDqI8Unroll];
#pragma unroll
    for (int u = 0; u < kDqI8Unroll; ++u) {
      const uint64_t g64 = g0 + (uint64_t)u * kDqI8Threads;
      ok[u] = g64 < total_units;
      const uint32_t g = ok[u] ? (uint32_t)g64 : 0u;
      const uint32_t row = g / units_per_row, col = (g - row * units_per_row) * 8u;
      yo[u] = (int64_t)row * ld_y + col;
      c[u] = *reinterpret_cast<const v2u*>(codes + (int64_t)row * ld_codes + col);
      s[u] = scales[row];
    }
#pragma unroll
    for (int u = 0; u < kDqI8Unroll; ++u) {
      v4i o;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int w = (int)(c[u][h >> 1] >> (16 * (h & 1)));
        o[h] = (int)pack_bf16x2((float)(int8_t)w * s[u], (float)(int8_t)(w >> 8) * s[u]);
      }
      if (ok[u]) __builtin_nontemporal_store(o, reinterpret_cast<v4i*>(y + yo[u]));
    }
  }
}

}  // namespace

hipError_t launch_quantize_int8(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld_x, int8_t* codes,
                                int64_t ld_codes, float* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const uint32_t units = (uint32_t)(cols / 8);
  auto go = [&](auto kernel, int threads, int rows_per_block) {
    const int64_t blocks = (rows + rows_per_block - 1) / rows_per_block;
    const int64_t cap = (int64_t)1 << 20;   // blocks * threads stays below 2^32
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(threads), 0, stream, x, rows, units,
                       ld_x, codes, ld_codes, scales);
  };
  auto pick = [&](auto f_tag, auto s_tag) {
    constexpr bool F = decltype(f_tag)::value, S = decltype(s_tag)::value;
    if (units <= 8)
      go(int8_quantize_short_kernel<F, S, 8>, 256, 32 * 4);
    else if (units <= 16)
      go(int8_quantize_short_kernel<F, S, 16>, 256, 16 * 4);
    else if (units <= 32)
      go(int8_quantize_short_kernel<F, S, 32>, 256, 8 * 4);
    else if (units <= 64)
      go(int8_quantize_kernel<F, S, 1, 1>, 256, 4);
    else if (units <= 128)
      go(int8_quantize_kernel<F, S, 1, 2>, 256, 4);
    else if (units <= 256)
      go(int8_quantize_kernel<F, S, 1, 4>, 256, 4);
    else if (units <= 256 * 4)
      go(int8_quantize_kernel<F, S, 4, 4>, 256, 1);
    else if (units <= 512 * 4)
      go(int8_quantize_kernel<F, S, 8, 4>, 512, 1);
    else if (units <= 1024 * 8)
      go(int8_quantize_kernel<F, S, 16, 8>, 1024, 1);
    else
      go(int8_quantize_long_kernel<F>, 1024, 1);
  };
  // An input that fits the 256 MB of memory-side cache may be there still from the kernel
  // that wrote it, and ordinary loads find it (20000 x 5120 bf16: 43 us, 47 with streaming
  // loads); a larger one is only slowed down by passing through (75600 x 5120: 200 and 180 us).
  const bool stream_loads = rows * cols * (f32 ? 4 : 2) > ((int64_t)256 << 20);
  using T = std::true_type;
  using N = std::false_type;
  if (f32)
    stream_loads ? pick(T{}, T{}) : pick(T{}, N{});
  else
    stream_loads ? pick(N{}, T{}) : pick(N{}, N{});
  return hipGetLastError();
}

hipError_t launch_dequantize_int8(const int8_t* codes, int64_t ld_codes, const float* scales, int64_t rows,
                                  int64_t cols, uint16_t* y, int64_t ld_y, hipStream_t stream) {
  const int64_t upr = cols / 8;
  const int64_t total = rows * upr;       // below 2^32 (the API bounds rows * cols / 8)
  if (total == 0) return hipSuccess;
  const int64_t per = (int64_t)kDqI8Threads * kDqI8Unroll, cap = 256 * 64;
  const int64_t blocks = (total + per - 1) / per;
  hipLaunchKernelGGL(int8_dequantize_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(kDqI8Threads), 0,
                     stream, codes, ld_codes, scales, y, ld_y, (uint32_t)upr, (uint32_t)total);
  return hipGetLastError();
}

}  // namespace mxq
