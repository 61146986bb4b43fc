// Weight gradient of the 8-bit product from the codes that its forward pass took:
//   dW[n,k] = sum_m dy[m,n] * bf16(code[m,k] * scale[m])
// with dy in bf16 and the sum in binary32.  The rounding of code * scale to bf16 (relative
// error 2^-9 at most, beside the half step of the codes themselves) is the one of
// mxq_dequantize_int8: the matrix cores take it as an operand, and the products are exact.
//
// The codes are widened into a workspace first.  The product contracts over rows of both
// operands, while an MFMA takes 8 consecutive values of the contraction in a lane: fragments
// come from LDS by ds_read_b64_tr_b16, in which 16 lanes read 4 rows of 16 columns and each
// gets the 4 values of one column.
#include <type_traits>
#include <utility>

#include "mxq_device.hpp"
#include "mxq_internal.hpp"

namespace mxq {
namespace {

constexpr int kWinRows = 64;   // rows of both operands in LDS at once: two MFMA steps

struct GradParams {
  const uint16_t* dy;
  const uint16_t* x;
  void* out;
  float* part;              // sums of the parts of M, [splits][N][K]
  int64_t ld_dy, ld_x, ld_out;
  int M, N, K;
  int nwin, tiles_n, tiles_k, splits;
  int accumulate, vec;      // vec: rows of the output are aligned for whole stores of 4
};

enum { GRAD_BF16 = 0, GRAD_F32 = 1, GRAD_PART = 2 };

// MI x MJ fragments of 16 x 16 outputs (k, n) in a wave, WK x WN waves.
template <int MI, int MJ, int WK, int WN>
struct GradTile {
  static constexpr int THREADS = 64 * WK * WN, BK = 16 * MI * WK, BN = 16 * MJ * WN;
  static constexpr uint32_t X_TILE = kWinRows * BK * 2, Y_TILE = kWinRows * BN * 2;
};

__device__ __forceinline__ void grad_line_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds_line, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_line, 16, voff, soff, 0, 0);
}

typedef short v4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v2u read_transposed(const uint8_t* lds) {
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)lds));
}

// 4 sums of columns k .. k + 3 of row n (some of them past K unless `whole`).
template <int OUT>
__device__ __forceinline__ void store_sums(const GradParams& p, int n, int k, v4f v) {
  if constexpr (OUT == GRAD_PART) {
    // K is a multiple of 16, and so is every part's row
    *reinterpret_cast<v4f*>(p.part + ((int64_t)blockIdx.y * p.N + n) * p.K + k) = v;
  } else if constexpr (OUT == GRAD_F32) {
    float* o = static_cast<float*>(p.out) + (int64_t)n * p.ld_out + k;
    if (p.vec) {
      if (p.accumulate) v += *reinterpret_cast<const v4f*>(o);
      *reinterpret_cast<v4f*>(o) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = p.accumulate ? o[e] + v[e] : v[e];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + (int64_t)n * p.ld_out + k;
    if (p.accumulate)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += __uint_as_float((unsigned)o[e] << 16);
    const unsigned lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (p.vec) {
      *reinterpret_cast<v2u*>(o) = v2u{lo, hi};
    } else {
      o[0] = (uint16_t)lo;
      o[1] = (uint16_t)(lo >> 16);
      o[2] = (uint16_t)hi;
      o[3] = (uint16_t)(hi >> 16);
    }
  }
}

template <int OUT, int MI, int MJ, int WK, int WN>
__global__ __launch_bounds__(64 * WK * WN, 1) void grad_weight_kernel(GradParams p) {
  using T = GradTile<MI, MJ, WK, WN>;
  constexpr int WAVES = WK * WN;
  constexpr int LX = (int)(T::X_TILE / 1024) / WAVES, LY = (int)(T::Y_TILE / 1024) / WAVES;   // 1 KB lines per wave
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::X_TILE + T::Y_TILE];
  uint8_t* const lx = lds;
  uint8_t* const ly = lds + T::X_TILE;

  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
  const uint32_t wk = wave % WK, wn = wave / WK;
  const int tile = blockIdx.x, k0 = tile / p.tiles_n * T::BK, n0 = tile % p.tiles_n * T::BN;
  const int w_lo = OUT == GRAD_PART ? (int)((int64_t)blockIdx.y * p.nwin / p.splits) : 0;
  const int w_hi = OUT == GRAD_PART ? (int)((int64_t)(blockIdx.y + 1) * p.nwin / p.splits) : p.nwin;

  // A window's rows start at r0: a resource of its own for each (64-bit base, offsets below 2^31)
  auto rows_of = [&](const uint16_t* base, int64_t ld, int cols, int col0, int w) {
    const int left = p.M - w * kWinRows, rows = left < kWinRows ? left : kWinRows;
    const uint32_t bytes = rows > 0 ? (uint32_t)(((int64_t)(rows - 1) * ld + cols - col0) * 2) : 0u;
    return make_rsrc(base + (int64_t)w * kWinRows * ld + col0, bytes);
  };
  // LDS: rows of BC columns, 32-byte unit u of row r at u ^ (r & 7) (the 8 rows that half a wave
  // reads at one column are then on distinct banks)
  auto fill = [&](__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t ld, auto bc_tag, auto lines_tag) {
    constexpr uint32_t BC = decltype(bc_tag)::value, CPR = BC / 8, RPL = 64 / CPR;   // 16-byte chunks per row, rows per line
    constexpr int L = decltype(lines_tag)::value;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const uint32_t line = wave * L + j, row = line * RPL + lane / CPR, slot = lane % CPR;
      grad_line_to_lds(r, to + line * 1024, row * ld * 2 + ((slot ^ ((row & 7) << 1)) << 4), 0);
    }
  };
  // the fragment of 16 columns from c0, tokens 32 t + 4 g + (0 .. 3) and 16 more, g = lane / 16
  auto read = [&](const uint8_t* from, uint32_t pitch, uint32_t c0, int t) {
    const uint32_t q = lane & 15, row = 32 * t + 4 * (lane >> 4) + (q >> 2);
    const uint32_t unit = c0 / 16, at = row * pitch + ((unit ^ (row & 7)) << 5) + 8 * (q & 3);
    const v2u lo = read_transposed(from + at), hi = read_transposed(from + at + 16 * pitch);
    return v4u{lo[0], lo[1], hi[0], hi[1]};
  };

  v4f acc[MI][MJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  for (int w = w_lo; w < w_hi; ++w) {
    __syncthreads();
    fill(rows_of(p.x, p.ld_x, p.K, k0, w), lx, (uint32_t)p.ld_x, std::integral_constant<uint32_t, T::BK>{}, std::integral_constant<int, LX>{});
    fill(rows_of(p.dy, p.ld_dy, p.N, n0, w), ly, (uint32_t)p.ld_dy, std::integral_constant<uint32_t, T::BN>{}, std::integral_constant<int, LY>{});
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      v4u fx[MI], fy[MJ];
#pragma unroll
      for (int i = 0; i < MI; ++i) fx[i] = read(lx, T::BK * 2, (wk * MI + i) * 16, t);
#pragma unroll
      for (int j = 0; j < MJ; ++j) fy[j] = read(ly, T::BN * 2, (wn * MJ + j) * 16, t);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fx[i]),
                                                              __builtin_bit_cast(bf16x8, fy[j]), acc[i][j], 0, 0, 0);
    }
  }
  // lane l holds columns k 4 (l / 16) .. + 3 of row n l % 16 of each block; K is a multiple of 16
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int n = n0 + (int)(wn * MJ + j) * 16 + (int)(lane & 15);
    if (n < p.N) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int k = k0 + (int)(wk * MI + i) * 16 + 4 * (int)(lane >> 4);
        if (k < p.K) store_sums<OUT>(p, n, k, acc[i][j]);
      }
    }
  }
}

// Joins the parts of M in order; 4 columns for each thread.
template <int OUT>
__global__ __launch_bounds__(256) void grad_weight_sums_kernel(GradParams p) {
  const int64_t quads = (int64_t)p.N * (p.K / 4);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < p.splits; ++s) v += *reinterpret_cast<const v4f*>(p.part + ((int64_t)s * quads + i) * 4);
  const int n = (int)(i / (p.K / 4)), k = (int)(i - (int64_t)n * (p.K / 4)) * 4;
  store_sums<OUT>(p, n, k, v);
}

struct GradPlan {
  int big, splits, tiles_n, tiles_k;
};
GradPlan plan_grad(int64_t M, int64_t N, int64_t K) {
  GradPlan g;
  const int64_t t256 = ((N + 255) / 256) * ((K + 255) / 256);
  g.big = t256 >= 128;
  const int64_t b = g.big ? 256 : 128, nwin = (M + kWinRows - 1) / kWinRows;
  g.tiles_n = (int)((N + b - 1) / b);
  g.tiles_k = (int)((K + b - 1) / b);
  const int64_t tiles = (int64_t)g.tiles_n * g.tiles_k;
  int64_t s = 1;
  while (!g.big && tiles * s * 2 <= 512 && nwin / (s * 2) >= 4) s *= 2;
  g.splits = (int)s;
  return g;
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t grad_weight_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const GradPlan g = plan_grad(M, N, K);
  return round256((size_t)M * (size_t)K * 2) + (g.splits > 1 ? (size_t)g.splits * (size_t)N * (size_t)K * 4 : 0);
}

hipError_t launch_grad_weight_int8(const uint16_t* dy, int64_t ld_dy, const int8_t* codes, int64_t ld_codes,
                                   const float* scales, int64_t M, int64_t N, int64_t K, void* out, bool f32_out,
                                   int64_t ld_out, bool accumulate, void* workspace, hipStream_t stream) {
  if (N == 0 || K == 0 || (M == 0 && accumulate)) return hipSuccess;
  const GradPlan g = plan_grad(M, N, K);
  uint16_t* x = static_cast<uint16_t*>(workspace);
  const hipError_t e = launch_dequantize_int8(codes, ld_codes, scales, M, K, x, K, stream);
  if (e != hipSuccess) return e;
  GradParams p;
  p.dy = dy;
  p.x = x;
  p.out = out;
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + round256((size_t)M * (size_t)K * 2));
  p.ld_dy = ld_dy;
  p.ld_x = K;
  p.ld_out = ld_out;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.nwin = (int)((M + kWinRows - 1) / kWinRows);
  p.tiles_n = g.tiles_n;
  p.tiles_k = g.tiles_k;
  p.splits = g.splits;
  p.accumulate = accumulate;
  const uintptr_t step = f32_out ? 4 : 2;
  p.vec = reinterpret_cast<uintptr_t>(out) % (4 * step) == 0 && ld_out % 4 == 0;
  auto go = [&](auto out_tag) {
    constexpr int OUT = decltype(out_tag)::value;
    const dim3 grid((unsigned)(g.tiles_n * g.tiles_k), (unsigned)g.splits);
    if (g.big)
      hipLaunchKernelGGL((grad_weight_kernel<OUT, 4, 8, 4, 2>), grid, dim3(512), 0, stream, p);
    else
      hipLaunchKernelGGL((grad_weight_kernel<OUT, 2, 4, 4, 2>), grid, dim3(512), 0, stream, p);
  };
  using B = std::integral_constant<int, GRAD_BF16>;
  using F = std::integral_constant<int, GRAD_F32>;
  using P = std::integral_constant<int, GRAD_PART>;
  if (g.splits > 1) {
    go(P{});
    const int64_t blocks = (N * (K / 4) + 255) / 256;
    if (f32_out)
      hipLaunchKernelGGL(grad_weight_sums_kernel<GRAD_F32>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL(grad_weight_sums_kernel<GRAD_BF16>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
  } else {
    f32_out ? go(F{}) : go(B{});
  }
  return hipGetLastError();
}

}  // namespace mxq
