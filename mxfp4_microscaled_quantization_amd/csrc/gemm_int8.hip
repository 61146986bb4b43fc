// 8-bit integer GEMMs for gfx950, out = (A * W^T) scaled by a token scale and a channel
// scale:
//   acc[m,n] = sum_k qa[m,k] * qw[n,k]            int32, exact (K < 2^17)
//   t = fl32(fl32(acc) * sa[m]);  v = fl32(t * sw[n]), or fma(t, sw[n], bias[n])
//   out = v rounded to bf16 (nearest even), or v
// The sum is exact in any order, so every kernel here gives the same bits.
//
// gemm_i8_kernel, one workgroup = WM x WN waves = a (16 MJ WM) x (16 MI WN) output tile,
// 16 x 16 x 64 MFMAs:
//  * the weight tile is the MFMA A operand and the activation tile the B operand, so a
//    lane finishes with 4 consecutive output columns of one row.  Lane l holds row l & 15
//    of a fragment and K-group l >> 4 (16 bytes); both operands share that layout, so any
//    assignment of K to lane groups is valid.
//  * K advances in windows of 128 bytes per row (two MFMA steps), streamed global -> LDS
//    by buffer_load ... lds into rings of NA activation and NW weight tiles.  16-byte
//    chunk c of row r sits at c ^ ((r >> 1) & 7): the fragment reads are then free of bank
//    conflicts.
//  * ragged M and N: rows past the end are outside the buffer resource and read as zeros.
//    Ragged K: in the last window the activation chunks past K are fetched from outside
//    the resource, i.e. as zeros, which cancel whatever the weight row holds there.
#include <type_traits>
#include <utility>

#include "mxq_int8.hpp"
#include "mxq_internal.hpp"

namespace mxq {
namespace {

struct I8Params {
  const int8_t* a;
  const float* a_scales;
  const int8_t* w;
  const float* w_scales;
  const float* bias;       // or null
  void* out;
  int64_t ld_out, inc_as, inc_ws;
  int M, N, K;
  uint32_t ld_a, ld_w;
  int nwin, tiles_m, tiles_n;
  int vec;                 // rows of the output start on 16-byte boundaries
};

constexpr uint32_t kOutside = 0x80000000u;   // a byte offset past every resource here
constexpr int kWin = 128;                    // K elements (bytes) per row per window

// s_waitcnt immediate (gfx9 encoding): vmcnt <= vm, lgkmcnt <= 0, expcnt unconstrained
constexpr int wait_vm(int vm) { return (vm & 0xF) | ((vm >> 4) << 14) | (0x7 << 4); }

// Barrier without the release fence of __syncthreads(), which would drain the loads of
// later windows: the caller has waited for exactly what has to have landed.
__device__ __forceinline__ void handover_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_slot(uint32_t row, uint32_t chunk) {
  return row * 128u + ((chunk ^ ((row >> 1) & 7u)) << 4);
}

__device__ __forceinline__ void line_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds_line, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_line, 16, voff, soff, 0, 0);
}

// which of n loads spread over rd reads go out right after read k
constexpr int loads_after(int k, int n, int rd) { return (k + 1) * n / rd - k * n / rd; }

// Scheduling pattern of one MFMA region: unit I is one fragment read, then the tile loads
// that fall there, then its share of the region's MFMAs.
template <int ID, int R, int MFMAS, int VM, int I>
__device__ __forceinline__ void region_unit() {
  __builtin_amdgcn_sched_group_barrier(0x100, 1, ID);                                    // DS read
  constexpr int l = loads_after(I, VM, R);
  if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(0x020, l, ID);               // VMEM read
  constexpr int n = (I + 1) * MFMAS / R - I * MFMAS / R;
  if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x008, n, ID);               // MFMA
}
template <int ID, int R, int MFMAS, int VM, int... Is>
__device__ __forceinline__ void region_units(std::integer_sequence<int, Is...>) {
  (region_unit<ID, R, MFMAS, VM, Is>(), ...);
}

// The epilogue's arithmetic, the same in every kernel.
__device__ __forceinline__ float scaled(int acc, float sa, float sw, float bias, bool has_bias) {
#pragma clang fp contract(off)
  const float t = (float)acc * sa;
  return has_bias ? __builtin_fmaf(t, sw, bias) : t * sw;
}

// Origin of this workgroup's tile: every XCD (workgroups are dealt to them in turn) walks
// a contiguous run of tiles along N, whose activation rows then stay in its L2.
template <int BM, int BN>
__device__ __forceinline__ void i8_tile_origin(const I8Params& p, int& m0, int& n0) {
  const int nt = p.tiles_m * p.tiles_n, bid = blockIdx.x;
  const int xcd = bid & 7, q8 = nt >> 3, r8 = nt & 7;
  const int seq = xcd * q8 + min(xcd, r8) + (bid >> 3);
  m0 = seq / p.tiles_n * BM;
  n0 = seq % p.tiles_n * BN;
}

template <int MI, int MJ, int WM, int WN, int NA, int NW, bool F32OUT>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_kernel(I8Params p) {
  constexpr int WAVES = WM * WN, BM = 16 * MJ * WM, BN = 16 * MI * WN;
  constexpr uint32_t A_TILE = BM * kWin, W_TILE = BN * kWin;
  constexpr int LA = (int)(A_TILE / 1024) / WAVES, LW = (int)(W_TILE / 1024) / WAVES;   // 1 KB lines per wave
  constexpr int RD = MI + MJ, VM = LA + LW;
  static_assert(LA >= 1 && LW >= 1 && LA * WAVES * 1024 == (int)A_TILE && LW * WAVES * 1024 == (int)W_TILE, "whole lines");
  static_assert(NW >= 2 && (NA == NW || NA == NW + 1), "ring depths");
  // loads issued after the last piece of window w+1 when window w ends
  constexpr int IN_FLIGHT = (NW - 2) * VM + (NA > NW ? LA : 0);
  static_assert(IN_FLIGHT < 64 && (NW - 1) * VM + (NA > NW ? LA : 0) < 64, "vmcnt range");
  constexpr uint32_t W_BASE = NA * A_TILE;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NA * A_TILE + NW * W_TILE];

  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
  const uint32_t wm = wave % WM, wn = wave / WM;
  int m0, n0;
  i8_tile_origin<BM, BN>(p, m0, n0);
  const uint32_t rows_a = (uint32_t)min(BM, p.M - m0), rows_w = (uint32_t)min(BN, p.N - n0);
  const uint32_t bytes_a = (rows_a - 1) * p.ld_a + (uint32_t)p.K, bytes_w = (rows_w - 1) * p.ld_w + (uint32_t)p.K;
  const int8_t* base_a = p.a + (int64_t)m0 * p.ld_a;
  const int8_t* base_w = p.w + (int64_t)n0 * p.ld_w;

  // direct-to-LDS lines: LDS line q holds rows 8q .. 8q+7; lane i lands at byte 16 i, in
  // row i / 8 at slot i % 8, and fetches the chunk the swizzle maps there (whose term
  // (r >> 1) & 7 depends on the line's parity)
  const uint32_t drow = lane >> 3, dslot = lane & 7;
  const uint32_t chunk0 = (dslot ^ ((drow >> 1) & 7u)) * 16, chunk1 = (dslot ^ (((8u + drow) >> 1) & 7u)) * 16;
  const int nwin = p.nwin;
  const uint32_t last_bytes = (uint32_t)(p.K - (nwin - 1) * kWin);   // of the last window: 16 .. 128
  auto issue_a = [&](int w, int j) {
    const uint32_t line = wave * LA + j;
    const uint32_t chunk = (line & 1) ? chunk1 : chunk0;
    const uint32_t valid = w + 1 < nwin ? (uint32_t)kWin : last_bytes;
    line_to_lds(make_rsrc(base_a, w < nwin ? bytes_a : 0u), lds + (uint32_t)(w % NA) * A_TILE + line * 1024,
                chunk < valid ? drow * p.ld_a + chunk : kOutside, (uint32_t)w * kWin + line * 8 * p.ld_a);
  };
  auto issue_w = [&](int w, int j) {
    const uint32_t line = wave * LW + j;
    line_to_lds(make_rsrc(base_w, w < nwin ? bytes_w : 0u), lds + W_BASE + (uint32_t)(w % NW) * W_TILE + line * 1024,
                drow * p.ld_w + ((line & 1) ? chunk1 : chunk0), (uint32_t)w * kWin + line * 8 * p.ld_w);
  };

  v4i acc[MI][MJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  v4i f0[RD], f1[RD];
  const uint32_t r16 = lane & 15, g = lane >> 4;
  // step-t fragments of window w: weight rows, then activation rows; after(k) follows read k
  auto read = [&](v4i(&f)[RD], int w, int t, auto&& after) {
    const uint8_t* la = lds + (uint32_t)(w % NA) * A_TILE;
    const uint8_t* lw = lds + W_BASE + (uint32_t)(w % NW) * W_TILE;
    const uint32_t chunk = g + 4 * t;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      f[i] = *reinterpret_cast<const v4i*>(lw + lds_slot(wn * (16 * MI) + 16 * i + r16, chunk));
      after(i);
    }
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      f[MI + j] = *reinterpret_cast<const v4i*>(la + lds_slot(wm * (16 * MJ) + 16 * j + r16, chunk));
      after(MI + j);
    }
  };
  auto step = [&](const v4i(&f)[RD]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[i], f[MI + j], acc[i][j], 0, 0, 0);
  };

  if (nwin > 0) {
    // prologue, in the order of the steady state: the weight tile of a window, then the
    // activation tile NA - NW windows further on
    if constexpr (NA > NW)
#pragma unroll
      for (int j = 0; j < LA; ++j) issue_a(0, j);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
#pragma unroll
      for (int j = 0; j < LW; ++j) issue_w(w, j);
#pragma unroll
      for (int j = 0; j < LA; ++j) issue_a(w + NA - NW, j);
    }
    __builtin_amdgcn_s_waitcnt(wait_vm((NW - 1) * VM + (NA > NW ? LA : 0)));   // window 0 landed
    handover_barrier();
    read(f0, 0, 0, [](int) {});
    // One window: step 0 under the reads of step 1; the hand-over waits for window w+1 and
    // releases this window's slots; step 1 under the reads of window w+1's step 0 and the
    // loads that refill those slots.  Windows past the last are loads outside the resource:
    // no memory is read for them, and the count of loads in flight stays what the waits assume.
    for (int w = 0; w < nwin; ++w) {
      read(f1, w, 1, [](int) {});
      step(f0);
      region_units<0, RD, MI * MJ, 0>(std::make_integer_sequence<int, RD>{});
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm(IN_FLIGHT));
      handover_barrier();
      __builtin_amdgcn_sched_barrier(0);
      read(f0, w + 1, 0, [&](int k) {
#pragma unroll
        for (int l = 0; l < VM; ++l)
          if (l >= k * VM / RD && l < (k + 1) * VM / RD) {
            if (l < LW)
              issue_w(w + NW, l);
            else
              issue_a(w + NA, l - LW);
          }
      });
      step(f1);
      region_units<1, RD, MI * MJ, VM>(std::make_integer_sequence<int, RD>{});
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(0);   // nothing may land in LDS after this workgroup has ended
  }

  // ---- epilogue: lane l holds columns 4g .. 4g+3 of row l & 15 of every block ----
  const bool has_bias = p.bias != nullptr;
  float sw[MI][4], bs[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = min(n0 + (int)(wn * (16 * MI) + 16 * i + 4 * g) + e, p.N - 1);
      sw[i][e] = p.w_scales[n * p.inc_ws];
      bs[i][e] = has_bias ? p.bias[n] : 0.0f;
    }
  const int mw = m0 + (int)wm * (16 * MJ), nw = n0 + (int)wn * (16 * MI);
  const bool whole = p.vec && n0 + BN <= p.N;
  if (!F32OUT && whole) {
    // park the wave's sub-tile in LDS (16-byte chunk c of row r at c ^ (r & (CPR - 1))) and
    // store whole row segments
    constexpr uint32_t CPR = 2 * MI, RB = 32 * MI;   // chunks, bytes per row of the sub-tile
    static_assert((CPR & (CPR - 1)) == 0 && CPR <= 64, "a power of two");
    static_assert(WAVES * 16 * MJ * RB <= sizeof(lds), "staging fits the rings");
    __syncthreads();
    uint8_t* sub = lds + wave * (16 * MJ * RB);
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const uint32_t row = 16 * j + r16;
      const int m = mw + (int)row;
      const float sa = p.a_scales[min(m, p.M - 1) * p.inc_as];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][j][e], sa, sw[i][e], bs[i][e], has_bias);
        const uint32_t c = 2 * i + (g >> 1);
        *reinterpret_cast<v2u*>(sub + row * RB + ((c ^ (row & (CPR - 1))) << 4) + 8 * (g & 1)) =
            v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
    constexpr uint32_t RPI = 64 / CPR;               // rows per store instruction
    uint16_t* obase = static_cast<uint16_t*>(p.out) + (int64_t)mw * p.ld_out + nw;
#pragma unroll
    for (uint32_t q = 0; q < 16 * MJ / RPI; ++q) {
      const uint32_t row = RPI * q + lane / CPR, c = lane % CPR;
      const v4i v = *reinterpret_cast<const v4i*>(sub + row * RB + ((c ^ (row & (CPR - 1))) << 4));
      if (mw + (int)row < p.M) *reinterpret_cast<v4i*>(obase + (int64_t)row * p.ld_out + c * 8) = v;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int m = mw + (int)(16 * j + r16);
    if (m >= p.M) continue;
    const float sa = p.a_scales[m * p.inc_as];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int n = nw + 16 * i + 4 * (int)g;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][j][e], sa, sw[i][e], bs[i][e], has_bias);
      if constexpr (F32OUT) {
        float* o = static_cast<float*>(p.out) + (int64_t)m * p.ld_out + n;
        if (whole) {
          *reinterpret_cast<v4f*>(o) = v4f{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) o[e] = v[e];
        }
      } else {
        uint16_t* o = static_cast<uint16_t*>(p.out) + (int64_t)m * p.ld_out + n;
        const unsigned lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
        if (n + 0 < p.N) o[0] = (uint16_t)lo;
        if (n + 1 < p.N) o[1] = (uint16_t)(lo >> 16);
        if (n + 2 < p.N) o[2] = (uint16_t)hi;
        if (n + 3 < p.N) o[3] = (uint16_t)(hi >> 16);
      }
    }
  }
}

// ---------------------------------------------------------------------------------
// A few tokens: the weights' bytes are what counts, each used by one workgroup only, so
// they go from memory to registers.  One workgroup = 16 NI channels x 16 MJ tokens, its
// WAVES waves splitting K (window w to wave w mod WAVES) with U windows of loads in flight
// each; the partial sums meet in LDS (integers: the order changes nothing).
template <int NI, int MJ, int WAVES, int U, bool F32OUT>
__global__ __launch_bounds__(64 * WAVES) void gemm_i8_few_kernel(I8Params p) {
  __shared__ __attribute__((aligned(16))) v4i part[WAVES][NI][MJ][64];
  const uint32_t tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(tid >> 6));
  const int n0 = (int)(blockIdx.x % (unsigned)p.tiles_n) * (16 * NI), m0 = (int)(blockIdx.x / (unsigned)p.tiles_n) * (16 * MJ);
  const uint32_t rows_a = (uint32_t)min(16 * MJ, p.M - m0), rows_w = (uint32_t)min(16 * NI, p.N - n0);
  const bool any = p.nwin > 0;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + (int64_t)m0 * p.ld_a, any ? (rows_a - 1) * p.ld_a + (uint32_t)p.K : 0u);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + (int64_t)n0 * p.ld_w, any ? (rows_w - 1) * p.ld_w + (uint32_t)p.K : 0u);
  v4i acc[NI][MJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  for (int w0 = wave; w0 < p.nwin; w0 += WAVES * U) {
    v4i fw[U][2][NI], fa[U][2][MJ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // lane group g takes chunk g of each 64-byte half window; past K both operands read
        // from outside their resource, i.e. zeros
        const uint32_t k = (uint32_t)(w0 + u * WAVES) * kWin + 64u * t + 16u * g;
        const bool in = k < (uint32_t)p.K;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          fw[u][t][i] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, in ? (16 * i + r16) * p.ld_w + k : kOutside, 0, 0));
#pragma unroll
        for (int j = 0; j < MJ; ++j)
          fa[u][t][j] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? (16 * j + r16) * p.ld_a + k : kOutside, 0, 0));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < MJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][t][i], fa[u][t][j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) part[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  // thread e takes output (token e / (16 NI), channel e % (16 NI)) of the tile
  const bool has_bias = p.bias != nullptr;
  for (uint32_t e = tid; e < 16 * NI * rows_a; e += 64 * WAVES) {
    const uint32_t m = e / (16 * NI), n = e % (16 * NI);
    if (n >= rows_w) continue;
    const uint32_t from = ((n & 15) >> 2) * 16 + (m & 15);
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += reinterpret_cast<const int*>(&part[w][n >> 4][m >> 4][from])[n & 3];
    const int64_t mm = m0 + (int)m, nn = n0 + (int)n;
    const float v = scaled(sum, p.a_scales[mm * p.inc_as], p.w_scales[nn * p.inc_ws], has_bias ? p.bias[nn] : 0.0f, has_bias);
    if constexpr (F32OUT)
      static_cast<float*>(p.out)[mm * p.ld_out + nn] = v;
    else
      static_cast<uint16_t*>(p.out)[mm * p.ld_out + nn] = (uint16_t)pack_bf16x2(v, 0.0f);
  }
}

}  // namespace

hipError_t launch_gemm_w8a8(const int8_t* a, int64_t ld_a, const float* a_scales, int64_t inc_as, const int8_t* w,
                            int64_t ld_w, const float* w_scales, int64_t inc_ws, const float* bias, int64_t M,
                            int64_t N, int64_t K, void* out, bool f32_out, int64_t ld_out, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  I8Params p;
  p.a = a;
  p.a_scales = a_scales;
  p.w = w;
  p.w_scales = w_scales;
  p.bias = bias;
  p.out = out;
  p.ld_out = ld_out;
  p.inc_as = inc_as;
  p.inc_ws = inc_ws;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.ld_a = (uint32_t)ld_a;
  p.ld_w = (uint32_t)ld_w;
  p.nwin = (int)((K + kWin - 1) / kWin);
  p.vec = (ld_out * (f32_out ? 4 : 2)) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  auto tile = [&](auto kernel, int bm, int bn, int waves) {
    p.tiles_m = (int)((M + bm - 1) / bm);
    p.tiles_n = (int)((N + bn - 1) / bn);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.tiles_m * p.tiles_n)), dim3(64 * waves), 0, stream, p);
  };
  auto pick = [&](auto f_tag) {
    constexpr bool F = decltype(f_tag)::value;
    if (M <= 16)
      tile(gemm_i8_few_kernel<1, 1, 8, 4, F>, 16, 16, 8);
    else if (M <= 32)
      tile(gemm_i8_few_kernel<1, 2, 8, 4, F>, 32, 16, 8);
    else if (M <= 64)
      tile(gemm_i8_few_kernel<2, 4, 8, 2, F>, 64, 32, 8);
    else
      tile(gemm_i8_kernel<4, 8, 2, 4, 3, 2, F>, 256, 256, 8);
  };
  f32_out ? pick(std::true_type{}) : pick(std::false_type{});
  return hipGetLastError();
}

}  // namespace mxq
