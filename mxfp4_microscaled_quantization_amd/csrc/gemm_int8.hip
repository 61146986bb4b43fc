// 8-bit integer GEMMs for gfx950, out = (A * W^T) scaled by a token scale and a channel
// scale:
//   acc[m,n] = sum_k qa[m,k] * qw[n,k]            int32, exact (K < 2^17)
//   t = fl32(fl32(acc) * sa[m]);  v = fl32(t * sw[n]), or fma(t, sw[n], bias[n])
//   out = v rounded to bf16 (nearest even), or v
// The sum is exact in any order, so every kernel here gives the same bits.
//
// i8_tile, one workgroup = WM x WN waves = a (16 MJ WM) x (16 MI WN) output tile,
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
//  * rows that do not start on a cache line (128 bytes): a window of such a row takes three
//    half lines instead of two, and the path of the loads into LDS is what bounds the smaller
//    tiles.  Their SHIFT form loads whole lines, block w of a row being its line w, and a
//    fragment read takes its chunk from block w or w + 1, which the ring holds both (pitches
//    are multiples of 16, so that a row's offset in its line is the same every 8 rows).
//
// What bounds it: power on large shapes.  75600 x 5120 x 13824 takes 3.92 to 3.95 ms on codes of
// normal values, 4.05 ms on uniform ones, and 3.75 to 4.18 ms over all GPUs and profiled runs (2.56 to
// 2.86 POP/s), with the matrix cores 75 % busy; the same MFMAs from registers alone run at 3.87
// POP/s on such codes.  Where each CU has a tile or two, the latencies at a tile's ends and the 64
// bytes a clock that a CU's loads into LDS take (512 x 5120 x 5120: 28 us, 0.96 POP/s); with few
// rows the weights' bytes (48 x 13824 x 5120, K in 6 parts: 20.5 us, 3.5 TB/s; 18.0 us where the
// memory-side cache holds the weights).
#include <type_traits>
#include <utility>

#include "mxq_int8.hpp"
#include "mxq_internal.hpp"
#include "w8a8_plan.hpp"

namespace mxq {
namespace {

struct I8Params {
  const int8_t* a;
  const float* a_scales;
  const int8_t* w;
  const float* w_scales;
  const float* bias;       // or null
  void* out;
  const void* x;           // unquantized activations, and their row pitch in elements
  int64_t ld_x;
  int64_t ld_out, inc_as, inc_ws;
  int M, N, K;
  uint32_t ld_a, ld_w;
  int nwin, tiles_m, tiles_n;
  int* part;               // int32 sums of the parts of K, [splits][M][ld_part]
  int splits, ld_part;
  int whole;               // gemm_i8_tail_kernel: tiles in whole rounds
  int vec;                 // rows of the output start on 16-byte boundaries
  int past;                // rows are stored past the caches
  int vec_channels;        // channel scales and biases are contiguous and 16-byte aligned
};

constexpr uint32_t kOutside = 0x80000000u;   // a byte offset past every resource here

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

// f(0) && f(1) && ... && f(N - 1), the arguments as integral constants.
template <class F, int... Is>
__device__ __forceinline__ bool each_of(F&& f, std::integer_sequence<int, Is...>) {
  return (f(std::integral_constant<int, Is>{}) && ...);
}
template <int N, class F>
__device__ __forceinline__ bool each(F&& f) {
  return each_of(f, std::make_integer_sequence<int, N>{});
}

// The epilogue's arithmetic, the same in every kernel.
__device__ __forceinline__ float scaled(int acc, float sa, float sw, float bias, bool has_bias) {
#pragma clang fp contract(off)
  const float t = (float)acc * sa;
  return has_bias ? __builtin_fmaf(t, sw, bias) : t * sw;
}

// Origin of tile `seq` of nt: bands of kBand rows of tiles, in which the index runs down the
// rows first.  Every XCD (workgroups are dealt to them in turn) walks a contiguous run, so 4
// rows of tiles by 8 columns run at once on its 32 CUs and share their operands in its L2
// (2 % to 6 % faster than one row by 32 at 75600 x 5120 x 13824 and 3584 x 5120 x 15360, and
// than 8 by 4 at long K).
constexpr int kBand = 4;

__device__ __forceinline__ int xcd_run(int bid, int nt) {
  const int xcd = bid & 7, q8 = nt >> 3, r8 = nt & 7;
  return xcd * q8 + min(xcd, r8) + (bid >> 3);
}

__device__ __forceinline__ void tile_at(const I8Params& p, int seq, int& tm, int& tn) {
  const int band = seq / (kBand * p.tiles_n), first = band * kBand, rows = min(kBand, p.tiles_m - first);
  const int in = seq - band * kBand * p.tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// Scales and biases of 4 consecutive channels from n (clamped to the last one).
__device__ __forceinline__ void load_channels(const I8Params& p, int n, float (&sw)[4], float (&bs)[4]) {
  const bool has_bias = p.bias != nullptr;
  if (p.vec_channels && n + 4 <= p.N) {
    const v4f s = *reinterpret_cast<const v4f*>(p.w_scales + n);
    const v4f b = has_bias ? *reinterpret_cast<const v4f*>(p.bias + n) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sw[e] = s[e];
      bs[e] = b[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = min(n + e, p.N - 1);
      sw[e] = p.w_scales[c * p.inc_ws];
      bs[e] = has_bias ? p.bias[c] : 0.0f;
    }
  }
}

// 4 finished values of row m, columns n .. n + 3 (n + 4 <= N when `four`).
template <bool F32OUT>
__device__ __forceinline__ void store_channels(const I8Params& p, int m, int n, const float (&v)[4], bool four) {
  const int64_t at = (int64_t)m * p.ld_out + n;
  if constexpr (F32OUT) {
    float* o = static_cast<float*>(p.out) + at;
    if (four) {
      *reinterpret_cast<v4f*>(o) = v4f{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) o[e] = v[e];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
    const unsigned lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (four) {
      *reinterpret_cast<v2u*>(o) = v2u{lo, hi};
    } else {
      if (n + 0 < p.N) o[0] = (uint16_t)lo;
      if (n + 1 < p.N) o[1] = (uint16_t)(lo >> 16);
      if (n + 2 < p.N) o[2] = (uint16_t)hi;
      if (n + 3 < p.N) o[3] = (uint16_t)(hi >> 16);
    }
  }
}

template <bool PAST, class V>
__device__ __forceinline__ void store16(V* at, V v) {
  if constexpr (PAST)
    __builtin_nontemporal_store(v, at);
  else
    *at = v;
}

// What a workgroup leaves: finished bf16 or binary32 outputs, or the int32 sums of its part
// of K (blockIdx.y of p.splits) for i8_reduce_kernel.
enum { OUT_BF16 = 0, OUT_F32 = 1, OUT_PART = 2 };

// SHIFT: for operands whose rows do not all start on a cache line (128 bytes).
template <int MI, int MJ, int WM, int WN, int NA, int NW, bool SHIFT = false>
struct Tile {
  static constexpr int WAVES = WM * WN, BM = 16 * MJ * WM, BN = 16 * MI * WN;
  static constexpr uint32_t A_TILE = BM * kWin, W_TILE = BN * kWin, LDS = NA * A_TILE + NW * W_TILE;
};
using Tile256x256 = Tile<4, 8, 2, 4, 3, 2>;
using Tile128x256 = Tile<4, 4, 2, 4, 3, 3>;
using Tile128x128 = Tile<2, 4, 2, 4, 4, 4>;

// The same tile for rows off the cache lines: the rings need a third weight block.
template <class T> struct Shift;
template <int MI, int MJ, int WM, int WN, int NA, int NW>
struct Shift<Tile<MI, MJ, WM, WN, NA, NW>> { using type = Tile<MI, MJ, WM, WN, NW == 3 ? 4 : NA, NW, NW >= 3>; };
template <class T> using Shifted = typename Shift<T>::type;

// One output tile from (m0, n0) by the whole workgroup, with LDS_BYTES of LDS.
template <int OUT, uint32_t LDS_BYTES, int MI, int MJ, int WM, int WN, int NA, int NW, bool SHIFT>
__device__ __forceinline__ void i8_tile(Tile<MI, MJ, WM, WN, NA, NW, SHIFT>, const I8Params& p, uint8_t* lds, int m0, int n0) {
  using T = Tile<MI, MJ, WM, WN, NA, NW, SHIFT>;
  constexpr int WAVES = T::WAVES, BM = T::BM, BN = T::BN;
  constexpr uint32_t A_TILE = T::A_TILE, W_TILE = T::W_TILE;
  constexpr int LA = (int)(A_TILE / 1024) / WAVES, LW = (int)(W_TILE / 1024) / WAVES;   // 1 KB lines per wave
  constexpr int RD = MI + MJ, VM = LA + LW;
  static_assert(LA >= 1 && LW >= 1 && LA * WAVES * 1024 == (int)A_TILE && LW * WAVES * 1024 == (int)W_TILE, "whole lines");
  static_assert(NW >= 2 && (NA == NW || NA == NW + 1) && (!SHIFT || NA + NW >= 7), "ring depths");
  static_assert(T::LDS <= LDS_BYTES, "rings fit");
  // a window's reads reach AHEAD further blocks; the loads issued after the last piece of block
  // w+1+AHEAD when window w ends
  constexpr int AHEAD = SHIFT ? 1 : 0;
  constexpr int IN_FLIGHT = (NW - 2 - AHEAD) * VM + (NA > NW ? LA : 0);
  static_assert((NW - 1) * VM + (NA > NW ? LA : 0) < 64, "vmcnt range");
  constexpr uint32_t W_BASE = NA * A_TILE;

  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
  const uint32_t wm = wave % WM, wn = wave / WM;
  // this workgroup's windows of K
  const int w_lo = OUT == OUT_PART ? (int)((int64_t)blockIdx.y * p.nwin / p.splits) : 0;
  const int w_hi = OUT == OUT_PART ? (int)((int64_t)(blockIdx.y + 1) * p.nwin / p.splits) : p.nwin;
  const int nwin = w_hi - w_lo, K = min(p.K, w_hi * kWin) - w_lo * kWin;
  const uint32_t rows_a = (uint32_t)min(BM, p.M - m0), rows_w = (uint32_t)min(BN, p.N - n0);
  const int8_t* base_a = p.a + (int64_t)m0 * p.ld_a + w_lo * kWin;
  const int8_t* base_w = p.w + (int64_t)n0 * p.ld_w + w_lo * kWin;
  // SHIFT: the resources start at the cache line of their first row
  const uint32_t off_a = SHIFT ? (uint32_t)(uintptr_t)base_a & 127u : 0u, off_w = SHIFT ? (uint32_t)(uintptr_t)base_w & 127u : 0u;
  base_a -= off_a;
  base_w -= off_w;
  const uint32_t bytes_a = off_a + (rows_a - 1) * p.ld_a + (uint32_t)K, bytes_w = off_w + (rows_w - 1) * p.ld_w + (uint32_t)K;

  // direct-to-LDS lines: LDS line q holds rows 8q .. 8q+7; lane i lands at byte 16 i, in
  // row i / 8 at slot i % 8, and fetches the chunk the swizzle maps there (whose term
  // (r >> 1) & 7 depends on the line's parity)
  const uint32_t drow = lane >> 3, dslot = lane & 7;
  const uint32_t chunk0 = (dslot ^ ((drow >> 1) & 7u)) * 16, chunk1 = (dslot ^ (((8u + drow) >> 1) & 7u)) * 16;
  const uint32_t last_bytes = (uint32_t)(K - (nwin - 1) * kWin);   // of the last window: 16 .. 128
  // line j of this wave's share of window w, into ring slot `slot`; past the last window the
  // resource is empty, so that no memory is read and the loads in flight stay what the waits assume
  // SHIFT: block w of a row is its cache line w, which starts `ph` bytes before window w; ph is
  // the same every 8 rows, since pitches are multiples of 16
  const uint32_t ph_a = (off_a + (SHIFT ? drow * p.ld_a : 0u)) & 127u, ph_w = (off_w + (SHIFT ? drow * p.ld_w : 0u)) & 127u;
  // its chunks lie as those of window w would, so that the fragment reads stay free of conflicts:
  // ka, kw: the K (from that of the block's window) that a lane fetches, negative before the window
  auto in_line = [](uint32_t chunk, uint32_t ph) { return SHIFT ? ((chunk + ph) & 127u) - ph : chunk; };
  const uint32_t ka0 = in_line(chunk0, ph_a), ka1 = in_line(chunk1, ph_a), kw0 = in_line(chunk0, ph_w), kw1 = in_line(chunk1, ph_w);
  const uint32_t row_a = drow * p.ld_a + off_a, row_w = drow * p.ld_w + off_w;
  const uint32_t va0 = row_a + ka0, va1 = row_a + ka1, vw0 = row_w + kw0, vw1 = row_w + kw1;
  const bool in0 = chunk0 < last_bytes, in1 = chunk1 < last_bytes;   // of the last window
  auto issue_a = [&](int w, uint32_t slot, int j) {
    const uint32_t line = wave * LA + j;
    const bool odd = LA % 2 == 0 ? j & 1 : line & 1;
    const bool in = SHIFT ? (uint32_t)w * kWin + (odd ? ka1 : ka0) < (uint32_t)K
                          : w + 1 < nwin || (odd ? in1 : in0);
    line_to_lds(make_rsrc(base_a, SHIFT || w < nwin ? bytes_a : 0u), lds + slot * A_TILE + line * 1024,
                in ? (odd ? va1 : va0) : kOutside, (uint32_t)w * kWin + line * 8 * p.ld_a);
  };
  auto issue_w = [&](int w, uint32_t slot, int j) {
    const uint32_t line = wave * LW + j;
    const bool odd = LW % 2 == 0 ? j & 1 : line & 1;
    const bool in = !SHIFT || (uint32_t)w * kWin + (odd ? kw1 : kw0) < (uint32_t)K;
    line_to_lds(make_rsrc(base_w, SHIFT || w < nwin ? bytes_w : 0u), lds + W_BASE + slot * W_TILE + line * 1024,
                in ? (odd ? vw1 : vw0) : kOutside, (uint32_t)w * kWin + line * 8 * p.ld_w);
  };

  v4i acc[MI][MJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  v4i f0[RD], f1[RD];
  const uint32_t r16 = lane & 15, g = lane >> 4;
  // step-t fragments of the window in ring slots u mod NA, u mod NW: weight rows, then
  // activation rows; after(k) follows read k.  A lane reads chunk g + 4t of rows r16 + 16 i,
  // whose swizzle is that of r16: one offset for t = 0, and the same with bit 6 turned for t = 1
  const uint32_t frag = lds_slot(r16, g);
  // SHIFT: the chunks of a row are counted from its block, and those past 7 are in the next
  const uint32_t ca = g + (((off_a + r16 * p.ld_a) & 127u) >> 4), cw = g + (((off_w + r16 * p.ld_w) & 127u) >> 4);
  auto read = [&](v4i(&f)[RD], uint32_t u, int t, auto&& after) {
    const uint32_t at = frag ^ (64u * t);
    const uint32_t ua = SHIFT && ca + 4 * t > 7 ? (u + 1) % NA : u % NA, uw = SHIFT && cw + 4 * t > 7 ? (u + 1) % NW : u % NW;
    const uint8_t* la = lds + (at + wm * (16 * MJ * 128) + ua * A_TILE);
    const uint8_t* lw = lds + (at + wn * (16 * MI * 128) + W_BASE + uw * W_TILE);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      f[i] = *reinterpret_cast<const v4i*>(lw + 2048 * i);
      after(i);
    }
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      f[MI + j] = *reinterpret_cast<const v4i*>(la + 2048 * j);
      after(MI + j);
    }
  };
  auto step = [&](const v4i(&f)[RD]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int jj = 0; jj < MJ; ++jj) {
        // back and forth along the activations, so that one operand stays from each product to
        // the next (0.6 % on the largest tile, whose clock the toggling operand bits hold down)
        const int j = i & 1 ? MJ - 1 - jj : jj;
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[i], f[MI + j], acc[i][j], 0, 0, 0);
      }
  };
  // Window w, in ring position U: step 0 under the reads of step 1; the hand-over waits for
  // window w+1 and releases this window's slots; step 1 under the reads of window w+1's
  // step 0 and the loads that refill those slots.
  auto window = [&](int w, auto u_tag) {
    constexpr uint32_t U = decltype(u_tag)::value;
    read(f1, U, 1, [](int) {});
    step(f0);
    region_units<0, RD, MI * MJ, 0>(std::make_integer_sequence<int, RD>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_vm(IN_FLIGHT));
    handover_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(f0, U + 1, 0, [&](int k) {
#pragma unroll
      for (int l = 0; l < VM; ++l)
        if (l >= k * VM / RD && l < (k + 1) * VM / RD) {
          if (l < LW)
            issue_w(w + NW, (U + NW) % NW, l);
          else
            issue_a(w + NA, (U + NA) % NA, l - LW);
        }
    });
    step(f1);
    region_units<1, RD, MI * MJ, VM>(std::make_integer_sequence<int, RD>{});
    __builtin_amdgcn_sched_barrier(0);
  };
  // The loop runs once round both rings without a branch back: the ring slots are then
  // constants and the compiler's waits count exactly the reads that a product needs
  // (2.5 % to 4 % faster than one window per turn on the largest tile).
  constexpr int TURN = NA == NW ? NA : NA * NW;
  auto turn = [&](int w) {
    return each<TURN>([&](auto u_tag) {
      if (w + decltype(u_tag)::value >= nwin) return false;
      window(w + decltype(u_tag)::value, u_tag);
      return true;
    });
  };

  if (nwin > 0) {
    // prologue, in the order of the steady state: the weight tile of a window, then the
    // activation tile NA - NW windows further on
    if constexpr (NA > NW)
#pragma unroll
      for (int j = 0; j < LA; ++j) issue_a(0, 0, j);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
#pragma unroll
      for (int j = 0; j < LW; ++j) issue_w(w, w, j);
#pragma unroll
      for (int j = 0; j < LA; ++j) issue_a(w + NA - NW, w + NA - NW, j);
    }
    __builtin_amdgcn_s_waitcnt(wait_vm((NW - 1 - AHEAD) * VM + (NA > NW ? LA : 0)));   // window 0 landed
    handover_barrier();
    read(f0, 0, 0, [](int) {});
    for (int w = 0; turn(w); w += TURN) {
    }
    __builtin_amdgcn_s_waitcnt(0);   // nothing may land in LDS after this workgroup has ended
  }

  // ---- epilogue: lane l holds columns 4g .. 4g+3 of row l & 15 of every block ----
  const int mw = m0 + (int)wm * (16 * MJ), nw = n0 + (int)wn * (16 * MI);
  if constexpr (OUT == OUT_PART) {
    int* part = p.part + (int64_t)blockIdx.y * p.M * p.ld_part;
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const int m = mw + (int)(16 * j + r16);
      if (m >= p.M) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int n = nw + 16 * i + 4 * (int)g;
        if (n < p.N) *reinterpret_cast<v4i*>(part + (int64_t)m * p.ld_part + n) = acc[i][j];
      }
    }
    return;
  }
  // one branch around all the stores, so that the reads before them go out together
  auto store_rows = [&](auto&& rows) {
    if (p.past)
      rows(std::true_type{});
    else
      rows(std::false_type{});
  };
  const bool has_bias = p.bias != nullptr;
  float sw[MI][4], bs[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i) load_channels(p, nw + 16 * i + 4 * (int)g, sw[i], bs[i]);
  constexpr uint32_t CPR = 2 * MI, RB = 32 * MI;   // 16-byte chunks, bytes per bf16 row of the wave's sub-tile
  constexpr uint32_t RPI = 64 / CPR;               // rows per store instruction
  if constexpr (OUT == OUT_BF16 && 16 * MJ >= RPI) {
    if (p.vec && n0 + BN <= p.N) {
      // park the wave's sub-tile in LDS (chunk c of row r at c ^ (r & (CPR - 1))) and store
      // whole row segments
      static_assert((CPR & (CPR - 1)) == 0 && CPR <= 64, "a power of two");
      static_assert(WAVES * 16 * MJ * RB <= LDS_BYTES, "staging fits the rings");
      __syncthreads();
      uint8_t* sub = lds + wave * (16 * MJ * RB);
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        const uint32_t row = 16 * j + r16;
        const float sa = p.a_scales[min(mw + (int)row, p.M - 1) * p.inc_as];
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
      uint16_t* obase = static_cast<uint16_t*>(p.out) + (int64_t)mw * p.ld_out + nw;
      store_rows([&](auto past) {
#pragma unroll
        for (uint32_t q = 0; q < 16 * MJ / RPI; ++q) {
          const uint32_t row = RPI * q + lane / CPR, c = lane % CPR;
          const v4i v = *reinterpret_cast<const v4i*>(sub + row * RB + ((c ^ (row & (CPR - 1))) << 4));
          if (mw + (int)row < p.M) store16<decltype(past)::value>(reinterpret_cast<v4i*>(obase + (int64_t)row * p.ld_out + c * 8), v);
        }
      });
      return;
    }
  }
  // binary32 outputs, and rows that are not 16-byte aligned or end inside the tile: the same
  // through a binary32 image of CJ blocks of rows, stored in the order of the rows
  // (1001 x 1360 x 2051 to binary32 took 2.4 us longer with each lane storing its own columns)
  constexpr int PITCH = 16 * MI + 4;               // floats per row in LDS
  constexpr int FIT = (int)(LDS_BYTES / (WAVES * 16 * PITCH * 4));
  constexpr int CJ = FIT >= MJ ? MJ : FIT >= 4 ? 4 : FIT >= 2 ? 2 : 1;
  static_assert(FIT >= 1 && MJ % CJ == 0, "whole passes");
  __syncthreads();
  float* sub = reinterpret_cast<float*>(lds) + wave * (CJ * 16 * PITCH);
  const bool whole = OUT == OUT_F32 && p.vec && n0 + BN <= p.N;
#pragma unroll
  for (int jb = 0; jb < MJ; jb += CJ) {
#pragma unroll
    for (int j = 0; j < CJ; ++j) {
      const float sa = p.a_scales[min(mw + 16 * (jb + j) + (int)r16, p.M - 1) * p.inc_as];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][jb + j][e], sa, sw[i][e], bs[i][e], has_bias);
        *reinterpret_cast<v4f*>(sub + (16 * j + r16) * PITCH + 16 * i + 4 * g) = v4f{v[0], v[1], v[2], v[3]};
      }
    }
    const int mb = mw + 16 * jb;
    if (whole) {
      constexpr int LPR = 4 * MI;                  // lanes per row, 4 columns each
      store_rows([&](auto past) {
#pragma unroll
        for (int q = 0; q < 16 * CJ * LPR / 64; ++q) {
          const int row = (int)(64 * q + lane) / LPR, col = (int)(64 * q + lane) % LPR * 4;
          const v4f v = *reinterpret_cast<const v4f*>(sub + row * PITCH + col);
          if (mb + row < p.M)
            store16<decltype(past)::value>(reinterpret_cast<v4f*>(static_cast<float*>(p.out) + (int64_t)(mb + row) * p.ld_out + nw + col), v);
        }
      });
    } else if (n0 + BN <= p.N) {
      // 16 bytes from the first 16-byte boundary of each row on, then the E elements that are left
      // over at its two ends (9000 x 512 x 9001: 86 us; with single elements 103, with pairs 120)
      using Elem = std::conditional_t<OUT == OUT_F32, float, uint16_t>;
      constexpr int W = 16 * MI, E = 16 / (int)sizeof(Elem), GROUPS = 16 * CJ * W / E, REST = 16 * CJ * E;
      auto row_at = [&](int row) { return static_cast<Elem*>(p.out) + (int64_t)(mb + row) * p.ld_out + nw; };
      auto to_boundary = [&](const Elem* o) { return (int)(-(reinterpret_cast<uintptr_t>(o) / sizeof(Elem)) & (E - 1)); };
#pragma unroll 4
      for (int q = 0; q < (GROUPS + 63) / 64; ++q) {
        const int at = 64 * q + (int)lane, row = at / (W / E);
        Elem* o = row_at(row);
        const int col = at % (W / E) * E + to_boundary(o);
        if (at < GROUPS && mb + row < p.M && col + E <= W) {
          const float* v = sub + row * PITCH + col;
          if constexpr (OUT == OUT_F32)
            *reinterpret_cast<v4f*>(o + col) = v4f{v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<v4u*>(o + col) =
                v4u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        }
      }
#pragma unroll 4
      for (int q = 0; q < (REST + 63) / 64; ++q) {
        const int at = 64 * q + (int)lane, row = at / E, e = at % E;
        Elem* o = row_at(row);
        const int head = to_boundary(o), col = e < head ? e : W - E + e;
        if (at < REST && mb + row < p.M && head > 0) {
          const float v = sub[row * PITCH + col];
          if constexpr (OUT == OUT_F32)
            o[col] = v;
          else
            o[col] = (uint16_t)pack_bf16x2(v, 0.0f);
        }
      }
    } else {
#pragma unroll 4
      for (int q = 0; q < 16 * CJ * 16 * MI / 64; ++q) {
        const int row = (int)(64 * q + lane) / (16 * MI), col = (int)(64 * q + lane) % (16 * MI);
        const float v = sub[row * PITCH + col];
        if (mb + row < p.M && nw + col < p.N) {
          const int64_t at = (int64_t)(mb + row) * p.ld_out + nw + col;
          if constexpr (OUT == OUT_F32)
            static_cast<float*>(p.out)[at] = v;
          else
            static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack_bf16x2(v, 0.0f);
        }
      }
    }
  }
}

// Plain tiles, blockIdx.y the part of K.
template <class T, int OUT>
__global__ __launch_bounds__(64 * T::WAVES) void gemm_i8_kernel(I8Params p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  int tm, tn;
  tile_at(p, xcd_run(blockIdx.x, p.tiles_m * p.tiles_n), tm, tn);
  i8_tile<OUT, T::LDS>(T{}, p, lds, tm * T::BM, tn * T::BN);
}

// 256 x 256 tiles in whole rounds of the GPU (the first p.whole workgroups), and the tiles of
// the last, partial round cut into PARTS smaller ones of type S, so that it keeps more of
// the CUs busy.  Against whole tiles to the end: 3584 x 5120 x 5120 (280 tiles, 24 in the last
// round, quarters) 110 -> 86 us, 4096 x 5120 x 5120 118 -> 91, 5000 x 2048 x 4096 58 -> 49,
// 3584 x 5120 x 15360 238 -> 229; a last round of more than 128 tiles gains nothing.
template <class S, int OUT>
__global__ __launch_bounds__(512) void gemm_i8_tail_kernel(I8Params p) {
  using T = Tile256x256;
  constexpr int DOWN = T::BM / S::BM, PARTS = DOWN * (T::BN / S::BN);
  static_assert(S::WAVES == T::WAVES, "one workgroup size");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int bid = blockIdx.x;
  int tm, tn;
  if (bid < p.whole) {
    tile_at(p, xcd_run(bid, p.whole), tm, tn);
    i8_tile<OUT, T::LDS>(T{}, p, lds, tm * T::BM, tn * T::BN);
  } else {
    const int part = (bid - p.whole) % PARTS;
    tile_at(p, p.whole + (bid - p.whole) / PARTS, tm, tn);
    const int m0 = tm * T::BM + part % DOWN * S::BM, n0 = tn * T::BN + part / DOWN * S::BN;
    if (m0 < p.M && n0 < p.N) i8_tile<OUT, T::LDS>(S{}, p, lds, m0, n0);
  }
}

// Sums of the parts of K (p.splits of them), then the epilogue: one thread, 4 columns.
template <bool F32OUT>
__global__ __launch_bounds__(256) void i8_reduce_kernel(I8Params p) {
  const uint32_t quads = (uint32_t)p.ld_part / 4;
  const int64_t total = (int64_t)p.M * quads, plane = (int64_t)p.M * p.ld_part;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int m = (int)(e / quads), n = (int)(e % quads) * 4;
    const int* src = p.part + (int64_t)m * p.ld_part + n;
    // all loads at once (250 x 13824 x 272: 11.3 us, one after another 12.5)
    v4i part[kMaxSplits];
#pragma unroll
    for (int z = 0; z < kMaxSplits; ++z) {
      part[z] = v4i{0, 0, 0, 0};
      if (z < p.splits) part[z] = *reinterpret_cast<const v4i*>(src + z * plane);
    }
    const bool has_bias = p.bias != nullptr;
    const float sa = p.a_scales[m * p.inc_as];
    float sw[4], bs[4], v[4];
    load_channels(p, n, sw, bs);
    v4i s = part[0];
#pragma unroll
    for (int z = 1; z < kMaxSplits; ++z) s += part[z];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = scaled(s[i], sa, sw[i], bs[i], has_bias);
    store_channels<F32OUT>(p, m, n, v, p.vec && n + 4 <= p.N);
  }
}

// ---------------------------------------------------------------------------------
// Up to 8 tokens: the weights' bytes are what counts.  One workgroup = 16 NI channels, its
// WAVES waves splitting K (window w to wave w mod WAVES).  Each wave streams its windows
// through a ring of D slots of its own in LDS, so nothing is synchronized until the partial
// sums meet (integers: the order changes nothing).  The workgroups start at windows spread
// over K: started together, they would read the same columns of all rows at once, which a
// row pitch of a power of two maps to a few memory channels (1 x 8192 x 4096: 12.0 -> 9.0 us).
// Bound by the weights' bytes: 1 x 5120 x 13824 takes 15.0 us, 4.7 TB/s, with the next call's launch behind
// it (12.1 us where the memory-side cache holds the weights); with the activations made here 1 x 13824 x 5120
// takes 16.6 us, two launches 18.5 (13.5 and 15.7).  For 9 to 64 tokens such a kernel with 2 to 8 lines of
// activations is no faster than the tiles (weights not in a cache, side by side: 16 x 5120 x 5120 8.9 and 9.0
// us, 48 x 13824 x 5120 24 and 21).
//
// A_BF16, A_F32: the activations come unquantized, and every workgroup makes the codes of
// all tokens itself, into LDS, while its first weight windows are on their way: at a few KB
// that costs less than a launch of its own.
enum { A_CODES = 0, A_BF16 = 1, A_F32 = 2 };
constexpr uint32_t kFewCodes = 15872;              // bytes of codes that a workgroup holds: two fit a CU

__device__ __host__ constexpr uint32_t few_pitch(int nwin) { return (uint32_t)nwin * kWin + 16u; }

template <int NI, int WAVES, int D, int A, bool F32OUT>
__global__ __launch_bounds__(64 * WAVES) void gemm_i8_few_kernel(I8Params p) {
  constexpr int LINES = 2 * NI + (A == A_CODES ? 1 : 0);   // 1 KB lines of 8 rows: weights, then activations
  constexpr uint32_t SLOT = LINES * 1024;
  constexpr int T = 64 * WAVES;
  static_assert((D - 1) * LINES < 64, "vmcnt range");
  // one array for everything: with several, the compiler orders every read of LDS behind all
  // loads into it
  constexpr uint32_t RING = WAVES * D * SLOT, CODES = A == A_CODES ? 0 : kFewCodes;
  constexpr uint32_t SMALL = A == A_CODES ? 0 : 4 * kFewTokens * (3 + WAVES);
  static_assert(RING + CODES + SMALL <= 81920, "two workgroups on a CU");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[RING + CODES + SMALL];
  const uint32_t tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(tid >> 6));
  const int n0 = (int)blockIdx.x * (16 * NI);
  const uint32_t rows_w = (uint32_t)min(16 * NI, p.N - n0);
  const uint32_t bytes_a = (uint32_t)(p.M - 1) * p.ld_a + (uint32_t)p.K, bytes_w = (rows_w - 1) * p.ld_w + (uint32_t)p.K;
  const int8_t* base_w = p.w + (int64_t)n0 * p.ld_w;
  const int nwin = p.nwin, start = (int)((int64_t)blockIdx.x * nwin / gridDim.x);
  const uint32_t last_bytes = (uint32_t)(p.K - (nwin - 1) * kWin);
  const uint32_t drow = lane >> 3, dslot = lane & 7;   // as in i8_tile
  const uint32_t chunk0 = (dslot ^ ((drow >> 1) & 7u)) * 16, chunk1 = (dslot ^ (((8u + drow) >> 1) & 7u)) * 16;
  uint8_t* ring = lds + (uint32_t)wave * (D * SLOT);
  auto window = [&](int w) { return w + start >= nwin ? w + start - nwin : w + start; };
  auto issue = [&](int w, uint32_t slot) {
    const int k = window(w);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(base_w, w < nwin ? bytes_w : 0u);
#pragma unroll
    for (int j = 0; j < 2 * NI; ++j)
      line_to_lds(rw, ring + slot * SLOT + j * 1024, drow * p.ld_w + ((j & 1) ? chunk1 : chunk0),
                  (uint32_t)k * kWin + j * 8 * p.ld_w);
    if constexpr (A == A_CODES) {
      const uint32_t valid = k + 1 < nwin ? (uint32_t)kWin : last_bytes;
      line_to_lds(make_rsrc(p.a, w < nwin ? bytes_a : 0u), ring + slot * SLOT + 2 * NI * 1024,
                  chunk0 < valid ? drow * p.ld_a + chunk0 : kOutside, (uint32_t)k * kWin);
    }
  };

  // the codes of all tokens, rows few_pitch apart, and their scales
  uint8_t* codes = lds + RING;
  float* scales = reinterpret_cast<float*>(codes + CODES);
  float* invs = scales + kFewTokens;
  unsigned* keeps = reinterpret_cast<unsigned*>(invs + kFewTokens);
  unsigned* red = keeps + kFewTokens;                      // [kFewTokens][WAVES]
  const uint32_t pitch = few_pitch(nwin);
  if constexpr (A != A_CODES) {
    constexpr bool F32 = A == A_F32;
    constexpr int C = (int)(kFewCodes / 8 + T - 1) / T;     // units of 8 elements per thread
    const uint32_t upr = (uint32_t)p.K / 8, total = upr * (uint32_t)p.M;
    Unit<F32> u[C];
    uint32_t row[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      row[c] = 0;
      for (int m = 1; m < p.M; ++m) row[c] += i >= (uint32_t)m * upr ? 1u : 0u;
      u[c] = i < total ? load_unit<F32, false>(p.x, (int64_t)row[c] * p.ld_x + (i - row[c] * upr) * 8) : zero_unit<F32>();
    }
    // the loads above are older than these: they are waited for alone
#pragma unroll
    for (int d = 0; d < D; ++d) issue(wave + d * WAVES, d);
    unsigned most[C];
#pragma unroll
    for (int c = 0; c < C; ++c) most[c] = unit_max<F32>(u[c]);
    for (int m = 0; m < p.M; ++m) {
      unsigned v = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) v = max(v, row[c] == (uint32_t)m ? most[c] : 0u);
      v = wave_max_u32(v);
      if (lane == 0) red[m * WAVES + wave] = v;
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(63));               // the LDS writes; the weights stay in flight
    handover_barrier();
    if (tid < (uint32_t)p.M) {
      unsigned v = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v = max(v, red[tid * WAVES + w]);
      const Int8Scale sc = int8_scale(v);
      scales[tid] = sc.s;
      invs[tid] = sc.inv;
      keeps[tid] = sc.keep;
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(63));
    handover_barrier();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = c * T + tid;
      if (i < total) {
        const Int8Scale sc = {0.0f, invs[row[c]], keeps[row[c]]};
        *reinterpret_cast<v2u*>(codes + row[c] * pitch + (i - row[c] * upr) * 8) = unit_codes<F32>(u[c], sc);
      }
    }
    // zeros from K to the end of the last window
    if (tid < 8u * (uint32_t)p.M) {
      const uint32_t k = (uint32_t)(nwin - 1) * kWin + (tid & 7) * 16;
      if (nwin > 0 && k >= (uint32_t)p.K) *reinterpret_cast<v4i*>(codes + (tid >> 3) * pitch + k) = v4i{0, 0, 0, 0};
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(63));
    handover_barrier();
  } else {
#pragma unroll
    for (int d = 0; d < D; ++d) issue(wave + d * WAVES, d);
  }

  v4i acc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) acc[i] = v4i{0, 0, 0, 0};
  uint32_t slot = 0;
  for (int w = wave; w < nwin; w += WAVES) {
    __builtin_amdgcn_s_waitcnt(wait_vm((D - 1) * LINES));   // window w landed
    asm volatile("" ::: "memory");
    const uint8_t* s = ring + slot * SLOT;
    v4i fw[2][NI], fa[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < NI; ++i) fw[t][i] = *reinterpret_cast<const v4i*>(s + lds_slot(16 * i + r16, g + 4 * t));
      // columns of the product past the tokens are not used: they repeat others
      if constexpr (A == A_CODES)
        fa[t] = *reinterpret_cast<const v4i*>(s + NI * 2048 + lds_slot(r16 & 7, g + 4 * t));
      else
        fa[t] = *reinterpret_cast<const v4i*>(codes + min(r16, (uint32_t)p.M - 1) * pitch + (uint32_t)window(w) * kWin + 64 * t + 16 * g);
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(63));                // the reads are done: the slot can be refilled
    asm volatile("" ::: "memory");
    issue(w + D * WAVES, slot);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[t][i], fa[t], acc[i], 0, 0, 0);
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  v4i* part = reinterpret_cast<v4i*>(lds);
#pragma unroll
  for (int i = 0; i < NI; ++i) part[(wave * NI + i) * 64 + lane] = acc[i];
  __syncthreads();
  // thread e: token e / (4 NI), 4 channels from 4 (e % (4 NI))
  for (uint32_t e = tid; e < 4 * NI * (uint32_t)p.M; e += T) {
    const uint32_t m = e / (4 * NI), q = e % (4 * NI);
    const int n = n0 + 4 * (int)q;
    if (n >= p.N) continue;
    v4i sum = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[(w * NI + (q >> 2)) * 64 + (q & 3) * 16 + m];
    float sw[4], bs[4], v[4];
    load_channels(p, n, sw, bs);
    const float sa = A == A_CODES ? p.a_scales[m * p.inc_as] : scales[m];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = scaled(sum[k], sa, sw[k], bs[k], p.bias != nullptr);
    store_channels<F32OUT>(p, (int)m, n, v, p.vec && n + 4 <= p.N);
  }
}

}  // namespace

size_t gemm_w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= kFewTokens) return 0;
  const int splits = plan_w8a8(M, N, K, true).splits;
  return splits == 1 ? 0 : (size_t)splits * (size_t)M * (size_t)((N + 3) / 4 * 4) * 4;
}

bool gemm_w8a8_one_launch(int64_t M, int64_t K) {
  return M <= kFewTokens && M * (int64_t)few_pitch((int)((K + kWin - 1) / kWin)) <= (int64_t)kFewCodes;
}

namespace {

// What does not depend on the activations.
I8Params i8_params(const int8_t* w, int64_t ld_w, const float* w_scales, int64_t inc_ws, const float* bias, int64_t M,
                   int64_t N, int64_t K, void* out, bool f32_out, int64_t ld_out) {
  I8Params p = {};
  p.w = w;
  p.w_scales = w_scales;
  p.bias = bias;
  p.out = out;
  p.ld_out = ld_out;
  p.inc_ws = inc_ws;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.ld_w = (uint32_t)ld_w;
  p.nwin = (int)((K + kWin - 1) / kWin);
  auto aligned16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  p.vec = (ld_out * (f32_out ? 4 : 2)) % 16 == 0 && aligned16(out);
  // Rows of whole 64-byte pieces are stored past the caches: the output is not read again here, and
  // the operands of the neighbouring tiles stay (75600 x 128 x 4000: 191 us, 215 through the caches);
  // smaller pieces meet their other parts in the L2 (9000 x 512 x 9000: 107 us past the caches, 73).
  p.past = (ld_out * (f32_out ? 4 : 2)) % 64 == 0 && reinterpret_cast<uintptr_t>(out) % 64 == 0;
  p.vec_channels = inc_ws == 1 && aligned16(w_scales) && aligned16(bias);
  p.splits = 1;
  return p;
}

template <int A>
void launch_few(const I8Params& p, bool f32_out, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)p.N + 31) / 32)), block(256);
  if (f32_out)
    hipLaunchKernelGGL((gemm_i8_few_kernel<2, 4, 4, A, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((gemm_i8_few_kernel<2, 4, 4, A, false>), grid, block, 0, stream, p);
}

}  // namespace

hipError_t launch_gemm_w8a8_unquantized(const void* x, bool f32, int64_t ld_x, const int8_t* w, int64_t ld_w,
                                        const float* w_scales, int64_t inc_ws, const float* bias, int64_t M, int64_t N,
                                        int64_t K, void* out, bool f32_out, int64_t ld_out, hipStream_t stream) {
  I8Params p = i8_params(w, ld_w, w_scales, inc_ws, bias, M, N, K, out, f32_out, ld_out);
  p.x = x;
  p.ld_x = ld_x;
  f32 ? launch_few<A_F32>(p, f32_out, stream) : launch_few<A_BF16>(p, f32_out, stream);
  return hipGetLastError();
}

hipError_t launch_gemm_w8a8(const int8_t* a, int64_t ld_a, const float* a_scales, int64_t inc_as, const int8_t* w,
                            int64_t ld_w, const float* w_scales, int64_t inc_ws, const float* bias, int64_t M,
                            int64_t N, int64_t K, void* out, bool f32_out, int64_t ld_out, void* workspace,
                            hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  I8Params p = i8_params(w, ld_w, w_scales, inc_ws, bias, M, N, K, out, f32_out, ld_out);
  p.a = a;
  p.a_scales = a_scales;
  p.inc_as = inc_as;
  p.ld_a = (uint32_t)ld_a;
  p.part = static_cast<int*>(workspace);
  p.ld_part = (int)((N + 3) / 4 * 4);
  if (M <= kFewTokens) {
    launch_few<A_CODES>(p, f32_out, stream);
    return hipGetLastError();
  }
  const Plan plan = plan_w8a8(M, N, K, workspace != nullptr);
  p.splits = plan.splits;
  const bool shift = shifted(K, (uintptr_t)a, ld_a, (uintptr_t)w, ld_w);
  auto tile = [&](auto tile_tag, auto o_tag) {
    using T = decltype(tile_tag);
    p.tiles_m = (int)((M + T::BM - 1) / T::BM);
    p.tiles_n = (int)((N + T::BN - 1) / T::BN);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(p.tiles_m * p.tiles_n), (unsigned)p.splits), dim3(64 * T::WAVES), 0, stream, p);
    };
    if (shift)
      go(gemm_i8_kernel<Shifted<T>, decltype(o_tag)::value>);
    else
      go(gemm_i8_kernel<T, decltype(o_tag)::value>);
  };
  auto with_tail = [&](auto small_tag, auto o_tag) {
    using T = Tile256x256;
    using S = decltype(small_tag);
    p.tiles_m = (int)((M + T::BM - 1) / T::BM);
    p.tiles_n = (int)((N + T::BN - 1) / T::BN);
    const int tiles = p.tiles_m * p.tiles_n, parts = (T::BM / S::BM) * (T::BN / S::BN);
    p.whole = tiles / 256 * 256;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(p.whole + (tiles - p.whole) * parts)), dim3(64 * T::WAVES), 0, stream, p);
    };
    if (shift)
      go(gemm_i8_tail_kernel<Shifted<S>, decltype(o_tag)::value>);
    else
      go(gemm_i8_tail_kernel<S, decltype(o_tag)::value>);
  };
  auto pick = [&](auto o_tag) {
    if constexpr (decltype(o_tag)::value != OUT_PART) {
      if (plan.tail == TILE_128x256) return with_tail(Tile128x256{}, o_tag);
      if (plan.tail == TILE_128x128) return with_tail(Tile128x128{}, o_tag);
    }
    switch (plan.tile) {
      case TILE_256x256: return tile(Tile256x256{}, o_tag);
      case TILE_128x256: return tile(Tile128x256{}, o_tag);
      case TILE_128x128: return tile(Tile128x128{}, o_tag);
      case TILE_64x128: return tile(Tile<2, 2, 2, 4, 6, 6>{}, o_tag);
      case TILE_128x64: return tile(Tile<2, 4, 2, 2, 6, 6>{}, o_tag);
      case TILE_64x64: return tile(Tile<2, 2, 2, 2, 4, 4>{}, o_tag);
      case TILE_64x32: return tile(Tile<1, 2, 2, 2, 6, 6>{}, o_tag);
      case TILE_32x64: return tile(Tile<2, 1, 2, 2, 6, 6>{}, o_tag);
      case TILE_32x32: return tile(Tile<1, 1, 2, 2, 8, 8>{}, o_tag);
      default: return tile(Tile<2, 4, 2, 4, 2, 2>{}, o_tag);
    }
  };
  if (p.splits > 1) {
    pick(std::integral_constant<int, OUT_PART>{});
    const int64_t blocks = (M * (p.ld_part / 4) + 255) / 256;
    auto reduce = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, p);
    };
    f32_out ? reduce(i8_reduce_kernel<true>) : reduce(i8_reduce_kernel<false>);
  } else if (f32_out) {
    pick(std::integral_constant<int, OUT_F32>{});
  } else {
    pick(std::integral_constant<int, OUT_BF16>{});
  }
  return hipGetLastError();
}

}  // namespace mxq
