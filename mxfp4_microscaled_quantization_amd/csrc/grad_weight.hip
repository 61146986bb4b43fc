// Weight gradient of the 8-bit product from the codes that its forward pass took:
//   dW[n,k] = sum_m dy[m,n] * bf16(code[m,k] * scale[m])
// with dy in bf16 and the sum in binary32.  The rounding of code * scale to bf16 (relative
// error 2^-9 at most, beside the half step of the codes themselves) is the one of
// mxq_dequantize_int8: the matrix cores take it as an operand, and the products are exact.
//
// The largest tile takes values that a launch ahead of it has widened into a workspace (its registers are full, and each
// code meets many tiles); the smaller one widens the codes on their way into LDS.  The product contracts over rows of both
// operands, while an MFMA takes 8 consecutive values of the contraction in a lane: fragments
// come from LDS by ds_read_b64_tr_b16, in which 16 lanes read 4 rows of 16 columns and each
// gets the 4 values of one column.
//
// Bound by the matrix cores, whose clock gives way first: 75600 tokens, 13824 x 5120 to binary32 8.25 ms, 1.30 PFLOP/s (9.0 on
// another card), the product itself 7.95 with the matrix cores 75 % busy at 1.6 GHz (a library product of this layout on bf16
// operands that are there already: 10.5 ms; a square one of 8192 reaches 1.37 PFLOP/s with rows along the contraction).
#include <type_traits>
#include <utility>

#include "mxq_device.hpp"
#include "mxq_internal.hpp"

namespace mxq {
namespace {

constexpr int kWinRows = 64;   // rows of both operands in LDS at once: two MFMA steps

struct GradParams {
  const uint16_t* dy;
  const uint16_t* x;        // the codes' values, or (CODES)
  const int8_t* codes;      // the codes themselves
  const float* scales;
  int64_t ld_codes;
  void* out;
  float* part;              // sums of the parts of M, [tile - whole][splits][rows of a tile][columns]
  int64_t ld_dy, ld_x, ld_out;
  int M, N, K;
  int nwin, tiles_n, tiles_k;
  int whole, splits;        // tiles whose workgroup takes all of M; parts of M for each of the others
  int accumulate, vec;      // vec: rows of the output are aligned for whole stores of 4
};

// MI x MJ fragments of 16 x 16 outputs (k, n) in a wave, WK x WN waves; rings of NX windows of x and NY of dy.
template <int MI_, int MJ_, int WK_, int WN_, int NY_>
struct GradTile {
  static constexpr int MI = MI_, MJ = MJ_, WK = WK_, WN = WN_, NX = 2, NY = NY_;
  static constexpr int THREADS = 64 * WK * WN, BK = 16 * MI * WK, BN = 16 * MJ * WN;
  static constexpr uint32_t X_TILE = kWinRows * BK * 2, Y_TILE = kWinRows * BN * 2;
};

__device__ __forceinline__ void grad_line_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds_line, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_line, 16, voff, soff, 0, 0);
}

// __restrict__ tells the compiler that no load into LDS in flight is what this reads: without it, it waits for all of
// them before the read (the hand-overs wait for what has to have landed).
typedef short v4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v2u read_transposed(__attribute__((address_space(3))) v4s* __restrict__ lds) {
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds));
}

// Tile `seq`: bands of kGradBand tiles along K, in which the index runs along K first, so that the tiles an XCD runs at once
// share their panels in its L2.
constexpr int kGradBand = 4;
__device__ __forceinline__ void grad_tile_at(const GradParams& p, int seq, int& tk, int& tn) {
  const int band = seq / (kGradBand * p.tiles_n), first = band * kGradBand, rows = min(kGradBand, p.tiles_k - first);
  const int in = seq - band * kGradBand * p.tiles_n;
  tk = first + in % rows;
  tn = in / rows;
}
// Workgroups are dealt to the XCDs in turn: a contiguous run of n indexes for each.
__device__ __forceinline__ int grad_xcd_run(int bid, int n) {
  const int xcd = bid & 7, q8 = n >> 3, r8 = n & 7;
  return xcd * q8 + min(xcd, r8) + (bid >> 3);
}

// 4 sums of columns k .. k + 3 of row n; K is a multiple of 16, so that all are there.
template <bool F32OUT>
__device__ __forceinline__ void store_sums(const GradParams& p, int n, int k, v4f v) {
  if constexpr (F32OUT) {
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

// s_waitcnt immediate (gfx9 encoding): vmcnt <= vm, lgkmcnt <= 0, expcnt unconstrained
constexpr int grad_wait_vm(int vm) { return (vm & 0xF) | ((vm >> 4) << 14) | (0x7 << 4); }

// which of n loads spread over rd reads go out right after read k
constexpr int grad_loads_after(int k, int n, int rd) { return (k + 1) * n / rd - k * n / rd; }

// f(0) && f(1) && ... && f(N - 1), the arguments as integral constants.
template <class F, int... Is>
__device__ __forceinline__ bool each_window_of(F&& f, std::integer_sequence<int, Is...>) {
  return (f(std::integral_constant<int, Is>{}) && ...);
}
template <int N, class F>
__device__ __forceinline__ bool each_window(F&& f) {
  return each_window_of(f, std::make_integer_sequence<int, N>{});
}

// Scheduling pattern of one MFMA region: unit I is the two reads of a fragment, then the tile loads
// that fall there, then its share of the region's MFMAs.
template <int ID, int R, int MFMAS, int VM, int I>
__device__ __forceinline__ void grad_region_unit() {
  __builtin_amdgcn_sched_group_barrier(0x100, 2, ID);                                    // DS read
  constexpr int l = grad_loads_after(I, VM, R);
  if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(0x020, l, ID);               // VMEM read
  constexpr int n = (I + 1) * MFMAS / R - I * MFMAS / R;
  if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x008, n, ID);               // MFMA
}
template <int ID, int R, int MFMAS, int VM, int... Is>
__device__ __forceinline__ void grad_region(std::integer_sequence<int, Is...>) {
  (grad_region_unit<ID, R, MFMAS, VM, Is>(), ...);
}

// CODES: the codes are loaded and widened into the ring by the kernel itself.
template <bool F32OUT, bool CODES, class T>
__global__ __launch_bounds__(T::THREADS, 2) void grad_weight_kernel(GradParams p) {
  constexpr int MI = T::MI, MJ = T::MJ, WK = T::WK, WN = T::WN, WAVES = WK * WN, NX = T::NX, NY = T::NY;
  constexpr int D = CODES ? NY - 1 : 1;   // windows of codes in registers, on their way
  constexpr int LX = (int)(T::X_TILE / 1024) / WAVES, LY = (int)(T::Y_TILE / 1024) / WAVES;   // 1 KB lines per wave
  constexpr int RD = MI + MJ, DX = CODES ? 0 : LX, VM = DX + LY;   // loads into LDS for each window
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NX * T::X_TILE + NY * T::Y_TILE];
  constexpr uint32_t Y_BASE = NX * T::X_TILE;

  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
  const uint32_t wk = wave % WK, wn = wave / WK;
  // this workgroup's tile, and its windows of M: all, or one of the parts (part by part, so that
  // what runs at once shares its rows)
  int seq, part = -1, w_lo = 0, w_hi = p.nwin;
  if ((int)blockIdx.x < p.whole) {
    seq = grad_xcd_run(blockIdx.x, p.whole);
  } else {
    const int rest = p.tiles_n * p.tiles_k - p.whole, i = grad_xcd_run((int)blockIdx.x - p.whole, rest * p.splits);
    part = i / rest;
    seq = p.whole + i - part * rest;
    w_lo = (int)((int64_t)part * p.nwin / p.splits);
    w_hi = (int)((int64_t)(part + 1) * p.nwin / p.splits);
  }
  int tk, tn;
  grad_tile_at(p, seq, tk, tn);
  // quotients are formed in vector registers: back to scalar ones, for the resources
  auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int k0 = scalar(tk) * T::BK, n0 = scalar(tn) * T::BN;
  w_lo = scalar(w_lo);
  w_hi = scalar(w_hi);

  // A window's rows have a resource of their own (64-bit base, offsets below 2^31), empty past the part's
  // last window, so that the loads in flight stay what the waits assume.  An empty one's size comes out as the
  // unused end of a row, negated.
  const int m_hi = min(p.M, w_hi * kWinRows);
  auto rows_of = [&](const uint16_t* base, int ld, int cols, int col0, int w) {
    const int rows = max(0, min(m_hi - w * kWinRows, kWinRows));
    const int elems = scalar(max(rows * ld - (ld - (cols - col0)), 0));
    return make_rsrc(base + (int64_t)w * kWinRows * ld + col0, (uint32_t)elems * 2u);
  };
  // LDS: rows of BC columns, 32-byte unit u of row r at u ^ (r & 7) (the 8 rows that half a wave
  // reads at one column are then on distinct banks).  Line `line` of a window, by one wave:
  auto fill = [&](__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t ld, uint32_t line, auto bc_tag) {
    constexpr uint32_t BC = decltype(bc_tag)::value, CPR = BC / 8, RPL = 64 / CPR;   // 16-byte chunks per row, rows per line
    const uint32_t row = line * RPL + lane / CPR, slot = lane % CPR;
    grad_line_to_lds(r, to + line * 1024, lane / CPR * ld * 2 + ((slot ^ ((row & 7) << 1)) << 4), line * RPL * ld * 2);
  };
  const int ld_x = (int)p.ld_x, ld_dy = (int)p.ld_dy;
  auto x_rows = [&](int w) { return rows_of(p.x, ld_x, p.K, k0, w); };
  auto y_rows = [&](int w) { return rows_of(p.dy, ld_dy, p.N, n0, w); };
  auto issue_x = [&](__amdgpu_buffer_rsrc_t r, uint32_t slot, int j) {
    fill(r, lds + slot * T::X_TILE, (uint32_t)p.ld_x, wave * LX + j, std::integral_constant<uint32_t, T::BK>{});
  };
  auto issue_y = [&](__amdgpu_buffer_rsrc_t r, uint32_t slot, int j) {
    fill(r, lds + Y_BASE + slot * T::Y_TILE, (uint32_t)p.ld_dy, wave * LY + j, std::integral_constant<uint32_t, T::BN>{});
  };
  // CODES: a thread widens units of 16 codes, of a row and of every ROWS-th one further, into 32 bytes each
  constexpr uint32_t TPR = T::BK / 16, ROWS = 64 * WAVES / TPR;
  constexpr int UPT = kWinRows / ROWS;
  static_assert(!CODES || (UPT * ROWS == kWinRows && ROWS % 8 == 0), "whole rounds, and one swizzle for a thread's rows");
  const uint32_t crow = tid / TPR, cunit = tid % TPR;
  struct Raw {
    v4u c[UPT];
    float s[UPT];
  };
  auto load_codes = [&](int w) {
    const int rows = max(0, min(m_hi - w * kWinRows, kWinRows)), ld = (int)p.ld_codes;
    const int bytes = scalar(max(rows * ld - (ld - (p.K - k0)), 0));
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.codes + (int64_t)w * kWinRows * ld + k0, (uint32_t)bytes);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.scales + (int64_t)w * kWinRows, (uint32_t)scalar(rows) * 4u);
    Raw r;   // rows past the end: zeros
#pragma unroll
    for (int j = 0; j < UPT; ++j) {
      r.c[j] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rc, crow * ld + cunit * 16, j * ROWS * ld, 0));
      r.s[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, crow * 4, j * ROWS * 4, 0));
    }
    return r;
  };
  auto store_codes = [&](const Raw& r, uint32_t slot) {
    uint8_t* to = lds + slot * T::X_TILE + crow * (T::BK * 2) + ((cunit ^ (crow & 7)) << 5);
#pragma unroll
    for (int j = 0; j < UPT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4u o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int pair = (int)(r.c[j][2 * h + (e >> 1)] >> (16 * (e & 1)));
          o[e] = pack_bf16x2((float)(int8_t)pair * r.s[j], (float)(int8_t)(pair >> 8) * r.s[j]);
        }
        *reinterpret_cast<v4u*>(to + j * (ROWS * T::BK * 2) + 16 * h) = o;
      }
  };
  // the fragment of 16 columns from unit u, tokens 32 t + 4 g + (0 .. 3) and 16 more, g = lane / 16
  const uint32_t q = lane & 15, row0 = 4 * (lane >> 4) + (q >> 2);
  const uint32_t at_x = row0 * (T::BK * 2) + ((row0 & 7) << 5) + 8 * (q & 3), at_y = row0 * (T::BN * 2) + ((row0 & 7) << 5) + 8 * (q & 3);
  auto read1 = [&](const uint8_t* tile_at, uint32_t pitch, uint32_t at, uint32_t u, int t) {
    const uint8_t* from = tile_at + (at ^ (u << 5)) + 32 * t * pitch;
    const v2u lo = read_transposed((__attribute__((address_space(3))) v4s*)from);
    const v2u hi = read_transposed((__attribute__((address_space(3))) v4s*)(from + 16 * pitch));
    return v4u{lo[0], lo[1], hi[0], hi[1]};
  };
  auto read = [&](v4u(&f)[RD], uint32_t sx, uint32_t sy, int t, auto&& after) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      f[i] = read1(lds + sx * T::X_TILE, T::BK * 2, at_x, wk * MI + i, t);
      after(i);
    }
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      f[MI + j] = read1(lds + Y_BASE + sy * T::Y_TILE, T::BN * 2, at_y, wn * MJ + j, t);
      after(MI + j);
    }
  };

  v4f acc[MI][MJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto step = [&](const v4u(&f)[RD]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int jj = 0; jj < MJ; ++jj) {
        const int j = i & 1 ? MJ - 1 - jj : jj;
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f[i]),
                                                            __builtin_bit_cast(bf16x8, f[MI + j]), acc[i][j], 0, 0, 0);
      }
  };
  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // prologue: the loads of window w_lo and, in the order of the steady state, of the next windows; then w_lo resident
  v4u f0[RD], f1[RD];
  Raw raw[D];   // CODES: window w's in raw[(w - w_lo) % D]
  if (w_lo < w_hi) {
    Raw first;
    if constexpr (CODES) {
      first = load_codes(w_lo);
    } else {
#pragma unroll
      for (int j = 0; j < LX; ++j) issue_x(x_rows(w_lo), 0, j);
    }
#pragma unroll
    for (int j = 0; j < LY; ++j) issue_y(y_rows(w_lo), 0, j);
    __builtin_amdgcn_sched_barrier(0);   // the waits count on this order
#pragma unroll
    for (int k = 1; k < NY; ++k) {
      if constexpr (CODES) {
        raw[k % D] = load_codes(w_lo + k);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (!CODES && k == NY - 1)
#pragma unroll
        for (int j = 0; j < LX; ++j) issue_x(x_rows(w_lo + 1), 1, j);
#pragma unroll
      for (int j = 0; j < LY; ++j) issue_y(y_rows(w_lo + k), k, j);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (CODES) store_codes(first, 0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(grad_wait_vm((NY - 1) * LY + (CODES ? (NY - 1) * 2 * UPT : LX)));
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(f0, 0, 0, 0, [](int) {});
  }
  // One window: step 0 on f0 under the reads of step 1 into f1; the hand-over waits for window w+1 and releases window w's
  // slots; step 1 on f1 under the reads of window w+1's step 0 and the loads of dy of window w+NY into its slot.
  // x of window w+1: CODES, written ahead of the hand-over into the slot that the last one released, whereupon the codes
  // of window w+NY are loaded; else, loaded into LDS ahead of dy by the window before.
  // In flight behind dy of window w+1 at the hand-over: dy of NY - 2 windows, and the codes of NY - 1.
  constexpr int IN_FLIGHT = (NY - 2) * LY + (CODES ? (NY - 1) * 2 * UPT : 0);
  static_assert(IN_FLIGHT < 64 && (CODES || NY == 3), "what the waits count");
  uint32_t sx = 0, sy = 0;
  auto window = [&](int w, auto i_tag) {
    constexpr int NEXT = (decltype(i_tag)::value + 1) % D;
    const __amdgpu_buffer_rsrc_t rx = x_rows(w + NX), ry = y_rows(w + NY);
    const uint32_t sx1 = sx ^ 1, sy1 = sy == NY - 1 ? 0 : sy + 1;
    read(f1, sx, sy, 1, [](int) {});
    if constexpr (CODES) {
      store_codes(raw[NEXT], sx1);
      raw[NEXT] = load_codes(w + NY);
    }
    step(f0);
    if constexpr (!CODES) grad_region<0, RD, MI * MJ, 0>(std::make_integer_sequence<int, RD>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(grad_wait_vm(IN_FLIGHT));
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(f0, sx1, sy1, 0, [&](int k) {
      if (grad_loads_after(k, VM, RD) > 0) {
        const int j = k * VM / RD;
        if (j < DX)
          issue_x(rx, sx, j);
        else
          issue_y(ry, sy, j - DX);
      }
    });
    step(f1);
    grad_region<1, RD, MI * MJ, VM>(std::make_integer_sequence<int, RD>{});
    __builtin_amdgcn_sched_barrier(0);
    sx = sx1;
    sy = sy1;
  };
  // D windows at a time, so that the registers of codes on their way need not move; no way out between them, whose state
  // the compiler would join with that of the next turn.  The codes that a window of the tail loads are not used, and the compiler leaves
  // the loads out: its hand-over waits for fewer loads than IN_FLIGHT counts on, and dy of the window behind it may
  // not have landed.  No window reads that dy, as long as the tail is one window, the last.
  static_assert(!CODES || D <= 2, "a tail of more windows needs waits of its own");
  int w = w_lo;
  for (; w + D <= w_hi; w += D)
    each_window<D>([&](auto i_tag) {
      window(w + decltype(i_tag)::value, i_tag);
      return true;
    });
  each_window<D>([&](auto i_tag) {
    if (w + decltype(i_tag)::value >= w_hi) return false;
    window(w + decltype(i_tag)::value, i_tag);
    return true;
  });
  // lane l holds columns k 4 (l / 16) .. + 3 of row n l % 16 of each block
  float* const sums = part >= 0 ? p.part + ((int64_t)(seq - p.whole) * p.splits + part) * (T::BN * T::BK) : nullptr;
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int nl = (int)(wn * MJ + j) * 16 + (int)(lane & 15);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int kl = (int)(wk * MI + i) * 16 + 4 * (int)(lane >> 4);
      if (n0 + nl < p.N && k0 + kl < p.K) {
        if (sums)
          *reinterpret_cast<v4f*>(sums + nl * T::BK + kl) = acc[i][j];
        else
          store_sums<F32OUT>(p, n0 + nl, k0 + kl, acc[i][j]);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(grad_wait_vm(0));   // no load into LDS outlives the workgroup
}

// Joins the parts of M of the tiles from p.whole on, in a fixed order; 4 columns for each thread, blockIdx.y the tile.
// RUNS threads share those columns, each with every RUNS-th part, where there are many parts of few tiles: one
// thread would wait for one load after another (75600 x 128 x 128, 460 parts of one tile: the call 34 us, so 17.5).
// Not for up to 16 parts, where tiles are many (16384 x 1024 x 640, 12 parts of 40 tiles: 42.5 us for 45).
template <bool F32OUT, int BN, int BK, int RUNS>
__global__ __launch_bounds__(256) void grad_weight_sums_kernel(GradParams p) {
  constexpr int COLS = 256 / RUNS;
  __shared__ v4f runs[RUNS][COLS];
  int tk, tn;
  grad_tile_at(p, p.whole + (int)blockIdx.y, tk, tn);
  const int c = (int)threadIdx.x % COLS, run = (int)threadIdx.x / COLS;
  const int i = (int)blockIdx.x * COLS + c, nl = i / (BK / 4), kl = i % (BK / 4) * 4;
  const int n = tn * BN + nl, k = tk * BK + kl;
  const bool in = n < p.N && k < p.K;
  v4f v = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  if (in) {
    const float* from = p.part + (int64_t)blockIdx.y * p.splits * (BN * BK) + nl * BK + kl;
#pragma unroll 4
    for (int s = run; s < p.splits; s += RUNS) v += *reinterpret_cast<const v4f*>(from + (int64_t)s * (BN * BK));
  }
  if constexpr (RUNS > 1) {
    runs[run][c] = v;
    __syncthreads();
    if (run > 0) return;
#pragma unroll
    for (int r = 1; r < RUNS; ++r) v += runs[r][c];
  }
  if (in) store_sums<F32OUT>(p, n, k, v);
}

// Which tile, and how the tiles share the GPU: as many whole rounds of it as there are, and the rest of the
// tiles cut into parts of M.  Times in us.  Measured, tokens x N x K:
//                         256-wide  128-wide    not cut
//   64 x 13824 x 5120           64        56         56
//   700 x 3000 x 3008           33        30         30
//   2000 x 1024 x 1024          32        25         28
//   4096 x 2048 x 2048          55        55         55
//   16384 x 1024 x 640          48        41        177
//   3584 x 5120 x 5120         177       217        177
//   60000 x 2048 x 512         144       160        655
//   20000 x 64 x 5120          101        43        217
struct GradPlan {
  int size, splits, tiles_n, tiles_k, whole;
};
GradPlan plan_grad(int64_t M, int64_t N, int64_t K) {
  GradPlan best = {};
  double least = 0.0;
  const int nwin = (int)((M + kWinRows - 1) / kWinRows);
  for (const int size : {256, 128}) {
    const int64_t slots = size == 256 ? 256 : 512;                  // workgroups at once
    const double window = size == 256 ? 1.65 : 1.15;                // of a workgroup on a full GPU,
    const double alone = size == 256 ? 1.65 : 0.72;                 // and with a CU to itself
    const double ends = size == 256 ? 10.0 : 5.0;                   // first loads, last stores
    const int64_t tn = (N + size - 1) / size, tk = (K + size - 1) / size, tiles = tn * tk;
    const int64_t whole = tiles / slots * slots, rest = tiles - whole;
    auto rounds = [&](int64_t n, int windows) {                     // of n workgroups
      const int64_t full = n / slots, left = n - full * slots;
      return (double)full * (windows * window + ends) + (left > 0 ? windows * (left <= 256 ? alone : window) + ends : 0.0);
    };
    // the largest tile's operand is widened by a launch of its own
    const double base = rounds(whole, nwin) + (size == 256 ? 4.0 + (double)M * K * 3 / 5.5e6 : 0.0);
    // every number of parts up to 32, then steps of 1 in 32, for the host's time (75600 x 128 x 128: 7.5 us, so 2.8)
    for (int s = 1; s == 1 || (s * 2 <= nwin && rest * s <= 4 * slots); s += 1 + s / 32) {
      double t = base;
      if (rest > 0) {
        t += rounds(rest * s, (nwin + s - 1) / s);
        if (s > 1) t += 5.0 + (double)(rest * s * size * size) * 4.0 / 5.5e6;
      }
      if (least == 0.0 || t < least) {
        least = t;
        best = {size, s, (int)tn, (int)tk, s > 1 ? (int)whole : (int)tiles};
      }
      if (rest == 0) break;
    }
  }
  return best;
}

// The values of the codes, where they are widened ahead of the product.
size_t values_bytes(const GradPlan& g, int64_t M, int64_t K) {
  return g.size == 256 ? ((size_t)M * (size_t)K * 2 + 255) / 256 * 256 : 0;
}

}  // namespace

size_t grad_weight_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const GradPlan g = plan_grad(M, N, K);
  return values_bytes(g, M, K) + (size_t)(g.tiles_n * g.tiles_k - g.whole) * g.splits * g.size * g.size * 4;
}

hipError_t launch_grad_weight_int8(const uint16_t* dy, int64_t ld_dy, const int8_t* codes, int64_t ld_codes,
                                   const float* scales, int64_t M, int64_t N, int64_t K, void* out, bool f32_out,
                                   int64_t ld_out, bool accumulate, void* workspace, hipStream_t stream) {
  if (N == 0 || K == 0 || (M == 0 && accumulate)) return hipSuccess;
  const GradPlan g = plan_grad(M, N, K);
  uint16_t* x = static_cast<uint16_t*>(workspace);
  if (g.size == 256) {
    const hipError_t e = launch_dequantize_int8(codes, ld_codes, scales, M, K, x, K, stream);
    if (e != hipSuccess) return e;
  }
  GradParams p;
  p.dy = dy;
  p.x = x;
  p.codes = codes;
  p.scales = scales;
  p.ld_codes = ld_codes;
  p.out = out;
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + values_bytes(g, M, K));
  p.ld_dy = ld_dy;
  p.ld_x = K;
  p.ld_out = ld_out;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.nwin = (int)((M + kWinRows - 1) / kWinRows);
  p.tiles_n = g.tiles_n;
  p.tiles_k = g.tiles_k;
  p.whole = g.whole;
  p.splits = g.splits;
  p.accumulate = accumulate;
  const uintptr_t step = f32_out ? 4 : 2;
  p.vec = reinterpret_cast<uintptr_t>(out) % (4 * step) == 0 && ld_out % 4 == 0;
  const int rest = g.tiles_n * g.tiles_k - g.whole;
  const unsigned grid = (unsigned)(g.whole + rest * g.splits);
  auto go = [&](auto f_tag, auto c_tag, auto tile) {
    constexpr bool F = decltype(f_tag)::value, C = decltype(c_tag)::value;
    using T = decltype(tile);
    hipLaunchKernelGGL((grad_weight_kernel<F, C, T>), dim3(grid), dim3(T::THREADS), 0, stream, p);
    auto sums = [&](auto runs) {
      constexpr int R = decltype(runs)::value;
      hipLaunchKernelGGL((grad_weight_sums_kernel<F, T::BN, T::BK, R>), dim3(T::BN * T::BK / 1024 * R, rest), dim3(256), 0, stream, p);
    };
    if (rest > 0 && g.splits > 16)
      sums(std::integral_constant<int, 16>{});
    else if (rest > 0)
      sums(std::integral_constant<int, 1>{});
  };
  auto size = [&](auto f) {
    if (g.size == 256)
      go(f, std::false_type{}, GradTile<4, 8, 4, 2, 3>{});
    else
      go(f, std::true_type{}, GradTile<4, 4, 2, 2, 3>{});
  };
  f32_out ? size(std::true_type{}) : size(std::false_type{});
  return hipGetLastError();
}

}  // namespace mxq
