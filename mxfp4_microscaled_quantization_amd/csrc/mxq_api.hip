// C ABI of libmxq: argument validation, error reporting and dispatch to the gfx950
// launchers.  Every check runs before anything is enqueued, so an error return means the
// stream was not touched.  The only mutable state is the thread-local error message.
#include <float.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <string>

#include "../../include/mxq.h"
#include "mxq_internal.hpp"

namespace {

thread_local std::string g_error;

mxq_status fail(mxq_status code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_error = buf;
  return code;
}

mxq_status ok() {
  g_error.clear();
  return MXQ_OK;
}

mxq_status hip_status(const char* fn, hipError_t e) {
  if (e != hipSuccess) return fail(MXQ_ERR_HIP, "%s: HIP error %d (%s)", fn, (int)e, hipGetErrorString(e));
  return ok();
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Row pitches (elements or bytes) are below 2^32, dimensions below 2^31: every product the
// checks and the launchers form then stays inside int64.
constexpr int64_t kMaxPitch = ((int64_t)1 << 32) - 1;
constexpr int64_t kMaxDim = 0x7FFFFFFF;
bool pitch_ok(int64_t ld) { return ld <= kMaxPitch; }

int dtype_bytes(mxq_dtype dt) {
  switch (dt) {
    case MXQ_F32: return 4;
    case MXQ_BF16: return 2;
    default: return 0;   // unknown: rejected by the callers
  }
}

// Shared checks for a rows x cols input of dtype dt with pitch ld (elements).
mxq_status check_input(const char* fn, const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld,
                       int64_t col_multiple) {
  if (dtype_bytes(dt) == 0) return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
  if (rows < 0 || cols < 0) return fail(MXQ_ERR_INVALID_ARG, "%s: negative size (%lld x %lld)", fn, (long long)rows, (long long)cols);
  if (cols % col_multiple != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be a multiple of %lld", fn, (long long)cols,
                (long long)col_multiple);
  if (ld < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_x (%lld) < cols (%lld)", fn, (long long)ld, (long long)cols);
  if (rows > kMaxDim || cols > kMaxDim) return fail(MXQ_ERR_INVALID_ARG, "%s: dimension exceeds 2^31-1", fn);
  if (!pitch_ok(ld)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_x (%lld) must be below 2^32", fn, (long long)ld);
  if (rows > 0 && cols > 0) {
    if (!x) return fail(MXQ_ERR_INVALID_ARG, "%s: x is NULL", fn);
    if (!aligned(x, 16) || (ld * dtype_bytes(dt)) % 16 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: x base and row pitch must be 16-byte aligned", fn);
  }
  if ((rows * (cols / 8 > 0 ? cols / 8 : 1)) >= ((int64_t)1 << 32))
    return fail(MXQ_ERR_INVALID_ARG, "%s: tensor too large (more than 2^35 elements)", fn);
  return MXQ_OK;
}

mxq_status check_gemm(const char* fn, int64_t M, int64_t N, int64_t K, const void* out, int64_t ld_out) {
  if (M < 0 || N < 0 || K < 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: negative size (M=%lld N=%lld K=%lld)", fn, (long long)M, (long long)N,
                (long long)K);
  if (K % 32 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: K (%lld) must be a multiple of 32", fn, (long long)K);
  if (M > (int64_t)0x7FFFFFFF - 256 || N > (int64_t)0x7FFFFFFF - 256 || K > ((int64_t)1 << 21))
    return fail(MXQ_ERR_INVALID_ARG, "%s: dimension too large", fn);
  if (ld_out < N) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_out (%lld) < N (%lld)", fn, (long long)ld_out, (long long)N);
  if (!pitch_ok(ld_out)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_out (%lld) must be below 2^32", fn, (long long)ld_out);
  if (M > 0 && N > 0) {
    if (!out) return fail(MXQ_ERR_INVALID_ARG, "%s: out is NULL", fn);
    if (!aligned(out, 2)) return fail(MXQ_ERR_INVALID_ARG, "%s: out must be 2-byte aligned", fn);
    const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
    if (tiles > 0x7FFFFFFF) return fail(MXQ_ERR_INVALID_ARG, "%s: problem too large", fn);
  }
  return MXQ_OK;
}

mxq_status check_operand(const char* fn, const char* name, const void* p, int64_t rows, int64_t K, int align) {
  if (rows > 0 && K > 0) {
    if (!p) return fail(MXQ_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (!aligned(p, (uintptr_t)align)) return fail(MXQ_ERR_INVALID_ARG, "%s: %s must be %d-byte aligned", fn, name, align);
  }
  return MXQ_OK;
}

// Checks of the 8-bit product that do not concern the activations.
mxq_status check_w8(const char* fn, const int8_t* w, int64_t ld_w, const float* w_scales, int64_t inc_ws,
                    const float* bias, int64_t M, int64_t N, int64_t K, const void* out, mxq_dtype out_dt,
                    int64_t ld_out) {
  const int ob = dtype_bytes(out_dt);
  if (ob == 0) return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown output dtype %d", fn, (int)out_dt);
  if (M < 0 || N < 0 || K < 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: negative size (M=%lld N=%lld K=%lld)", fn, (long long)M, (long long)N,
                (long long)K);
  if (K % 16 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: K (%lld) must be a multiple of 16", fn, (long long)K);
  if (K >= ((int64_t)1 << 17))
    return fail(MXQ_ERR_INVALID_ARG, "%s: K (%lld) must be below 2^17 (int32 sums)", fn, (long long)K);
  if (M > kMaxDim - 256 || N > kMaxDim - 256) return fail(MXQ_ERR_INVALID_ARG, "%s: dimension too large", fn);
  if (ld_out < N) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_out (%lld) < N (%lld)", fn, (long long)ld_out, (long long)N);
  if (!pitch_ok(ld_out)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_out (%lld) must be below 2^32", fn, (long long)ld_out);
  if (ld_w < K || ld_w >= ((int64_t)1 << 23))
    return fail(MXQ_ERR_INVALID_ARG, "%s: ld_w (%lld) must be at least K and below 2^23", fn, (long long)ld_w);
  if (inc_ws < 0 || !pitch_ok(inc_ws)) return fail(MXQ_ERR_INVALID_ARG, "%s: inc_ws out of range", fn);
  if (M > 0 && N > 0) {
    // threads of a launch stay below 2^32: 512 for each 256 x 256 tile, 256 for each 32 channels
    // of a few tokens
    if (((M + 255) / 256) * ((N + 255) / 256) > ((int64_t)1 << 22) || N > ((int64_t)1 << 28))
      return fail(MXQ_ERR_INVALID_ARG, "%s: problem too large", fn);
    if (!out) return fail(MXQ_ERR_INVALID_ARG, "%s: out is NULL", fn);
    if (!aligned(out, (uintptr_t)ob)) return fail(MXQ_ERR_INVALID_ARG, "%s: out must be %d-byte aligned", fn, ob);
    if (!w_scales || !aligned(w_scales, 4))
      return fail(MXQ_ERR_INVALID_ARG, "%s: w_scales must be a non-NULL 4-byte aligned pointer", fn);
    if (!aligned(bias, 4)) return fail(MXQ_ERR_INVALID_ARG, "%s: bias must be 4-byte aligned", fn);
    if (K > 0) {
      if (!w) return fail(MXQ_ERR_INVALID_ARG, "%s: w is NULL", fn);
      if (!aligned(w, 16) || ld_w % 16 != 0)
        return fail(MXQ_ERR_INVALID_ARG, "%s: w base and ld_w must be multiples of 16 bytes", fn);
    }
  }
  return MXQ_OK;
}

// Shapes for which the 8-bit workspaces have a size.
bool w8_shape_ok(int64_t M, int64_t N, int64_t K) {
  return M > 0 && N > 0 && K >= 0 && K % 16 == 0 && M <= kMaxDim - 256 && N <= kMaxDim - 256 && K < ((int64_t)1 << 17);
}

// Codes and scales of quantized activations, in 16-byte steps.  Rows of codes start on cache
// lines (128 bytes), which the product reads faster than others (1144 x 4272 x 384: 18.8 ->
// 16.9 us, 3000 x 5008 x 5120: 87 -> 82).
int64_t fused_pitch(int64_t K) { return (K + 127) / 128 * 128; }
size_t fused_codes_bytes(int64_t M, int64_t K) { return (size_t)M * (size_t)fused_pitch(K) + ((size_t)M + 3) / 4 * 16; }

// Arguments of one side (queries or keys) of the head norm.
struct HeadArgs {
  const char* name;
  const void* x;
  int64_t heads, ld, hs;
  const void* w;
  void* out;
  int64_t ld_o, hs_o;
  float* scales;
  int64_t ld_s;
};

// Whether every (token, head) has `width` elements of its own at token * ld + head * hs, both
// pitches >= width.  The usual layouts hold all heads of a token between two tokens, or all tokens
// of a head between two heads.  In any other, places meet where some difference of a positive
// number of heads and of tokens comes closer than `width`: for each number on the axis with fewer,
// only the two multiples of the other pitch around it can (at most 65535 of them).
bool heads_apart(int64_t tokens, int64_t heads, int64_t ld, int64_t hs, int64_t width) {
  if (tokens <= 1 || heads <= 1 || ld >= (heads - 1) * hs + width || hs >= (tokens - 1) * ld + width) return true;
  const bool by_head = heads <= tokens;
  const int64_t few = by_head ? heads : tokens, many = by_head ? tokens : heads;
  const int64_t step = by_head ? hs : ld, other = by_head ? ld : hs;
  for (int64_t i = 1; i < few; ++i)
    for (int64_t j = i * step / other, end = j + 2; j < end; ++j) {
      const int64_t off = i * step - j * other;
      if (j >= 1 && j < many && off < width && -off < width) return false;
    }
  return true;
}

mxq_status check_heads(const char* fn, const HeadArgs& h, int bytes, int out_bytes, int out_align, int w_bytes,
                       int64_t tokens, int64_t head_dim, bool quant) {
  if (h.heads < 0 || h.heads > 65536)
    return fail(MXQ_ERR_INVALID_ARG, "%s: heads_%s (%lld) must be 0 to 65536", fn, h.name, (long long)h.heads);
  if (h.heads == 0 || tokens == 0) return MXQ_OK;
  if (h.ld < 0 || h.hs < 0 || h.ld_o < 0 || h.hs_o < 0 || !pitch_ok(h.ld) || !pitch_ok(h.hs) || !pitch_ok(h.ld_o) ||
      !pitch_ok(h.hs_o))
    return fail(MXQ_ERR_INVALID_ARG, "%s: pitches of %s must be 0 to 2^32 - 1", fn, h.name);
  // offsets inside a token, those of the 16 heads that the last set may reach past its end
  // included, stay below 2^31
  if (h.heads > 1 && ((h.heads + 16) * h.hs * bytes >= (int64_t)1 << 31 || (h.heads + 16) * h.hs_o * out_bytes >= (int64_t)1 << 31))
    return fail(MXQ_ERR_INVALID_ARG, "%s: the heads of a token in %s span too far (2^31 bytes with 16 more)", fn, h.name);
  if (!h.x || !h.out) return fail(MXQ_ERR_INVALID_ARG, "%s: %s or its output is NULL", fn, h.name);
  if (!aligned(h.x, 16) || h.ld * bytes % 16 != 0 || h.hs * bytes % 16 != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: %s base and pitches must be 16-byte aligned", fn, h.name);
  if (!aligned(h.out, (uintptr_t)out_align) || h.ld_o * out_bytes % out_align != 0 || h.hs_o * out_bytes % out_align != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: output base and pitches of %s must be %d-byte aligned", fn, h.name, out_align);
  if ((h.heads > 1 && h.hs_o < head_dim) || (tokens > 1 && h.ld_o < head_dim))
    return fail(MXQ_ERR_INVALID_ARG, "%s: output pitches of %s below head_dim", fn, h.name);
  if (!heads_apart(tokens, h.heads, h.ld_o, h.hs_o, head_dim))
    return fail(MXQ_ERR_INVALID_ARG, "%s: output heads of %s overlap", fn, h.name);
  if (h.w && !aligned(h.w, (uintptr_t)(4 * w_bytes)))
    return fail(MXQ_ERR_INVALID_ARG, "%s: w_%s must be %d-byte aligned", fn, h.name, 4 * w_bytes);
  if (quant) {
    if (!h.scales || !aligned(h.scales, 4))
      return fail(MXQ_ERR_INVALID_ARG, "%s: scales_%s must be a non-NULL 4-byte aligned pointer", fn, h.name);
    if (!pitch_ok(h.ld_s) || (tokens > 1 && h.ld_s < h.heads))
      return fail(MXQ_ERR_INVALID_ARG, "%s: ld of scales_%s below its heads", fn, h.name);
  }
  return MXQ_OK;
}

mxq_status qk_norm_rope(const char* fn, HeadArgs q, HeadArgs k, mxq_dtype dt, int64_t tokens, int64_t head_dim,
                        mxq_dtype w_dt, float eps, const float* cos, const float* sin, int64_t ld_table,
                        int64_t table_rows, int64_t rot_dim, const int64_t* positions, mxq_rope_style style,
                        bool quant, hipStream_t stream) {
  const int bytes = dtype_bytes(dt), w_bytes = dtype_bytes(w_dt);
  if (bytes == 0 || w_bytes == 0) return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown dtype %d or %d", fn, (int)dt, (int)w_dt);
  if (style != MXQ_ROPE_INTERLEAVED && style != MXQ_ROPE_HALVES)
    return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown rotation style %d", fn, (int)style);
  if (tokens < 0 || tokens > kMaxDim) return fail(MXQ_ERR_INVALID_ARG, "%s: tokens (%lld) out of range", fn, (long long)tokens);
  if (head_dim < 8 || head_dim > 512 || head_dim % 8 != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: head_dim (%lld) must be a multiple of 8, 8 to 512", fn, (long long)head_dim);
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 8 != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: rot_dim (%lld) must be a multiple of 8, 0 to head_dim", fn, (long long)rot_dim);
  if (!(eps >= 0.0f) || !(eps < __builtin_inff())) return fail(MXQ_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  const int out_bytes = quant ? 1 : bytes, out_align = quant ? 8 : 16;
  for (const HeadArgs* h : {&q, &k}) {
    const mxq_status st = check_heads(fn, *h, bytes, out_bytes, out_align, w_bytes, tokens, head_dim, quant);
    if (st != MXQ_OK) return st;
  }
  if (tokens == 0 || q.heads + k.heads == 0) return ok();
  if (rot_dim > 0) {
    if (!cos || !sin || !aligned(cos, 16) || !aligned(sin, 16))
      return fail(MXQ_ERR_INVALID_ARG, "%s: cos and sin must be non-NULL and 16-byte aligned", fn);
    if (ld_table < rot_dim / 2 || ld_table % 4 != 0 || !pitch_ok(ld_table))
      return fail(MXQ_ERR_INVALID_ARG, "%s: ld_table (%lld) must be a multiple of 4, at least rot_dim / 2", fn,
                  (long long)ld_table);
    if (table_rows < 0 || table_rows > kMaxDim || (!positions && table_rows < tokens))
      return fail(MXQ_ERR_INVALID_ARG, "%s: table_rows (%lld) below the tokens without positions", fn,
                  (long long)table_rows);
    if (!aligned(positions, 8)) return fail(MXQ_ERR_INVALID_ARG, "%s: positions must be 8-byte aligned", fn);
  }
  auto side = [&](const HeadArgs& h) {
    const bool many = h.heads > 1;   // a single head has no head pitch
    return mxq::QkSide{h.x, h.heads > 0 ? h.w : nullptr, h.out, h.scales, h.ld, many ? h.hs : head_dim, h.ld_o,
                       many ? h.hs_o : head_dim, h.ld_s, (int)h.heads};
  };
  mxq::QkNormParams p;
  p.q = side(q);
  p.k = side(k);
  p.tokens = tokens;
  p.ld_table = ld_table;
  p.table_rows = table_rows;
  p.cos = cos;
  p.sin = sin;
  p.positions = positions;
  p.head_dim = (int)head_dim;
  p.rot_dim = (int)rot_dim;
  p.w_f32 = w_dt == MXQ_F32 ? 1 : 0;
  p.eps = eps;
  p.inv_dim = 1.0f / (float)head_dim;
  return hip_status(fn, mxq::launch_qk_norm_rope(p, dt == MXQ_F32, quant, style == MXQ_ROPE_HALVES, stream));
}

// A rows x cols plane of elements of `bytes` besides the input: pitch, and where it is not empty,
// pointer and alignment.
mxq_status check_plane(const char* fn, const char* name, const void* ptr, int64_t rows, int64_t cols, int64_t ld,
                       int64_t bytes, int64_t align) {
  if (ld < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: ld of %s (%lld) < cols (%lld)", fn, name, (long long)ld, (long long)cols);
  if (!pitch_ok(ld)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld of %s (%lld) must be below 2^32", fn, name, (long long)ld);
  if (rows > 0 && cols > 0) {
    if (!ptr) return fail(MXQ_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (!aligned(ptr, (uintptr_t)align) || ld * bytes % align != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: %s base and row pitch must be %lld-byte aligned", fn, name, (long long)align);
  }
  return MXQ_OK;
}

// A float for each row, or none where `may_be_null`.
mxq_status check_row_values(const char* fn, const char* name, const float* ptr, int64_t rows, bool may_be_null) {
  if (rows > 0 && ((!ptr && !may_be_null) || !aligned(ptr, 4)))
    return fail(MXQ_ERR_INVALID_ARG, "%s: %s must be a %s4-byte aligned pointer", fn, name, may_be_null ? "" : "non-NULL ");
  return MXQ_OK;
}

mxq_status check_norm(const char* fn, int64_t cols, const void* w, const void* b, mxq_dtype w_dt) {
  if (dtype_bytes(w_dt) == 0) return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)w_dt);
  if (cols < 8 || cols > mxq::kNormMaxCols)
    return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be 8 to %lld", fn, (long long)cols, (long long)mxq::kNormMaxCols);
  if (!aligned(w, 16) || !aligned(b, 16)) return fail(MXQ_ERR_INVALID_ARG, "%s: w and b must be 16-byte aligned", fn);
  return MXQ_OK;
}

mxq_status layer_norm(const char* fn, const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                      const void* w, const void* b, mxq_dtype w_dt, float eps, void* y, int64_t ld_y, float* scales,
                      float* mean, float* rstd, int8_t* x_codes, int64_t ld_xc, float* x_scales, bool quant,
                      hipStream_t stream) {
  mxq_status st = check_input(fn, x, dt, rows, cols, ld_x, quant || x_codes ? 16 : 8);
  if (st != MXQ_OK) return st;
  if ((st = check_norm(fn, cols, w, b, w_dt)) != MXQ_OK) return st;
  if (!(eps >= 0.0f) || !(eps < __builtin_inff())) return fail(MXQ_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if ((st = check_plane(fn, quant ? "codes" : "y", y, rows, cols, ld_y, quant ? 1 : dtype_bytes(dt), 16)) != MXQ_OK) return st;
  if (quant && (st = check_row_values(fn, "scales", scales, rows, false)) != MXQ_OK) return st;
  if (!mean != !rstd) return fail(MXQ_ERR_INVALID_ARG, "%s: mean and rstd must be given together", fn);
  if ((st = check_row_values(fn, "mean", mean, rows, true)) != MXQ_OK) return st;
  if ((st = check_row_values(fn, "rstd", rstd, rows, true)) != MXQ_OK) return st;
  if (x_codes) {
    if ((st = check_plane(fn, "x_codes", x_codes, rows, cols, ld_xc, 1, 16)) != MXQ_OK) return st;
    if ((st = check_row_values(fn, "x_scales", x_scales, rows, false)) != MXQ_OK) return st;
  }
  mxq::NormParams p;
  p.x = x;
  p.w = w;
  p.b = b;
  p.y = y;
  p.scales = scales;
  p.mean = mean;
  p.rstd = rstd;
  p.kept = x_codes;
  p.kept_scales = x_scales;
  p.rows = rows;
  p.ld_x = ld_x;
  p.ld_y = ld_y;
  p.ld_kept = ld_xc;
  p.units = (uint32_t)(cols / 8);
  p.w_f32 = w_dt == MXQ_F32 ? 1 : 0;
  p.eps = eps;
  p.cols = (float)cols;
  p.inv_cols = 1.0f / (float)cols;
  return hip_status(fn, mxq::launch_layer_norm(p, dt == MXQ_F32, quant, stream));
}

mxq_status check_act(const char* fn, mxq_activation_kind act) {
  if (act != MXQ_ACT_GELU_TANH && act != MXQ_ACT_SILU)
    return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown activation %d", fn, (int)act);
  return MXQ_OK;
}

mxq_status activation(const char* fn, const void* u, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_u,
                      mxq_activation_kind act, void* y, int64_t ld_y, float* scales, int8_t* u_codes, int64_t ld_uc,
                      float* u_scales, bool quant, hipStream_t stream) {
  mxq_status st = check_act(fn, act);
  if (st != MXQ_OK) return st;
  if ((st = check_input(fn, u, dt, rows, cols, ld_u, quant || u_codes ? 16 : 8)) != MXQ_OK) return st;
  if (cols > mxq::kActMaxCols)
    return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be at most %lld", fn, (long long)cols, (long long)mxq::kActMaxCols);
  if ((st = check_plane(fn, quant ? "codes" : "y", y, rows, cols, ld_y, quant ? 1 : dtype_bytes(dt), 16)) != MXQ_OK) return st;
  if (quant && (st = check_row_values(fn, "scales", scales, rows, false)) != MXQ_OK) return st;
  if (u_codes) {
    if ((st = check_plane(fn, "u_codes", u_codes, rows, cols, ld_uc, 1, 16)) != MXQ_OK) return st;
    if ((st = check_row_values(fn, "u_scales", u_scales, rows, false)) != MXQ_OK) return st;
  }
  mxq::ActParams p;
  p.u = u;
  p.y = y;
  p.scales = scales;
  p.kept = u_codes;
  p.kept_scales = u_scales;
  p.rows = rows;
  p.ld_u = ld_u;
  p.ld_y = ld_y;
  p.ld_kept = ld_uc;
  p.units = (uint32_t)(cols / 8);
  return hip_status(fn, mxq::launch_activation(p, dt == MXQ_F32, quant,
                                               act == MXQ_ACT_GELU_TANH ? mxq::ACT_GELU_TANH : mxq::ACT_SILU, stream));
}

// Shapes of which the weight gradient has a plan.
bool grad_shape_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N > 0 && K > 0 && N % 8 == 0 && K % 16 == 0 && M <= kMaxDim - 256 && N <= ((int64_t)1 << 22) &&
         K <= ((int64_t)1 << 22) && N * K <= ((int64_t)1 << 36) && M * (K / 8) < ((int64_t)1 << 32);
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int mxq_abi_version(void) { return MXQ_ABI_VERSION; }

const char* mxq_last_error(void) { return g_error.c_str(); }

mxq_status mxq_quantize_rule(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* codes,
                             int64_t ld_codes, uint8_t* scales, int64_t ld_scales, mxq_scale_rule rule, void* stream) {
  const char* fn = "mxq_quantize";
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS)
    return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown scale rule %d", fn, (int)rule);
  mxq_status st = check_input(fn, x, dt, rows, cols, ld_x, 32);
  if (st != MXQ_OK) return st;
  if (ld_codes < cols / 2) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_codes (%lld) < cols/2", fn, (long long)ld_codes);
  if (ld_scales < cols / 32) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_scales (%lld) < cols/32", fn, (long long)ld_scales);
  if (!pitch_ok(ld_codes) || !pitch_ok(ld_scales)) return fail(MXQ_ERR_INVALID_ARG, "%s: pitch must be below 2^32", fn);
  if (rows > 0 && cols > 0) {
    if (!codes || !scales) return fail(MXQ_ERR_INVALID_ARG, "%s: codes/scales is NULL", fn);
    if (!aligned(codes, 16) || ld_codes % 16 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: codes base and ld_codes must be multiples of 16 bytes", fn);
  }
  return hip_status(fn, mxq::launch_quantize_mxfp4(x, dt == MXQ_F32, rows, cols, ld_x, codes, ld_codes, scales,
                                                   ld_scales, rule == MXQ_SCALE_UOS, as_stream(stream)));
}

mxq_status mxq_quantize(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* codes,
                        int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* stream) {
  return mxq_quantize_rule(x, dt, rows, cols, ld_x, codes, ld_codes, scales, ld_scales, MXQ_SCALE_OCP, stream);
}

mxq_status mxq_quantize_hadamard(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, int block_n,
                                 mxq_scale_rule rule, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                                 int64_t ld_scales, void* stream) {
  const char* fn = "mxq_quantize_hadamard";
  if (block_n != 16 && block_n != 64 && block_n != 256)
    return fail(MXQ_ERR_UNSUPPORTED, "%s: block_n must be 16, 64 or 256 (got %d)", fn, block_n);
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS)
    return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown scale rule %d", fn, (int)rule);
  mxq_status st = check_input(fn, x, dt, rows, cols, ld_x, 32);
  if (st != MXQ_OK) return st;
  if (cols % block_n != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be a multiple of block_n (%d)", fn, (long long)cols, block_n);
  if (ld_codes < cols / 2) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_codes (%lld) < cols/2", fn, (long long)ld_codes);
  if (ld_scales < cols / 32) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_scales (%lld) < cols/32", fn, (long long)ld_scales);
  if (!pitch_ok(ld_codes) || !pitch_ok(ld_scales)) return fail(MXQ_ERR_INVALID_ARG, "%s: pitch must be below 2^32", fn);
  if (rows > 0 && cols > 0) {
    if (!codes || !scales) return fail(MXQ_ERR_INVALID_ARG, "%s: codes/scales is NULL", fn);
    if (!aligned(codes, 16) || ld_codes % 16 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: codes base and ld_codes must be multiples of 16 bytes", fn);
  }
  return hip_status(fn, mxq::launch_quantize_mxfp4_rotated(x, dt == MXQ_F32, rows, cols, ld_x, block_n, codes, ld_codes,
                                                           scales, ld_scales, rule == MXQ_SCALE_UOS, as_stream(stream)));
}

mxq_status mxq_quantize_fp8(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, float inv_scale,
                            uint8_t* q, int64_t ld_q, void* stream) {
  const char* fn = "mxq_quantize_fp8";
  mxq_status st = check_input(fn, x, dt, rows, cols, ld_x, 16);
  if (st != MXQ_OK) return st;
  if (!(inv_scale > 0.0f) || !(inv_scale < __builtin_inff()))
    return fail(MXQ_ERR_INVALID_ARG, "%s: inv_scale must be finite and > 0", fn);
  if (ld_q < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_q (%lld) < cols", fn, (long long)ld_q);
  if (!pitch_ok(ld_q)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_q (%lld) must be below 2^32", fn, (long long)ld_q);
  if (rows > 0 && cols > 0) {
    if (!q) return fail(MXQ_ERR_INVALID_ARG, "%s: q is NULL", fn);
    if (!aligned(q, 16) || ld_q % 16 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: q base and ld_q must be multiples of 16 bytes", fn);
  }
  return hip_status(fn, mxq::launch_quantize_fp8(x, dt == MXQ_F32, rows, cols, ld_x, inv_scale, q, ld_q,
                                                 as_stream(stream)));
}

mxq_status mxq_fp8_static_scales(float amax, float* s_a, float* inv_s) {
  const char* fn = "mxq_fp8_static_scales";
  if (!s_a || !inv_s) return fail(MXQ_ERR_INVALID_ARG, "%s: s_a/inv_s is NULL", fn);
  if (!(amax > 0.0f) || !(amax <= FLT_MAX))
    return fail(MXQ_ERR_INVALID_ARG, "%s: amax must be finite and > 0 (got %g)", fn, (double)amax);
  // IEEE binary32 division rounds the exact quotient to nearest even: fl32(amax / 448)
  // and fl32(448 / amax)
  const float sa = amax / 448.0f;
  const float inv = 448.0f / amax;
  if (!(inv <= FLT_MAX))
    return fail(MXQ_ERR_INVALID_ARG, "%s: amax (%g) too small: 448 / amax overflows binary32", fn, (double)amax);
  *s_a = sa;
  *inv_s = inv;
  return ok();
}

mxq_status mxq_absmax(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, float* out,
                      void* stream) {
  const char* fn = "mxq_absmax";
  mxq_status st = check_input(fn, x, dt, rows, cols, ld_x, 8);
  if (st != MXQ_OK) return st;
  if (!out || !aligned(out, 4)) return fail(MXQ_ERR_INVALID_ARG, "%s: out must be a non-NULL 4-byte aligned pointer", fn);
  return hip_status(fn, mxq::launch_absmax(x, dt == MXQ_F32, rows, cols, ld_x, out, as_stream(stream)));
}

mxq_status mxq_gemm_w4a4(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                         const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, uint16_t* out_bf16,
                         int64_t ld_out, void* stream) {
  const char* fn = "mxq_gemm_w4a4";
  mxq_status st = check_gemm(fn, M, N, K, out_bf16, ld_out);
  if (st != MXQ_OK) return st;
  if (M > 0 && N > 0) {
    if ((st = check_operand(fn, "a_codes", a_codes, M, K, 16)) != MXQ_OK) return st;
    if ((st = check_operand(fn, "a_scales", a_scales, M, K, 1)) != MXQ_OK) return st;
    if ((st = check_operand(fn, "w_codes", w_codes, N, K, 16)) != MXQ_OK) return st;
    if ((st = check_operand(fn, "w_scales", w_scales, N, K, 1)) != MXQ_OK) return st;
  }
  return hip_status(fn, mxq::launch_gemm(mxq::GEMM_W4A4, a_codes, a_scales, w_codes, w_scales, 1.0f, M, N, K,
                                         out_bf16, ld_out, as_stream(stream)));
}

// Break-even of the fused W4A4 kernel: it quantizes every activation tile once per
// 256-column output tile, so its cost grows with N, while quantization in a pass of its
// own is paid once.  Measured on MI355X (M = 57344 and 75600): fused is the faster up to
// 3 column tiles (N <= 768) for K >= 8192 (K = 12288: 0.99 of the separate pair at N = 768,
// 1.05 at 1024; K = 13824: 0.96 and 1.02) and up to 1 tile for K = 3072 (0.96 at N = 256,
// 1.04 at 512).
int64_t fused_max_col_tiles(int64_t K) { return K >= 8192 ? 3 : 1; }
int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

size_t mxq_gemm_w4a4_fused_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 32 != 0) return 0;
  if (M > kMaxDim || N > kMaxDim || K > ((int64_t)1 << 21)) return 0;   // a shape the GEMM rejects
  if ((N + 255) / 256 <= fused_max_col_tiles(K)) return 0;
  return (size_t)(round16(M * (K / 2)) + M * (K / 32));
}

mxq_status mxq_gemm_w4a4_fused(const void* a, mxq_dtype dt, int64_t ld_a, const uint8_t* w_codes,
                               const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, mxq_scale_rule rule,
                               uint16_t* out_bf16, int64_t ld_out, void* workspace, size_t ws_bytes,
                               void* stream) {
  const char* fn = "mxq_gemm_w4a4_fused";
  if (rule != MXQ_SCALE_OCP && rule != MXQ_SCALE_UOS)
    return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown scale rule %d", fn, (int)rule);
  if (dtype_bytes(dt) == 0) return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
  mxq_status st = check_gemm(fn, M, N, K, out_bf16, ld_out);
  if (st != MXQ_OK) return st;
  if (M > 0 && N > 0) {
    if ((st = check_input(fn, a, dt, M, K, ld_a, 32)) != MXQ_OK) return st;
    if (ld_a * dtype_bytes(dt) * 256 >= ((int64_t)1 << 31))
      return fail(MXQ_ERR_INVALID_ARG, "%s: row pitch too large (256 * ld_a * element size must be below 2^31 bytes)",
                  fn);
    if ((st = check_operand(fn, "w_codes", w_codes, N, K, 16)) != MXQ_OK) return st;
    if ((st = check_operand(fn, "w_scales", w_scales, N, K, 1)) != MXQ_OK) return st;
    if (K > 0 && !a) return fail(MXQ_ERR_INVALID_ARG, "%s: a is NULL", fn);
  }
  const size_t need = mxq_gemm_w4a4_fused_workspace_bytes(M, N, K);
  if (workspace && need > 0) {
    // past the break-even: quantize into the workspace, then the W4A4 GEMM (the same bits)
    if (!aligned(workspace, 16) || ws_bytes < need)
      return fail(MXQ_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned and at least %zu bytes (got %zu)", fn,
                  need, ws_bytes);
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + round16(M * (K / 2));
    hipError_t e = mxq::launch_quantize_mxfp4(a, dt == MXQ_F32, M, K, ld_a, codes, K / 2, scales, K / 32,
                                              rule == MXQ_SCALE_UOS, as_stream(stream));
    if (e != hipSuccess) return hip_status(fn, e);
    return hip_status(fn, mxq::launch_gemm(mxq::GEMM_W4A4, codes, scales, w_codes, w_scales, 1.0f, M, N, K, out_bf16,
                                           ld_out, as_stream(stream)));
  }
  return hip_status(fn, mxq::launch_gemm_w4a4_fused(a, dt == MXQ_F32, ld_a, w_codes, w_scales, M, N, K,
                                                    rule == MXQ_SCALE_UOS, out_bf16, ld_out, as_stream(stream)));
}

mxq_status mxq_gemm_w4a8(const uint8_t* a_fp8, float a_scale, const uint8_t* w_codes, const uint8_t* w_scales,
                         int64_t M, int64_t N, int64_t K, uint16_t* out_bf16, int64_t ld_out, void* stream) {
  const char* fn = "mxq_gemm_w4a8";
  mxq_status st = check_gemm(fn, M, N, K, out_bf16, ld_out);
  if (st != MXQ_OK) return st;
  if (!(a_scale == a_scale) || a_scale == __builtin_inff() || a_scale == -__builtin_inff())
    return fail(MXQ_ERR_INVALID_ARG, "%s: a_scale must be finite", fn);
  if (M > 0 && N > 0) {
    if ((st = check_operand(fn, "a_fp8", a_fp8, M, K, 16)) != MXQ_OK) return st;
    if ((st = check_operand(fn, "w_codes", w_codes, N, K, 16)) != MXQ_OK) return st;
    if ((st = check_operand(fn, "w_scales", w_scales, N, K, 1)) != MXQ_OK) return st;
  }
  return hip_status(fn, mxq::launch_gemm(mxq::GEMM_W4A8, a_fp8, nullptr, w_codes, w_scales, a_scale, M, N, K,
                                         out_bf16, ld_out, as_stream(stream)));
}

mxq_status mxq_gemm_bf16(const uint16_t* a, const uint16_t* w, int64_t M, int64_t N, int64_t K, uint16_t* out,
                         int64_t ld_out, void* stream) {
  const char* fn = "mxq_gemm_bf16";
  mxq_status st = check_gemm(fn, M, N, K, out, ld_out);
  if (st != MXQ_OK) return st;
  if (M > 0 && N > 0) {
    if ((st = check_operand(fn, "a", a, M, K, 16)) != MXQ_OK) return st;
    if ((st = check_operand(fn, "w", w, N, K, 16)) != MXQ_OK) return st;
  }
  return hip_status(fn, mxq::launch_gemm(mxq::GEMM_BF16, a, nullptr, w, nullptr, 1.0f, M, N, K, out, ld_out,
                                         as_stream(stream)));
}

size_t mxq_sqnr_workspace_bytes(int64_t n_elements) { return mxq::sqnr_workspace_bytes(n_elements); }

mxq_status mxq_sqnr(const uint16_t* ref, const uint16_t* test, int64_t rows, int64_t cols, int64_t ld_ref,
                    int64_t ld_test, void* workspace, size_t ws_bytes, double* out3, void* stream) {
  const char* fn = "mxq_sqnr";
  if (rows < 0 || cols < 0) return fail(MXQ_ERR_INVALID_ARG, "%s: negative size", fn);
  if (cols % 8 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be a multiple of 8", fn, (long long)cols);
  if (ld_ref < cols || ld_test < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: pitch below cols", fn);
  if (ld_ref % 8 != 0 || ld_test % 8 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: pitches must be multiples of 8", fn);
  if (rows > kMaxDim || cols > kMaxDim || !pitch_ok(ld_ref) || !pitch_ok(ld_test) ||
      rows * (cols / 8) >= ((int64_t)1 << 32))
    return fail(MXQ_ERR_INVALID_ARG, "%s: tensor too large", fn);
  if (!out3 || !aligned(out3, 8)) return fail(MXQ_ERR_INVALID_ARG, "%s: out3 must be a non-NULL 8-byte aligned pointer", fn);
  if (!workspace || !aligned(workspace, 8) || ws_bytes < mxq::sqnr_workspace_bytes(rows * cols))
    return fail(MXQ_ERR_INVALID_ARG, "%s: workspace missing, misaligned or smaller than %zu bytes", fn,
                mxq::sqnr_workspace_bytes(rows * cols));
  if (rows > 0 && cols > 0) {
    if (!ref || !test) return fail(MXQ_ERR_INVALID_ARG, "%s: ref/test is NULL", fn);
    if (!aligned(ref, 16) || !aligned(test, 16)) return fail(MXQ_ERR_INVALID_ARG, "%s: ref/test must be 16-byte aligned", fn);
  }
  return hip_status(fn, mxq::launch_sqnr(ref, test, rows, cols, ld_ref, ld_test, workspace, out3, as_stream(stream)));
}

mxq_status mxq_sqnr_noalloc(const uint16_t* ref, const uint16_t* test, int64_t rows, int64_t cols, int64_t ld_ref,
                            int64_t ld_test, double* out3, void* stream) {
  const char* fn = "mxq_sqnr_noalloc";
  if (rows < 0 || cols < 0) return fail(MXQ_ERR_INVALID_ARG, "%s: negative size", fn);
  if (cols % 8 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be a multiple of 8", fn, (long long)cols);
  if (ld_ref < cols || ld_test < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: pitch below cols", fn);
  if (ld_ref % 8 != 0 || ld_test % 8 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: pitches must be multiples of 8", fn);
  if (rows > kMaxDim || cols > kMaxDim || !pitch_ok(ld_ref) || !pitch_ok(ld_test) ||
      rows * (cols / 8) >= ((int64_t)1 << 32))
    return fail(MXQ_ERR_INVALID_ARG, "%s: tensor too large", fn);
  const size_t need = mxq::sqnr_workspace_bytes(rows * cols);
  if (need > mxq::sqnr_scratch_bytes())
    return fail(MXQ_ERR_INVALID_ARG, "%s: needs %zu bytes of workspace, above the library's %zu-byte scratch", fn,
                need, mxq::sqnr_scratch_bytes());
  if (!out3 || !aligned(out3, 8)) return fail(MXQ_ERR_INVALID_ARG, "%s: out3 must be a non-NULL 8-byte aligned pointer", fn);
  if (rows > 0 && cols > 0) {
    if (!ref || !test) return fail(MXQ_ERR_INVALID_ARG, "%s: ref/test is NULL", fn);
    if (!aligned(ref, 16) || !aligned(test, 16)) return fail(MXQ_ERR_INVALID_ARG, "%s: ref/test must be 16-byte aligned", fn);
  }
  void* ws = nullptr;
  hipError_t e = mxq::sqnr_scratch(&ws);
  if (e != hipSuccess) return hip_status(fn, e);
  return hip_status(fn, mxq::launch_sqnr(ref, test, rows, cols, ld_ref, ld_test, ws, out3, as_stream(stream)));
}

mxq_status mxq_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                          int64_t rows, int64_t cols, uint16_t* y, int64_t ld_y, void* stream) {
  const char* fn = "mxq_dequantize";
  if (rows < 0 || cols < 0) return fail(MXQ_ERR_INVALID_ARG, "%s: negative size", fn);
  if (cols % 32 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be a multiple of 32", fn, (long long)cols);
  if (ld_codes < cols / 2 || ld_scales < cols / 32 || ld_y < cols)
    return fail(MXQ_ERR_INVALID_ARG, "%s: pitch below the row width", fn);
  if (rows > kMaxDim || cols > kMaxDim || !pitch_ok(ld_codes) || !pitch_ok(ld_scales) || !pitch_ok(ld_y) ||
      rows * (cols / 32) >= ((int64_t)1 << 30))
    return fail(MXQ_ERR_INVALID_ARG, "%s: tensor too large", fn);
  if (rows > 0 && cols > 0) {
    if (!codes || !scales || !y) return fail(MXQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(codes, 4) || ld_codes % 4 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: codes must be 4-byte aligned", fn);
    if (!aligned(y, 16) || ld_y % 8 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: y base and pitch must be 16-byte aligned", fn);
  }
  return hip_status(fn, mxq::launch_dequantize(codes, ld_codes, scales, ld_scales, rows, cols, y, ld_y,
                                               as_stream(stream)));
}

mxq_status mxq_dequantize_fp8(const uint8_t* q, int64_t ld_q, float a_scale, int64_t rows, int64_t cols,
                              uint16_t* y, int64_t ld_y, void* stream) {
  const char* fn = "mxq_dequantize_fp8";
  if (rows < 0 || cols < 0) return fail(MXQ_ERR_INVALID_ARG, "%s: negative size", fn);
  if (cols % 16 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: cols (%lld) must be a multiple of 16", fn, (long long)cols);
  if (ld_q < cols || ld_y < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: pitch below the row width", fn);
  if (!(a_scale == a_scale) || a_scale == __builtin_inff() || a_scale == -__builtin_inff())
    return fail(MXQ_ERR_INVALID_ARG, "%s: a_scale must be finite", fn);
  if (rows > kMaxDim || cols > kMaxDim || !pitch_ok(ld_q) || !pitch_ok(ld_y) || rows * (cols / 8) >= ((int64_t)1 << 32))
    return fail(MXQ_ERR_INVALID_ARG, "%s: tensor too large", fn);
  if (rows > 0 && cols > 0) {
    if (!q || !y) return fail(MXQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(q, 16) || ld_q % 16 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: q base and ld_q must be multiples of 16 bytes", fn);
    if (!aligned(y, 16) || ld_y % 8 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: y base and pitch must be 16-byte aligned", fn);
  }
  return hip_status(fn, mxq::launch_dequantize_fp8(q, ld_q, a_scale, rows, cols, y, ld_y, as_stream(stream)));
}

mxq_status mxq_mfma_ceiling(mxq_gemm_mode mode, const void* a, const uint8_t* a_scales, const void* w,
                            const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, int64_t waves, int64_t iters,
                            float* sink, void* stream) {
  const char* fn = "mxq_mfma_ceiling";
  if (mode != MXQ_GEMM_W4A4 && mode != MXQ_GEMM_W4A8 && mode != MXQ_GEMM_BF16)
    return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown mode %d", fn, (int)mode);
  if (M < 1 || N < 1 || K < 32 || K % 32 != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: need M, N >= 1 and K a positive multiple of 32 (M=%lld N=%lld K=%lld)", fn,
                (long long)M, (long long)N, (long long)K);
  if (M > (int64_t)0x7FFFFFFF || N > (int64_t)0x7FFFFFFF || K > ((int64_t)1 << 21))
    return fail(MXQ_ERR_INVALID_ARG, "%s: dimension too large", fn);
  if (waves < 4 || waves % 4 != 0 || waves > ((int64_t)1 << 20))
    return fail(MXQ_ERR_INVALID_ARG, "%s: waves (%lld) must be a multiple of 4 in [4, 2^20]", fn, (long long)waves);
  if (iters < 1 || iters > ((int64_t)1 << 24))
    return fail(MXQ_ERR_INVALID_ARG, "%s: iters (%lld) must be in [1, 2^24]", fn, (long long)iters);
  mxq_status st;
  if ((st = check_operand(fn, "a", a, M, K, 16)) != MXQ_OK) return st;
  if ((st = check_operand(fn, "w", w, N, K, 16)) != MXQ_OK) return st;
  if (mode != MXQ_GEMM_BF16 && !w_scales) return fail(MXQ_ERR_INVALID_ARG, "%s: w_scales is NULL", fn);
  if (mode == MXQ_GEMM_W4A4 && !a_scales) return fail(MXQ_ERR_INVALID_ARG, "%s: a_scales is NULL", fn);
  if (!sink || !aligned(sink, 4)) return fail(MXQ_ERR_INVALID_ARG, "%s: sink must be a non-NULL 4-byte aligned pointer", fn);
  const mxq::GemmMode gm = mode == MXQ_GEMM_W4A4 ? mxq::GEMM_W4A4 : (mode == MXQ_GEMM_W4A8 ? mxq::GEMM_W4A8 : mxq::GEMM_BF16);
  return hip_status(fn, mxq::launch_mfma_ceiling(gm, a, a_scales, w, w_scales, M, N, K, waves, iters, sink,
                                                 as_stream(stream)));
}

mxq_status mxq_quantize_int8(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, int8_t* codes,
                             int64_t ld_codes, float* scales, void* stream) {
  const char* fn = "mxq_quantize_int8";
  mxq_status st = check_input(fn, x, dt, rows, cols, ld_x, 16);
  if (st != MXQ_OK) return st;
  if (ld_codes < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_codes (%lld) < cols", fn, (long long)ld_codes);
  if (!pitch_ok(ld_codes)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld_codes (%lld) must be below 2^32", fn, (long long)ld_codes);
  if (rows > 0 && cols > 0) {
    if (!codes) return fail(MXQ_ERR_INVALID_ARG, "%s: codes is NULL", fn);
    if (!aligned(codes, 16) || ld_codes % 16 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: codes base and ld_codes must be multiples of 16 bytes", fn);
  }
  if (rows > 0 && (!scales || !aligned(scales, 4)))
    return fail(MXQ_ERR_INVALID_ARG, "%s: scales must be a non-NULL 4-byte aligned pointer", fn);
  return hip_status(fn, mxq::launch_quantize_int8(x, dt == MXQ_F32, rows, cols, ld_x, codes, ld_codes, scales,
                                                  as_stream(stream)));
}

mxq_status mxq_dequantize_int8(const int8_t* codes, int64_t ld_codes, const float* scales, int64_t rows, int64_t cols,
                               uint16_t* y, int64_t ld_y, void* stream) {
  const char* fn = "mxq_dequantize_int8";
  if (rows < 0 || cols < 0 || cols % 8 != 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: cols must be a multiple of 8, sizes not negative", fn);
  if (ld_codes < cols || ld_y < cols) return fail(MXQ_ERR_INVALID_ARG, "%s: pitch below the row width", fn);
  if (rows > kMaxDim || cols > kMaxDim) return fail(MXQ_ERR_INVALID_ARG, "%s: dimension exceeds 2^31-1", fn);
  if (!pitch_ok(ld_codes) || !pitch_ok(ld_y)) return fail(MXQ_ERR_INVALID_ARG, "%s: pitch must be below 2^32", fn);
  if (rows * (cols / 8) >= ((int64_t)1 << 32))
    return fail(MXQ_ERR_INVALID_ARG, "%s: tensor too large (more than 2^35 elements)", fn);
  if (rows > 0 && cols > 0) {
    if (!codes || !scales || !y) return fail(MXQ_ERR_INVALID_ARG, "%s: codes/scales/y is NULL", fn);
    if (!aligned(codes, 8) || ld_codes % 8 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: codes base and ld_codes must be multiples of 8 bytes", fn);
    if (!aligned(scales, 4)) return fail(MXQ_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", fn);
    if (!aligned(y, 16) || ld_y % 8 != 0)
      return fail(MXQ_ERR_INVALID_ARG, "%s: y base and row pitch must be 16-byte aligned", fn);
  }
  return hip_status(fn, mxq::launch_dequantize_int8(codes, ld_codes, scales, rows, cols, y, ld_y, as_stream(stream)));
}

size_t mxq_gemm_w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!w8_shape_ok(M, N, K)) return 0;
  return mxq::gemm_w8a8_workspace_bytes(M, N, K);
}

mxq_status mxq_gemm_w8a8(const int8_t* a, int64_t ld_a, const float* a_scales, int64_t inc_as, const int8_t* w,
                         int64_t ld_w, const float* w_scales, int64_t inc_ws, const float* bias, int64_t M, int64_t N,
                         int64_t K, void* out, mxq_dtype out_dt, int64_t ld_out, void* workspace, size_t ws_bytes,
                         void* stream) {
  const char* fn = "mxq_gemm_w8a8";
  mxq_status st = check_w8(fn, w, ld_w, w_scales, inc_ws, bias, M, N, K, out, out_dt, ld_out);
  if (st != MXQ_OK) return st;
  if (ld_a < K || ld_a >= ((int64_t)1 << 23))
    return fail(MXQ_ERR_INVALID_ARG, "%s: ld_a (%lld) must be at least K and below 2^23", fn, (long long)ld_a);
  if (inc_as < 0 || !pitch_ok(inc_as)) return fail(MXQ_ERR_INVALID_ARG, "%s: inc_as out of range", fn);
  if (M > 0 && N > 0) {
    if (!a_scales || !aligned(a_scales, 4))
      return fail(MXQ_ERR_INVALID_ARG, "%s: a_scales must be a non-NULL 4-byte aligned pointer", fn);
    if (K > 0) {
      if (!a) return fail(MXQ_ERR_INVALID_ARG, "%s: a is NULL", fn);
      if (!aligned(a, 16) || ld_a % 16 != 0)
        return fail(MXQ_ERR_INVALID_ARG, "%s: a base and ld_a must be multiples of 16 bytes", fn);
    }
    if (workspace && (!aligned(workspace, 16) || ws_bytes < mxq_gemm_w8a8_workspace_bytes(M, N, K)))
      return fail(MXQ_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned and hold %llu bytes", fn,
                  (unsigned long long)mxq_gemm_w8a8_workspace_bytes(M, N, K));
  }
  return hip_status(fn, mxq::launch_gemm_w8a8(a, ld_a, a_scales, inc_as, w, ld_w, w_scales, inc_ws, bias, M, N, K, out,
                                              out_dt == MXQ_F32, ld_out, workspace, as_stream(stream)));
}

size_t mxq_gemm_w8a8_fused_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!w8_shape_ok(M, N, K) || mxq::gemm_w8a8_one_launch(M, K)) return 0;
  return fused_codes_bytes(M, K) + mxq::gemm_w8a8_workspace_bytes(M, N, K);
}

mxq_status mxq_gemm_w8a8_fused(const void* a, mxq_dtype dt, int64_t ld_a, const int8_t* w, int64_t ld_w,
                               const float* w_scales, int64_t inc_ws, const float* bias, int64_t M, int64_t N,
                               int64_t K, void* out, mxq_dtype out_dt, int64_t ld_out, void* workspace,
                               size_t ws_bytes, void* stream) {
  const char* fn = "mxq_gemm_w8a8_fused";
  mxq_status st = check_w8(fn, w, ld_w, w_scales, inc_ws, bias, M, N, K, out, out_dt, ld_out);
  if (st != MXQ_OK) return st;
  st = check_input(fn, a, dt, M, K, ld_a, 16);
  if (st != MXQ_OK) return st;
  if (M == 0 || N == 0) return ok();
  const size_t need = mxq_gemm_w8a8_fused_workspace_bytes(M, N, K);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || ws_bytes < need))
    return fail(MXQ_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned and hold %llu bytes", fn,
                (unsigned long long)need);
  if (need == 0)
    return hip_status(fn, mxq::launch_gemm_w8a8_unquantized(a, dt == MXQ_F32, ld_a, w, ld_w, w_scales, inc_ws, bias, M, N,
                                                            K, out, out_dt == MXQ_F32, ld_out, as_stream(stream)));
  int8_t* codes = static_cast<int8_t*>(workspace);
  const int64_t pitch = fused_pitch(K);
  float* scales = reinterpret_cast<float*>(codes + M * pitch);
  void* rest = mxq::gemm_w8a8_workspace_bytes(M, N, K) > 0 ? codes + fused_codes_bytes(M, K) : nullptr;
  hipError_t e = mxq::launch_quantize_int8(a, dt == MXQ_F32, M, K, ld_a, codes, pitch, scales, as_stream(stream));
  if (e == hipSuccess)
    e = mxq::launch_gemm_w8a8(codes, pitch, scales, 1, w, ld_w, w_scales, inc_ws, bias, M, N, K, out, out_dt == MXQ_F32,
                              ld_out, rest, as_stream(stream));
  return hip_status(fn, e);
}

mxq_status mxq_qk_norm_rope(const void* q, int64_t heads_q, int64_t ld_q, int64_t hs_q, const void* k, int64_t heads_k,
                            int64_t ld_k, int64_t hs_k, mxq_dtype dt, int64_t tokens, int64_t head_dim,
                            const void* w_q, const void* w_k, mxq_dtype w_dt, float eps, const float* cos,
                            const float* sin, int64_t ld_table, int64_t table_rows, int64_t rot_dim,
                            const int64_t* positions, mxq_rope_style style, void* out_q, int64_t ld_oq, int64_t hs_oq,
                            void* out_k, int64_t ld_ok, int64_t hs_ok, void* stream) {
  return qk_norm_rope("mxq_qk_norm_rope", HeadArgs{"q", q, heads_q, ld_q, hs_q, w_q, out_q, ld_oq, hs_oq, nullptr, 0},
                      HeadArgs{"k", k, heads_k, ld_k, hs_k, w_k, out_k, ld_ok, hs_ok, nullptr, 0}, dt, tokens, head_dim,
                      w_dt, eps, cos, sin, ld_table, table_rows, rot_dim, positions, style, false, as_stream(stream));
}

mxq_status mxq_quantize_qk_norm_rope(const void* q, int64_t heads_q, int64_t ld_q, int64_t hs_q, const void* k,
                                     int64_t heads_k, int64_t ld_k, int64_t hs_k, mxq_dtype dt, int64_t tokens,
                                     int64_t head_dim, const void* w_q, const void* w_k, mxq_dtype w_dt, float eps,
                                     const float* cos, const float* sin, int64_t ld_table, int64_t table_rows,
                                     int64_t rot_dim, const int64_t* positions, mxq_rope_style style, int8_t* codes_q,
                                     int64_t ld_cq, int64_t hs_cq, float* scales_q, int64_t ld_sq, int8_t* codes_k,
                                     int64_t ld_ck, int64_t hs_ck, float* scales_k, int64_t ld_sk, void* stream) {
  return qk_norm_rope("mxq_quantize_qk_norm_rope",
                      HeadArgs{"q", q, heads_q, ld_q, hs_q, w_q, codes_q, ld_cq, hs_cq, scales_q, ld_sq},
                      HeadArgs{"k", k, heads_k, ld_k, hs_k, w_k, codes_k, ld_ck, hs_ck, scales_k, ld_sk}, dt, tokens,
                      head_dim, w_dt, eps, cos, sin, ld_table, table_rows, rot_dim, positions, style, true,
                      as_stream(stream));
}

mxq_status mxq_layer_norm(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, const void* w,
                          const void* b, mxq_dtype w_dt, float eps, void* y, int64_t ld_y, float* mean, float* rstd,
                          int8_t* x_codes, int64_t ld_xc, float* x_scales, void* stream) {
  return layer_norm("mxq_layer_norm", x, dt, rows, cols, ld_x, w, b, w_dt, eps, y, ld_y, nullptr, mean, rstd, x_codes,
                    ld_xc, x_scales, false, as_stream(stream));
}

mxq_status mxq_quantize_layer_norm(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, const void* w,
                                   const void* b, mxq_dtype w_dt, float eps, int8_t* codes, int64_t ld_codes,
                                   float* scales, float* mean, float* rstd, int8_t* x_codes, int64_t ld_xc,
                                   float* x_scales, void* stream) {
  return layer_norm("mxq_quantize_layer_norm", x, dt, rows, cols, ld_x, w, b, w_dt, eps, codes, ld_codes, scales, mean,
                    rstd, x_codes, ld_xc, x_scales, true, as_stream(stream));
}

size_t mxq_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || rows > kMaxDim || cols < 8 || cols > mxq::kNormMaxCols || cols % 8 != 0) return 0;
  return mxq::layer_norm_backward_workspace_bytes(rows, cols);
}

mxq_status mxq_layer_norm_backward(const void* dy, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_dy,
                                   const void* x, int64_t ld_x, const float* x_scales, const float* mean,
                                   const float* rstd, const void* w, mxq_dtype w_dt, void* dx, int64_t ld_dx, float* dw,
                                   float* db, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "mxq_layer_norm_backward";
  const bool codes = x_scales != nullptr;
  mxq_status st = check_input(fn, dy, dt, rows, cols, ld_dy, codes ? 16 : 8);
  if (st != MXQ_OK) return st;
  if ((st = check_norm(fn, cols, w, nullptr, w_dt)) != MXQ_OK) return st;
  if ((st = check_plane(fn, "x", x, rows, cols, ld_x, codes ? 1 : dtype_bytes(dt), 16)) != MXQ_OK) return st;
  if ((st = check_plane(fn, "dx", dx, rows, cols, ld_dx, dtype_bytes(dt), 16)) != MXQ_OK) return st;
  if ((st = check_row_values(fn, "x_scales", x_scales, rows, true)) != MXQ_OK) return st;
  if ((st = check_row_values(fn, "mean", mean, rows, false)) != MXQ_OK) return st;
  if ((st = check_row_values(fn, "rstd", rstd, rows, false)) != MXQ_OK) return st;
  if (!dw != !db) return fail(MXQ_ERR_INVALID_ARG, "%s: dw and db must be given together", fn);
  if (!aligned(dw, 16) || !aligned(db, 16)) return fail(MXQ_ERR_INVALID_ARG, "%s: dw and db must be 16-byte aligned", fn);
  const size_t need = dw ? mxq_layer_norm_backward_workspace_bytes(rows, cols) : 0;
  if (need > 0 && (!workspace || !aligned(workspace, 16) || ws_bytes < need))
    return fail(MXQ_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned and hold %llu bytes", fn, (unsigned long long)need);
  mxq::NormGradParams p;
  p.dy = dy;
  p.x = x;
  p.x_scales = x_scales;
  p.mean = mean;
  p.rstd = rstd;
  p.w = w;
  p.dx = dx;
  p.dw = dw;
  p.db = db;
  p.part = static_cast<float*>(workspace);
  p.rows = rows;
  p.ld_dy = ld_dy;
  p.ld_x = ld_x;
  p.ld_dx = ld_dx;
  p.units = (uint32_t)(cols / 8);
  p.w_f32 = w_dt == MXQ_F32 ? 1 : 0;
  p.inv_cols = 1.0f / (float)cols;
  return hip_status(fn, mxq::launch_layer_norm_backward(p, dt == MXQ_F32, codes, as_stream(stream)));
}

mxq_status mxq_activation(const void* u, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_u, mxq_activation_kind act,
                          void* y, int64_t ld_y, int8_t* u_codes, int64_t ld_uc, float* u_scales, void* stream) {
  return activation("mxq_activation", u, dt, rows, cols, ld_u, act, y, ld_y, nullptr, u_codes, ld_uc, u_scales, false,
                    as_stream(stream));
}

mxq_status mxq_quantize_activation(const void* u, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_u,
                                   mxq_activation_kind act, int8_t* codes, int64_t ld_codes, float* scales,
                                   int8_t* u_codes, int64_t ld_uc, float* u_scales, void* stream) {
  return activation("mxq_quantize_activation", u, dt, rows, cols, ld_u, act, codes, ld_codes, scales, u_codes, ld_uc,
                    u_scales, true, as_stream(stream));
}

mxq_status mxq_activation_backward(const void* dy, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_dy,
                                   const int8_t* u_codes, int64_t ld_uc, const float* u_scales, mxq_activation_kind act,
                                   void* du, int64_t ld_du, void* stream) {
  const char* fn = "mxq_activation_backward";
  mxq_status st = check_act(fn, act);
  if (st != MXQ_OK) return st;
  if ((st = check_input(fn, dy, dt, rows, cols, ld_dy, 16)) != MXQ_OK) return st;
  if ((st = check_plane(fn, "u_codes", u_codes, rows, cols, ld_uc, 1, 16)) != MXQ_OK) return st;
  if ((st = check_plane(fn, "du", du, rows, cols, ld_du, dtype_bytes(dt), 16)) != MXQ_OK) return st;
  if ((st = check_row_values(fn, "u_scales", u_scales, rows, false)) != MXQ_OK) return st;
  mxq::ActGradParams p;
  p.dy = dy;
  p.kept = u_codes;
  p.kept_scales = u_scales;
  p.dx = du;
  p.ld_dy = ld_dy;
  p.ld_kept = ld_uc;
  p.ld_dx = ld_du;
  p.units = (uint32_t)(cols / 8);
  p.total = (uint32_t)(rows * (cols / 8));
  return hip_status(fn, mxq::launch_activation_backward(
                            p, dt == MXQ_F32, act == MXQ_ACT_GELU_TANH ? mxq::ACT_GELU_TANH : mxq::ACT_SILU, as_stream(stream)));
}

size_t mxq_grad_weight_int8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return grad_shape_ok(M, N, K) ? mxq::grad_weight_workspace_bytes(M, N, K) : 0;
}

mxq_status mxq_grad_weight_int8(const uint16_t* dy, int64_t ld_dy, const int8_t* codes, int64_t ld_codes,
                                const float* scales, int64_t M, int64_t N, int64_t K, void* out, mxq_dtype out_dt,
                                int64_t ld_out, int accumulate, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "mxq_grad_weight_int8";
  const int ob = dtype_bytes(out_dt);
  if (ob == 0) return fail(MXQ_ERR_UNSUPPORTED, "%s: unknown output dtype %d", fn, (int)out_dt);
  if (M < 0 || N < 0 || K < 0)
    return fail(MXQ_ERR_INVALID_ARG, "%s: negative size (M=%lld N=%lld K=%lld)", fn, (long long)M, (long long)N, (long long)K);
  if (N % 8 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: N (%lld) must be a multiple of 8", fn, (long long)N);
  if (K % 16 != 0) return fail(MXQ_ERR_INVALID_ARG, "%s: K (%lld) must be a multiple of 16", fn, (long long)K);
  if (N > 0 && K > 0 && !grad_shape_ok(M, N, K)) return fail(MXQ_ERR_INVALID_ARG, "%s: problem too large", fn);
  if (ld_dy >= ((int64_t)1 << 23)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld of dy (%lld) must be below 2^23", fn, (long long)ld_dy);
  if (ld_codes >= ((int64_t)1 << 23)) return fail(MXQ_ERR_INVALID_ARG, "%s: ld of codes (%lld) must be below 2^23", fn, (long long)ld_codes);
  mxq_status st = check_plane(fn, "dy", dy, K > 0 ? M : 0, N, ld_dy, 2, 16);
  if (st != MXQ_OK) return st;
  if ((st = check_plane(fn, "codes", codes, N > 0 ? M : 0, K, ld_codes, 1, 16)) != MXQ_OK) return st;
  if ((st = check_plane(fn, "out", out, N, K, ld_out, ob, ob)) != MXQ_OK) return st;
  if (N == 0 || K == 0) return ok();
  if ((st = check_row_values(fn, "scales", scales, M, false)) != MXQ_OK) return st;
  const size_t need = mxq_grad_weight_int8_workspace_bytes(M, N, K);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || ws_bytes < need))
    return fail(MXQ_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned and hold %llu bytes", fn, (unsigned long long)need);
  return hip_status(fn, mxq::launch_grad_weight_int8(dy, ld_dy, codes, ld_codes, scales, M, N, K, out, out_dt == MXQ_F32,
                                                     ld_out, accumulate != 0, workspace, as_stream(stream)));
}

}  // extern "C"
