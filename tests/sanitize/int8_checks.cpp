// Host driver for a sanitizer build of the C-ABI validation layer: the 8-bit entry points
// with sizes and pitches up to the int64 limits, NULL and misaligned pointers, unknown
// enums, the workspace sizes and empty problems.  Nothing here reaches a GPU.  Exit status 0
// when every call returned what it should; the sanitizers abort on the first report.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/mxq.h"

namespace {

int failures = 0, checks = 0;
void* const P16 = reinterpret_cast<void*>(uintptr_t{1} << 20);   // never dereferenced

void expect(const char* what, mxq_status got, bool want_ok) {
  ++checks;
  const char* msg = mxq_last_error();
  if (want_ok ? (got == MXQ_OK && msg[0] == '\0') : (got != MXQ_OK && msg[0] != '\0')) return;
  ++failures;
  printf("FAIL %s: status %d, message '%s'\n", what, (int)got, msg);
}

const int64_t BIG = INT64_MAX, NEG = INT64_MIN;
const int64_t KS[] = {0, 16, 13824, 131056};
const int64_t ODD[] = {BIG, NEG, -1, int64_t{1} << 40, int64_t{1} << 32, int64_t{1} << 31, BIG - 15, BIG / 16 * 16};

}  // namespace

int main() {
  auto* i8 = static_cast<int8_t*>(P16);
  auto* u16 = static_cast<uint16_t*>(P16);
  auto* f = static_cast<float*>(P16);
  auto* i64 = static_cast<int64_t*>(P16);
  for (int64_t v : ODD) {
    expect("quantize rows", mxq_quantize_int8(P16, MXQ_BF16, v, 64, 64, i8, 32, f, nullptr), false);
    expect("quantize cols", mxq_quantize_int8(P16, MXQ_F32, 4, v, 64, i8, 64, f, nullptr), false);
    if (v < 64) expect("quantize ld", mxq_quantize_int8(P16, MXQ_F32, 4, 64, v, i8, 64, f, nullptr), false);
    if (v < 64 || v > (int64_t{1} << 32)) expect("quantize ldc", mxq_quantize_int8(P16, MXQ_F32, 4, 64, 64, i8, v, f, nullptr), false);
    expect("dequantize rows", mxq_dequantize_int8(i8, 64, f, v, 64, u16, 32, nullptr), false);
    expect("dequantize cols", mxq_dequantize_int8(i8, 64, f, 4, v, u16, 64, nullptr), false);
    expect("gemm M", mxq_gemm_w8a8(i8, 64, f, 1, i8, 64, f, 1, nullptr, v, 8, 64, P16, MXQ_BF16, 4, nullptr, 0, nullptr), false);
    expect("gemm N", mxq_gemm_w8a8(i8, 64, f, 1, i8, 64, f, 1, nullptr, 8, v, 64, P16, MXQ_BF16, 64, nullptr, 0, nullptr), false);
    expect("gemm K", mxq_gemm_w8a8(i8, 64, f, 1, i8, 64, f, 1, nullptr, 8, 8, v, P16, MXQ_F32, 8, nullptr, 0, nullptr), false);
    expect("gemm ld", mxq_gemm_w8a8(i8, v, f, 1, i8, 64, f, 1, nullptr, 8, 8, 64, P16, MXQ_F32, 8, nullptr, 0, nullptr), false);
    if (v < 0 || v > (int64_t{1} << 32) - 1)
      expect("gemm inc", mxq_gemm_w8a8(i8, 64, f, v, i8, 64, f, 1, nullptr, 8, 8, 64, P16, MXQ_F32, 8, nullptr, 0, nullptr), false);
    expect("fused M", mxq_gemm_w8a8_fused(P16, MXQ_BF16, 64, i8, 64, f, 1, nullptr, v, 8, 64, P16, MXQ_BF16, 4, nullptr, 0, nullptr), false);
    expect("fused K", mxq_gemm_w8a8_fused(P16, MXQ_BF16, 64, i8, 64, f, 1, nullptr, 8, 8, v, P16, MXQ_BF16, 8, nullptr, 0, nullptr), false);
    for (int64_t w : ODD) {
      ++checks;
      if ((v < 0 || w < 0 || v > 0x7FFFFFFF || w > 0x7FFFFFFF) &&
          (mxq_gemm_w8a8_workspace_bytes(v, w, 64) != 0 || mxq_gemm_w8a8_fused_workspace_bytes(v, w, 64) != 0))
        ++failures;
    }
    auto qk = [&](int64_t T, int64_t H, int64_t D, int64_t ld, int64_t hs, int64_t ldt, int64_t rows, int64_t R, int64_t lo, int64_t ho) {
      return mxq_qk_norm_rope(P16, H, ld, hs, P16, 1, 64, 64, MXQ_BF16, T, D, nullptr, nullptr, MXQ_F32, 1e-6f, f, f, ldt, rows, R,
                              i64, MXQ_ROPE_HALVES, P16, lo, ho, P16, 64, 64, nullptr);
    };
    expect("qk tokens", qk(v, 2, 64, 128, 64, 32, 4, 64, 32, 64), false);
    expect("qk heads", qk(4, v, 64, 128, 64, 32, 4, 64, 128, 64), false);
    expect("qk dim", qk(4, 2, v, 128, 64, 32, 4, 64, 128, 64), false);
    if (v < 0 || v > (int64_t{1} << 32)) expect("qk ld", qk(4, 2, 64, v, 64, 32, 4, 64, 128, 64), false);
    expect("qk hs", qk(4, 2, 64, 128, v, 32, 4, 64, 128, 64), false);
    if (v < 0 || v > (int64_t{1} << 32)) expect("qk ldt", qk(4, 2, 64, 128, 64, v, 4, 64, 128, 64), false);
    if (v < 0 || v > (int64_t{1} << 31)) expect("qk rows", qk(4, 2, 64, 128, 64, 32, v, 64, 128, 64), false);
    expect("qk rot", qk(4, 2, 64, 128, 64, 32, 4, v, 128, 64), false);
    expect("qk out hs", qk(4, 2, 64, 128, 64, 32, 4, 64, 128, v), false);
    expect("qk quant", mxq_quantize_qk_norm_rope(P16, 2, 128, 64, P16, 1, 64, 64, MXQ_F32, 4, 64, nullptr, nullptr, MXQ_F32, 1e-6f, f, f,
                                                 32, 4, 64, i64, MXQ_ROPE_INTERLEAVED, i8, 128, v, f, 2, i8, 64, 64, f, 1, nullptr), false);
  }
  expect("qk eps", mxq_qk_norm_rope(P16, 1, 64, 64, P16, 1, 64, 64, MXQ_BF16, 4, 64, nullptr, nullptr, MXQ_F32, NAN, f, f, 32, 4, 64,
                                    i64, MXQ_ROPE_HALVES, P16, 64, 64, P16, 64, 64, nullptr), false);
  expect("style", mxq_qk_norm_rope(P16, 1, 64, 64, P16, 1, 64, 64, MXQ_BF16, 4, 64, nullptr, nullptr, MXQ_F32, 0, f, f, 32, 4, 64,
                                   i64, (mxq_rope_style)9, P16, 64, 64, P16, 64, 64, nullptr), false);
  expect("dtype", mxq_gemm_w8a8(i8, 64, f, 1, i8, 64, f, 1, nullptr, 8, 8, 64, P16, (mxq_dtype)4, 8, nullptr, 0, nullptr), false);
  // plans of every size, the smallest and the largest: host arithmetic only
  for (int64_t M = 1; M < (int64_t{1} << 31) - 256; M = M * 3 + 1)
    for (int64_t N = 1; N < (int64_t{1} << 31) - 256; N = N * 5 + 2)
      for (int64_t K : KS) {
        ++checks;
        if (mxq_gemm_w8a8_workspace_bytes(M, N, K) > (uint64_t{1} << 40)) ++failures;
        (void)mxq_gemm_w8a8_fused_workspace_bytes(M, N, K);
      }
  expect("empty quantize", mxq_quantize_int8(nullptr, MXQ_BF16, 0, 64, 64, nullptr, 64, nullptr, nullptr), true);
  expect("empty gemm", mxq_gemm_w8a8(nullptr, 64, nullptr, 0, nullptr, 64, nullptr, 0, nullptr, 0, 8, 64, nullptr, MXQ_F32, 8, nullptr, 0, nullptr), true);
  printf("%d checks, %d failures\n", checks, failures);
  return failures ? 1 : 0;
}
