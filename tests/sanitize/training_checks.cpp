// Host driver for a sanitizer build of the C-ABI validation layer: layer norm, activation and weight gradient
// with sizes and pitches up to the int64 limits, unknown enums, the workspace sizes (and with them the plan of the
// weight gradient) over all sizes, and empty problems.  Nothing here reaches a GPU.  Exit status 0 when every call
// returned what it should; the sanitizers abort on the first report.
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
const int64_t ODD[] = {BIG, NEG, -1, int64_t{1} << 40, int64_t{1} << 32, int64_t{1} << 31, BIG - 15, BIG / 16 * 16};

}  // namespace

int main() {
  auto* i8 = static_cast<int8_t*>(P16);
  auto* u16 = static_cast<uint16_t*>(P16);
  auto* f = static_cast<float*>(P16);
  const size_t plenty = size_t{1} << 40;
  for (int64_t v : ODD) {
    auto norm = [&](int64_t T, int64_t C, int64_t ld, int64_t ldy, int64_t ldk) {
      return mxq_layer_norm(P16, MXQ_BF16, T, C, ld, P16, P16, MXQ_F32, 1e-6f, P16, ldy, f, f, i8, ldk, f, nullptr);
    };
    expect("norm rows", norm(v, 64, 64, 64, 32), false);
    expect("norm cols", norm(4, v, 64, 64, 64), false);
    if (v < 64 || v > int64_t{1} << 32) {
      expect("norm ld", norm(4, 64, v, 64, 64), false);
      expect("norm ldy", norm(4, 64, 64, v, 64), false);
      expect("norm ldk", norm(4, 64, 64, 64, v), false);
    }
    expect("norm8 rows", mxq_quantize_layer_norm(P16, MXQ_F32, v, 64, 64, P16, P16, MXQ_BF16, 0.0f, i8, 32, f, f, f, nullptr, 0, nullptr, nullptr), false);
    expect("norm8 cols", mxq_quantize_layer_norm(P16, MXQ_F32, 4, v, 64, P16, P16, MXQ_BF16, 0.0f, i8, 64, f, f, f, nullptr, 0, nullptr, nullptr), false);
    auto back = [&](int64_t T, int64_t C, int64_t ld, int64_t ldx, int64_t ldd) {
      return mxq_layer_norm_backward(P16, MXQ_F32, T, C, ld, P16, ldx, f, f, f, P16, MXQ_F32, P16, ldd, f, f, P16, plenty, nullptr);
    };
    expect("back rows", back(v, 64, 64, 32, 64), false);
    expect("back cols", back(4, v, 64, 64, 64), false);
    if (v < 64 || v > int64_t{1} << 32) {
      expect("back ld", back(4, 64, v, 64, 64), false);
      expect("back ldx", back(4, 64, 64, v, 64), false);
      expect("back ldd", back(4, 64, 64, 64, v), false);
    }
    expect("act rows", mxq_activation(P16, MXQ_F32, v, 64, 64, MXQ_ACT_SILU, P16, 32, i8, 64, f, nullptr), false);
    expect("act cols", mxq_activation(P16, MXQ_F32, 4, v, 64, MXQ_ACT_SILU, P16, 64, i8, 64, f, nullptr), false);
    expect("act8 rows", mxq_quantize_activation(P16, MXQ_BF16, v, 64, 64, MXQ_ACT_GELU_TANH, i8, 32, f, nullptr, 0, nullptr, nullptr), false);
    expect("act back rows", mxq_activation_backward(P16, MXQ_BF16, v, 64, 64, i8, 32, f, MXQ_ACT_SILU, P16, 64, nullptr), false);
    expect("act back cols", mxq_activation_backward(P16, MXQ_BF16, 4, v, 64, i8, 64, f, MXQ_ACT_SILU, P16, 64, nullptr), false);
    auto grad = [&](int64_t M, int64_t N, int64_t K, int64_t ldy, int64_t ldc, int64_t ldo) {
      return mxq_grad_weight_int8(u16, ldy, i8, ldc, f, M, N, K, P16, MXQ_F32, ldo, 1, P16, plenty, nullptr);
    };
    expect("grad M", grad(v, 64, 64, 32, 64, 64), false);
    expect("grad N", grad(4, v, 64, 64, 64, 64), false);
    expect("grad K", grad(4, 64, v, 64, 64, 64), false);
    expect("grad ldy", grad(4, 64, 64, v, 64, 64), false);
    expect("grad ldc", grad(4, 64, 64, 64, v, 64), false);
    if (v < 64 || v > int64_t{1} << 32) expect("grad ldo", grad(4, 64, 64, 64, 64, v), false);
    for (int64_t w : ODD) {
      ++checks;
      if (mxq_layer_norm_backward_workspace_bytes(v, w) != 0 || mxq_grad_weight_int8_workspace_bytes(64, v, w) != 0 ||
          mxq_grad_weight_int8_workspace_bytes(v, w, 64) != 0)
        ++failures;
    }
  }
  expect("eps", mxq_layer_norm(P16, MXQ_BF16, 4, 64, 64, P16, P16, MXQ_F32, NAN, P16, 64, f, f, nullptr, 0, nullptr, nullptr), false);
  expect("act", mxq_activation(P16, MXQ_F32, 4, 64, 64, (mxq_activation_kind)7, P16, 64, nullptr, 0, nullptr, nullptr), false);
  expect("dtype", mxq_grad_weight_int8(u16, 64, i8, 64, f, 4, 64, 64, P16, (mxq_dtype)4, 64, 0, P16, plenty, nullptr), false);
  // plans of every size, the smallest and the largest: host arithmetic only.  Parts of M never take more than
  // 300 MB beside the widened codes (four rounds of the largest tile are 256).
  for (int64_t M = 1; M < (int64_t{1} << 31) - 256; M = M * 3 + 1)
    for (int64_t N = 8; N <= int64_t{1} << 22; N = N / 8 * 24 + 8)
      for (int64_t K = 16; K <= int64_t{1} << 22; K = K / 16 * 64 + 16) {
        ++checks;
        const uint64_t got = mxq_grad_weight_int8_workspace_bytes(M, N, K);
        if (got > 2 * (uint64_t)M * (uint64_t)K + 256 + (uint64_t{300} << 20)) {
          ++failures;
          printf("FAIL plan %lld %lld %lld: %llu\n", (long long)M, (long long)N, (long long)K, (unsigned long long)got);
        }
      }
  for (int64_t T = 1; T < int64_t{1} << 31; T = T * 2 + 1)
    for (int64_t C = 8; C <= 16384; C += 8) {
      ++checks;
      if (mxq_layer_norm_backward_workspace_bytes(T, C) > (uint64_t)8 * C * 8192) ++failures;
    }
  expect("empty norm", mxq_layer_norm(nullptr, MXQ_BF16, 0, 64, 64, nullptr, nullptr, MXQ_F32, 0.0f, nullptr, 64, nullptr, nullptr, nullptr, 0, nullptr, nullptr), true);
  expect("empty act", mxq_activation(nullptr, MXQ_BF16, 0, 64, 64, MXQ_ACT_SILU, nullptr, 64, nullptr, 0, nullptr, nullptr), true);
  expect("empty grad", mxq_grad_weight_int8(nullptr, 0, nullptr, 64, nullptr, 4, 0, 64, nullptr, MXQ_F32, 64, 0, nullptr, 0, nullptr), true);
  printf("%d checks, %d failures\n", checks, failures);
  return failures ? 1 : 0;
}
