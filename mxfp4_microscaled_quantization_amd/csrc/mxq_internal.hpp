// Internal launcher interface between the C ABI layer (mxq_api.hip) and the kernels.
// Launchers assume validated arguments, enqueue on `stream`, and return the HIP error
// of the launch (hipSuccess when nothing needed launching).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

hipError_t launch_quantize_mxfp4(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld_x,
                                 uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                                 bool uos, hipStream_t stream);
hipError_t launch_quantize_mxfp4_rotated(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld_x, int n,
                                         uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                                         bool uos, hipStream_t stream);
hipError_t launch_quantize_fp8(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld_x,
                               float inv_scale, uint8_t* q, int64_t ld_q, hipStream_t stream);
hipError_t launch_absmax(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld_x, float* out,
                         hipStream_t stream);
hipError_t launch_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales,
                             int64_t ld_scales, int64_t rows, int64_t cols, uint16_t* y, int64_t ld_y,
                             hipStream_t stream);
hipError_t launch_dequantize_fp8(const uint8_t* q, int64_t ld_q, float a_scale, int64_t rows, int64_t cols,
                                 uint16_t* y, int64_t ld_y, hipStream_t stream);

enum GemmMode { GEMM_W4A4 = 0, GEMM_W4A8 = 1, GEMM_BF16 = 2 };
hipError_t launch_gemm(GemmMode mode, const void* a, const uint8_t* a_scales, const void* w,
                       const uint8_t* w_scales, float a_scale, int64_t M, int64_t N, int64_t K,
                       uint16_t* out, int64_t ld_out, hipStream_t stream);

// W4A4 with the activation quantization fused in: `a` is rows x K of bf16 (or binary32),
// pitch ld_a elements; uos selects the UOS scale rule.
hipError_t launch_gemm_w4a4_fused(const void* a, bool f32, int64_t ld_a, const uint8_t* w, const uint8_t* w_scales,
                                  int64_t M, int64_t N, int64_t K, bool uos, uint16_t* out, int64_t ld_out,
                                  hipStream_t stream);

// Register-only MFMA loop on fragments gathered from a GEMM call's operand planes
// (waves a multiple of 4; sink: one float per lane).
hipError_t launch_mfma_ceiling(GemmMode mode, const void* a, const uint8_t* a_scales, const void* w,
                               const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, int64_t waves, int64_t iters,
                               float* sink, hipStream_t stream);

// 8-bit row quantization and dequantization (int8.hip).
hipError_t launch_quantize_int8(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld_x, int8_t* codes,
                                int64_t ld_codes, float* scales, hipStream_t stream);
hipError_t launch_dequantize_int8(const int8_t* codes, int64_t ld_codes, const float* scales, int64_t rows,
                                  int64_t cols, uint16_t* y, int64_t ld_y, hipStream_t stream);

// 8-bit product with token and channel scales (gemm_int8.hip); inc_*: elements between
// consecutive scales; bias may be null.  workspace: gemm_w8a8_workspace_bytes, or null (K is
// then not split; the same bits).
size_t gemm_w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_w8a8(const int8_t* a, int64_t ld_a, const float* a_scales, int64_t inc_as, const int8_t* w,
                            int64_t ld_w, const float* w_scales, int64_t inc_ws, const float* bias, int64_t M,
                            int64_t N, int64_t K, void* out, bool f32_out, int64_t ld_out, void* workspace,
                            hipStream_t stream);

// The same from unquantized activations in one launch, where gemm_w8a8_one_launch (M, N > 0).
bool gemm_w8a8_one_launch(int64_t M, int64_t K);
hipError_t launch_gemm_w8a8_unquantized(const void* x, bool f32, int64_t ld_x, const int8_t* w, int64_t ld_w,
                                        const float* w_scales, int64_t inc_ws, const float* bias, int64_t M, int64_t N,
                                        int64_t K, void* out, bool f32_out, int64_t ld_out, hipStream_t stream);

// Norm and rotation of query and key heads (qk_norm.hip).  Pitches in elements of the
// tensor they belong to: ld_* between tokens, hs_* between heads.
struct QkSide {
  const void* x;
  const void* w;      // head_dim weights, or null for 1
  void* out;          // the input's type, or int8 codes
  float* scales;      // of the codes
  int64_t ld_x, hs_x, ld_o, hs_o, ld_s;
  int heads;
};
struct QkNormParams {
  QkSide q, k;
  int64_t tokens, ld_table, table_rows;
  const float *cos, *sin;
  const int64_t* positions;   // or null: token t has position t
  int head_dim, rot_dim, w_f32;
  int runs_q;                 // workgroups (blockIdx.y, or .x for pairs) below it: queries
  float eps, inv_dim;
};
hipError_t launch_qk_norm_rope(const QkNormParams& p, bool f32, bool quant, bool halves, hipStream_t stream);

// Layer norm and its gradient (layer_norm.hip).  units: columns / 8; pitches in elements of
// the tensor they belong to.
struct NormParams {
  const void* x;
  const void *w, *b;       // weights and biases of one type, either may be null
  void* y;                 // the input's type, or int8 codes
  float* scales;           // of the codes
  float *mean, *rstd;      // or both null
  int8_t* kept;            // codes of x, or null
  float* kept_scales;
  int64_t rows, ld_x, ld_y, ld_kept;
  uint32_t units;
  int w_f32;
  int past;                // loads and stores past the caches (set by the launcher)
  float eps, cols, inv_cols;
};
hipError_t launch_layer_norm(const NormParams& p, bool f32, bool quant, hipStream_t stream);

constexpr int kNormThreads = 1024;   // of the gradient's largest workgroup, with up to 2 units each
constexpr int64_t kNormMaxCols = 8 * 2 * kNormThreads;
struct NormGradParams {
  const void *dy, *x;      // x: of dy's type, or int8 codes
  const float *x_scales, *mean, *rstd;
  const void* w;           // or null
  void* dx;
  float *dw, *db;          // or both null
  float* part;             // sums of the workgroups
  int64_t rows, ld_dy, ld_x, ld_dx;
  uint32_t units;
  int w_f32;
  float inv_cols;
};
size_t layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols);
hipError_t launch_layer_norm_backward(const NormGradParams& p, bool f32, bool codes, hipStream_t stream);

// The feed-forward activation, its 8-bit checkpoint and its gradient (activation.hip).
enum ActKind { ACT_GELU_TANH = 0, ACT_SILU = 1 };
constexpr int64_t kActMaxCols = 8 * 8 * 1024;   // of the forward pass
struct ActParams {
  const void* u;
  void* y;                 // the input's type, or int8 codes
  float* scales;           // of the codes
  int8_t* kept;            // checkpoint, or null
  float* kept_scales;
  int64_t rows, ld_u, ld_y, ld_kept;
  uint32_t units;
};
hipError_t launch_activation(const ActParams& p, bool f32, bool quant, ActKind act, hipStream_t stream);
struct ActGradParams {
  const void* dy;
  const int8_t* kept;
  const float* kept_scales;
  void* dx;
  int64_t ld_dy, ld_kept, ld_dx;
  uint32_t units, total;   // of a row, of all rows
};
hipError_t launch_activation_backward(const ActGradParams& p, bool f32, ActKind act, hipStream_t stream);

// Weight gradient of the 8-bit product (grad_weight.hip): out (+)= dy^T * bf16(code * scale).
size_t grad_weight_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_grad_weight_int8(const uint16_t* dy, int64_t ld_dy, const int8_t* codes, int64_t ld_codes,
                                   const float* scales, int64_t M, int64_t N, int64_t K, void* out, bool f32_out,
                                   int64_t ld_out, bool accumulate, void* workspace, hipStream_t stream);

size_t sqnr_workspace_bytes(int64_t n);
// The library's own SQNR workspace on the current device (a static device array,
// sqnr_scratch_bytes() long): its device address, looked up once per device.
size_t sqnr_scratch_bytes();
hipError_t sqnr_scratch(void** ptr);
hipError_t launch_sqnr(const uint16_t* ref, const uint16_t* test, int64_t rows, int64_t cols,
                       int64_t ld_ref, int64_t ld_test, void* ws, double* out3, hipStream_t stream);

}  // namespace mxq
