/*
 * mxq.h -- C ABI of libmxq: OCP MXFP4 block quantization and the W4A4 / W4A8 GEMMs that
 * consume it, with a bf16 reference GEMM and whole-output SQNR; 8-bit products and the operators
 * between them, with backward passes from activations kept in 8 bits; for AMD Instinct MI355X
 * (gfx950).
 *
 * Sources (web pages, cited by title and section):
 *  [Q13] "AMD Quark adds native W4A8 mixed-precision for Wan2.2 video generation on
 *        MI350", section "Quark quantization pipeline and mixed-precision selection":
 *        MXFP4 weights in both modes; dynamic MXFP4 activations for W4A4; static FP8
 *        E4M3 activations for W4A8; BF16 is the quality ceiling; blocks are scored by
 *        the SQNR of their whole output against BF16.
 *  [FLX] "AMD Quark: 1.92x faster FLUX.1-dev with MXFP4 on Instinct MI350", sections
 *        "MXFP4 quantization for diffusion models" and "What is MXFP4": 4-bit
 *        elements; 32-element blocks sharing one scale; the GEMM consumes MXFP4 inputs
 *        directly, with no dequantization phase.
 *  [MXA] "MXAttention: Data-Free Optimal Scaling and Pre-Normalization Quantization for
 *        MXFP4 Attention", section "What it actually does": the shared scale is an
 *        E8M0 power of two with no mantissa.
 *  [ORK] "Exp 2026-08-22 W4A4 Reference Model", section "Status": a linear per-group
 *        scale factors out of each group's partial sum and is applied in the fp32 drain.
 *  Format details the pages leave open follow OCP Microscaling Formats v1.0: E2M1
 *  elements (values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives), E8M0 bias 127, OCP FP8
 *  E4M3 (max 448).
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers (HBM) owned by the caller; the library never
 *    allocates, frees or retains them.  Scalars are passed by value.  The one
 *    host-visible result (mxq_sqnr's three doubles) is written to device memory.  The
 *    exception is mxq_fp8_static_scales, a host computation on host pointers.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Every call only enqueues
 *    work on it and returns; nothing synchronizes.  Device-side faults surface at the
 *    caller's next synchronization.
 *  - Return value: MXQ_OK, or an error code with a message available from
 *    mxq_last_error() on the same thread.  Arguments are validated before anything is
 *    launched: an error return means nothing was enqueued.  MXQ_ERR_HIP reports a HIP
 *    launch error (e.g. no device present).
 *  - Empty problems (rows == 0, M == 0 or N == 0) are valid and enqueue nothing.
 *  - Sizes: dimensions below 2^31, row pitches (ld_*) below 2^32 elements, so every
 *    offset the library forms fits in int64; larger values are MXQ_ERR_INVALID_ARG.
 *  - Layouts (all row-major):
 *      MXFP4 codes  : uint8 [rows x ld_codes], byte j of a row holds element 2j in the
 *                     low nibble and element 2j+1 in the high nibble; an E2M1 code is
 *                     sign<<3 | exponent(2 bits, bias 1)<<1 | mantissa(1 bit).
 *      MXFP4 scales : uint8 [rows x ld_scales], one E8M0 byte per 32-element block
 *                     along the row; value 2^(byte - 127).
 *      FP8          : uint8 [rows x ld], OCP E4M3.
 *      int8         : two's complement codes, one binary32 scale for each row.
 *      bf16         : uint16 bit patterns.
 *    The quantizer's output is exactly the GEMMs' input: there is no hidden reshuffle.
 *    GEMM weights W are N x K with K contiguous (nn.Linear layout); out = A * W^T.
 *  - Thread safety: no global mutable state except the thread-local error message and
 *    the per-GPU scratch of mxq_sqnr_noalloc (calls of it that overlap on one GPU race).
 */
#ifndef MXQ_H
#define MXQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* 2: mxq_gemm_w4a4_fused takes a workspace; mxq_gemm_w4a4_fused_workspace_bytes */
#define MXQ_ABI_VERSION 2

typedef enum {
  MXQ_OK = 0,
  MXQ_ERR_INVALID_ARG = 1, /* bad size, pointer, alignment or leading dimension */
  MXQ_ERR_UNSUPPORTED = 2, /* well-formed request the library does not serve (e.g. unknown dtype) */
  MXQ_ERR_HIP = 3,         /* a HIP runtime call or kernel launch failed */
  MXQ_STATUS_MAX_ENUM = 0x7FFFFFFF
} mxq_status;

/* Every enum ends in a *_MAX_ENUM member so that it spans all int32 values: an unknown
 * value passed in is then a defined value the library rejects (MXQ_ERR_UNSUPPORTED). */
typedef enum { MXQ_F32 = 0, MXQ_BF16 = 1, MXQ_DTYPE_MAX_ENUM = 0x7FFFFFFF } mxq_dtype;

/*
 * mxq_quantize -- MXFP4 block quantization along each row ([FLX] "What is MXFP4";
 * [MXA] "What it actually does"; [Q13] dynamic activations).
 * For each row and each block of 32 consecutive elements starting at a multiple of 32:
 *   amax = max |x|;  scale byte s = max(E(amax) - 2, 0), E = biased binary32 exponent
 *   field, i.e. X = 2^(clamp(floor(log2 amax) - 2, -127, 127)), all-zero block -> 0x00;
 *   code = E2M1 round-to-nearest-even of x / X, saturated to +-6, sign bit from x.
 * x      : `rows` rows of `cols` elements of type `dt`, row pitch `ld_x` elements.
 *          Base and row pitch in bytes must be multiples of 16.  Finite values only: a
 *          block holding an infinity or a NaN gets scale byte 0xFF (the E8M0 NaN) and
 *          unspecified codes; the other blocks are unaffected.
 * codes  : out, rows x cols/2 bytes, pitch ld_codes bytes (multiple of 16, base 16-aligned).
 * scales : out, rows x cols/32 bytes, pitch ld_scales bytes (any alignment).
 * Errors : cols % 32 != 0, negative sizes, pitches below the row width, NULL pointers,
 *          misalignment -> MXQ_ERR_INVALID_ARG; unknown dt -> MXQ_ERR_UNSUPPORTED.
 */
mxq_status mxq_quantize(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                        uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                        void* stream);

/* Scale rule of mxq_quantize_rule. */
typedef enum {
  MXQ_SCALE_OCP = 0, /* X = 2^(floor(log2 amax) - 2): the rule of mxq_quantize */
  MXQ_SCALE_UOS = 1, /* X = smallest power of two with amax <= 7.25 X */
  MXQ_SCALE_RULE_MAX_ENUM = 0x7FFFFFFF
} mxq_scale_rule;

/*
 * mxq_quantize_rule -- mxq_quantize with a choice of block scale rule.
 * MXQ_SCALE_UOS follows [MXA] "What it actually does" (Universal Optimal Scaling, a
 * data-free scaling boundary Qmax = 7.25): X = 2^k with k the smallest integer such that
 * amax <= 7.25 * 2^k, clamped to [-127, 127]; all-zero block -> 0x00.  Equivalently the
 * OCP byte plus one when the significand of amax exceeds 1.8125, floored at 0.  The
 * element rounding, layout, arguments and errors are those of mxq_quantize; an unknown
 * rule -> MXQ_ERR_UNSUPPORTED.
 */
mxq_status mxq_quantize_rule(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                             uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                             mxq_scale_rule rule, void* stream);

/*
 * mxq_quantize_hadamard -- fixed block-Hadamard rotation, then MXFP4 ([Q13] the data-free
 * Hadamard transform of the block selector; [ORK] "Status": block-Hadamard with
 * per-group scales).  Every run of block_n consecutive elements along a row becomes
 * x H / sqrt(block_n) (H the Sylvester Hadamard matrix; block_n = 16, 64 or 256 so the
 * normalisation is a power of two), formed in binary32 by the radix-2 butterfly in stage
 * order h = 1, 2, 4, ... ((x_i, x_{i+h}) -> (x_i + x_{i+h}, x_i - x_{i+h}), each rounded),
 * then quantized like binary32 input of mxq_quantize_rule.  Rotating activations here
 * and weights with the same call leaves A W^T unchanged up to that rounding.
 * Arguments, layout and errors as mxq_quantize_rule; cols must be a multiple of block_n
 * (MXQ_ERR_INVALID_ARG); another block_n -> MXQ_ERR_UNSUPPORTED.  An infinity or NaN
 * reaches every element of its run, so every block of that run gets scale byte 0xFF.
 */
mxq_status mxq_quantize_hadamard(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                                 int block_n, mxq_scale_rule rule, uint8_t* codes, int64_t ld_codes,
                                 uint8_t* scales, int64_t ld_scales, void* stream);

/*
 * mxq_quantize_fp8 -- static FP8 E4M3 activation quantization for W4A8 ([Q13]).
 *   q = E4M3(fl32(x * inv_scale)): one binary32 multiply (round to nearest even), then
 *   E4M3 round-to-nearest-even saturating at +-448 (never NaN); sign bit from the product.
 * inv_scale is the static per-tensor multiplier, normally fl32(448 / amax) with amax
 * measured once ahead of time (mxq_absmax); the GEMM takes s_a = fl32(amax / 448).
 * mxq_fp8_static_scales forms both.
 * x : rows x cols of `dt`, pitch ld_x elements; base and pitch 16-byte aligned.
 * q : out, rows x cols bytes, pitch ld_q bytes; base and pitch multiples of 16.
 * cols must be a multiple of 16.  Errors as for mxq_quantize; inv_scale must be finite
 * and > 0.  Finite values only: an infinity saturates to +-448 like any large value; the
 * code of a NaN is unspecified.
 */
mxq_status mxq_quantize_fp8(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                            float inv_scale, uint8_t* q, int64_t ld_q, void* stream);

/*
 * mxq_fp8_static_scales -- the static per-tensor scales of FP8 E4M3 activations ([Q13]:
 * W4A8 takes static FP8 E4M3 activations; the per-tensor amax is mapped onto the largest
 * finite E4M3 value, 448):
 *   *s_a   = fl32(amax / 448)  -- the dequantization scale mxq_gemm_w4a8 takes (a_scale),
 *   *inv_s = fl32(448 / amax)  -- the multiplier mxq_quantize_fp8 takes (inv_scale),
 * each the binary32 quotient rounded to nearest even.  A host function: amax is a value,
 * s_a and inv_s are HOST pointers written only on success; nothing touches the GPU.
 * Errors: NULL s_a / inv_s, amax not finite or <= 0, or 448 / amax beyond binary32's
 * range (amax below 448 / FLT_MAX) -> MXQ_ERR_INVALID_ARG.
 */
mxq_status mxq_fp8_static_scales(float amax, float* s_a, float* inv_s);

/*
 * mxq_absmax -- max |x| over a rows x cols tensor, written as one float to *out (device).
 * The calibration step that fixes the static FP8 scale; not part of a W4A8 call.
 * Same layout and alignment rules as mxq_quantize_fp8 (cols % 8 == 0).
 */
mxq_status mxq_absmax(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                      float* out, void* stream);

/*
 * mxq_gemm_w4a4 -- out = bf16_RNE( sum_b 2^(SA[m,b] + SW[n,b] - 254) *
 *                  sum_{i<32} e2m1(QA[m,32b+i]) * e2m1(QW[n,32b+i]) ), fp32 accumulation
 * ([Q13] W4A4; [FLX] MXFP4 consumed directly; [ORK] scales applied to block partials).
 * a_codes  : M x K/2 bytes, contiguous rows; a_scales: M x K/32 bytes, contiguous rows.
 * w_codes  : N x K/2 bytes, contiguous rows; w_scales: N x K/32 bytes, contiguous rows.
 * out_bf16 : M x N bf16, row pitch ld_out elements (>= N).
 * K % 32 == 0 (K == 0 writes zeros).  Code bases must be 16-byte aligned.
 */
mxq_status mxq_gemm_w4a4(const uint8_t* a_codes, const uint8_t* a_scales,
                         const uint8_t* w_codes, const uint8_t* w_scales,
                         int64_t M, int64_t N, int64_t K, uint16_t* out_bf16, int64_t ld_out,
                         void* stream);

/*
 * mxq_gemm_w4a4_fused -- W4A4 with the dynamic activation quantization fused into the GEMM
 * ([Q13] dynamic MXFP4 activations; [FLX] "MXFP4 quantization for diffusion models": the
 * GEMM consumes MXFP4 with no separate conversion phase).  Equal, bit for bit, to
 * mxq_quantize_rule(a, rule) followed by mxq_gemm_w4a4 on the result, without the
 * quantized activations ever leaving the GPU's on-chip memory.
 * a        : M x K activations of type `dt` (bf16 or binary32), row pitch ld_a elements;
 *            base and row pitch (bytes) multiples of 16; finite values; 256 * ld_a * size
 *            below 2^31 bytes.
 * w_codes, w_scales, out_bf16, ld_out, K : as for mxq_gemm_w4a4.
 * rule     : MXQ_SCALE_OCP or MXQ_SCALE_UOS (as mxq_quantize_rule).
 * workspace, ws_bytes : NULL (0), or device memory of at least
 *            mxq_gemm_w4a4_fused_workspace_bytes(M, N, K) bytes, 16-byte aligned, owned by
 *            the caller and not used by anything else until the call's work on `stream` is
 *            done.  The fused kernel quantizes each activation tile once per 256 output
 *            columns; past the measured break-even (more than 3 column tiles for K >= 8192,
 *            more than 1 below) a pass of its own is faster, and with a workspace the call
 *            then quantizes into it and runs mxq_gemm_w4a4 (the same bits).  With NULL the
 *            fused kernel always runs.
 * Errors as for mxq_quantize_rule and mxq_gemm_w4a4; MXQ_ERR_INVALID_ARG for a non-NULL
 * workspace that is misaligned or smaller than the size above.
 */
mxq_status mxq_gemm_w4a4_fused(const void* a, mxq_dtype dt, int64_t ld_a,
                               const uint8_t* w_codes, const uint8_t* w_scales,
                               int64_t M, int64_t N, int64_t K, mxq_scale_rule rule,
                               uint16_t* out_bf16, int64_t ld_out, void* workspace,
                               size_t ws_bytes, void* stream);

/*
 * mxq_gemm_w4a4_fused_workspace_bytes -- bytes of workspace with which mxq_gemm_w4a4_fused
 * takes the separate-quantization route for this shape: 0 where the fused kernel is the
 * faster (or for an empty or invalid shape), else M * K / 2 rounded up to 16 plus
 * M * K / 32.  Host only; no device work.
 */
size_t mxq_gemm_w4a4_fused_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * mxq_gemm_w4a8 -- out = bf16_RNE( fl32( a_scale * sum_b 2^(SW[n,b] - 127) *
 *                  sum_{i<32} e4m3(QA8[m,32b+i]) * e2m1(QW[n,32b+i]) ) ) ([Q13] W4A8).
 * a_fp8   : M x K bytes (E4M3), contiguous rows, base 16-byte aligned.
 * a_scale : the static dequantization scale s_a (finite).
 * W, out and K as for mxq_gemm_w4a4.
 * Accuracy domain: the gfx950 FP8 x FP4 block-scaled MFMA adds each group of 8
 * consecutive K products on a fixed-point grid whose last bit is 2^(E - 13), E the
 * exponent of the group's largest product, and drops what lies below it (FP4 x FP4
 * products never span that many binades, so W4A4 is unaffected).  Outputs are within
 * 1e-5 * sum|a*b| + 1 bf16 ulp of the exact result except a few per million with heavy
 * cancellation, where one group of 8 holds E4M3 values ~2^14 apart.  Measured with
 * statically scaled activations drawn like the Wan2.2 FFN inputs (N(0,1) x LogNormal(0,1)
 * per channel; Student-t(3)), up to eight seeds per case, 17.2M outputs each: 0 to 7
 * outside for K = 2048 and 5120 (at most 1.91x the bound), 0 to 84 for K = 1024 (at most
 * 2.85x); at K = 288 / 416, 5 of ~425k (at most 1.31x).
 */
mxq_status mxq_gemm_w4a8(const uint8_t* a_fp8, float a_scale,
                         const uint8_t* w_codes, const uint8_t* w_scales,
                         int64_t M, int64_t N, int64_t K, uint16_t* out_bf16, int64_t ld_out,
                         void* stream);

/*
 * mxq_gemm_bf16 -- bf16 reference for SQNR ([Q13] BF16 quality ceiling):
 * out = bf16_RNE(sum_k a[m,k] * w[n,k]), fp32 accumulation, over unquantized operands.
 * a : M x K bf16, contiguous rows; w : N x K bf16, contiguous rows; bases 16-byte
 * aligned; K % 32 == 0.  out as for mxq_gemm_w4a4.
 */
mxq_status mxq_gemm_bf16(const uint16_t* a, const uint16_t* w, int64_t M, int64_t N, int64_t K,
                         uint16_t* out, int64_t ld_out, void* stream);

/*
 * mxq_sqnr -- whole-output SQNR of `test` against `ref` ([Q13] block-output SQNR):
 *   S = sum ref^2, N = sum (ref - test)^2 over all rows x cols bf16 elements (exactly
 *   widened), dB = 10 log10(S / N); N == 0 -> +inf, S == N == 0 -> NaN.
 * Deterministic: fixed partition; every value widened exactly and every difference,
 * square and sum formed in fp64 (per thread -> per workgroup -> one final pass), so
 * any finite bf16 inputs are in range.  workspace: device scratch of at least mxq_sqnr_workspace_bytes(rows*cols)
 * bytes (8-byte aligned), owned by the caller.  out3: device double[3] = {S, N, dB}.
 * ref/test pitches in elements; bases 16-byte aligned, pitches multiples of 8, cols % 8 == 0.
 */
size_t mxq_sqnr_workspace_bytes(int64_t n_elements);
mxq_status mxq_sqnr(const uint16_t* ref, const uint16_t* test, int64_t rows, int64_t cols,
                    int64_t ld_ref, int64_t ld_test, void* workspace, size_t ws_bytes,
                    double* out3, void* stream);

/*
 * mxq_sqnr_noalloc -- mxq_sqnr without a caller workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation).  Same arguments, checks and results as mxq_sqnr (the same
 * kernels, bit for bit), minus workspace / ws_bytes: the partial sums live in a 16 KB
 * static device array of the library, one per GPU, held until the process ends; its
 * address is looked up on the first call on each device.  Nothing is allocated or freed.
 * Every call on one GPU shares that array, so calls that may overlap on one GPU (streams
 * with no ordering between them) race: order them.  No state carries from one call to
 * the next (each call writes every slot it reads).  A request needing more than the
 * 16 KB -> MXQ_ERR_INVALID_ARG (no size does: the workspace is fixed).
 */
mxq_status mxq_sqnr_noalloc(const uint16_t* ref, const uint16_t* test, int64_t rows, int64_t cols,
                            int64_t ld_ref, int64_t ld_test, double* out3, void* stream);

/*
 * mxq_dequantize -- MXFP4 -> bf16: y = bf16(e2m1(code) * 2^(scale - 127)) (rounded to
 * nearest even only where the product leaves bf16's range: below 2^-133 or above 2^127).
 * The quantize-dequantize (QDQ) emulation step ([Q13]: W4A8 quality was measured by
 * QDQ emulation).  codes/scales as produced by mxq_quantize; y: rows x cols bf16, pitch
 * ld_y elements, base and pitch 16-byte aligned.
 */
mxq_status mxq_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales,
                          int64_t ld_scales, int64_t rows, int64_t cols, uint16_t* y,
                          int64_t ld_y, void* stream);

/*
 * mxq_dequantize_fp8 -- FP8 E4M3 -> bf16, the W4A8 activation half of quantize-dequantize
 * (QDQ) emulation ([Q13]: W4A8 quality was measured by QDQ emulation):
 *   y = bf16_RNE( fl32( e4m3(q) * a_scale ) )
 * i.e. the exact E4M3 value times the static dequantization scale s_a in one binary32
 * multiply (round to nearest even), then rounded to bf16 (nearest even).  NaN codes
 * (S.1111.111, which mxq_quantize_fp8 never writes) give NaN.
 * q : rows x cols bytes, pitch ld_q bytes; base and pitch multiples of 16.
 * y : out, rows x cols bf16, pitch ld_y elements; base 16-byte aligned, ld_y % 8 == 0.
 * cols % 16 == 0; a_scale finite.  Errors -> MXQ_ERR_INVALID_ARG before any launch.
 */
mxq_status mxq_dequantize_fp8(const uint8_t* q, int64_t ld_q, float a_scale, int64_t rows, int64_t cols,
                              uint16_t* y, int64_t ld_y, void* stream);

/*
 * 8-bit integers: one binary32 scale for each row (a token of the activations, an output
 * channel of the weights), for layers that need more than W4A4 and no calibration.
 *
 * mxq_quantize_int8 -- symmetric 8-bit quantization of each row:
 *   amax = max |x| of the row;  scale = fl32(amax / 127),  inv = fl32(127 / amax);
 *   code = RNE(fl32(x * inv)), in [-127, 127]; both quotients correctly rounded.
 * A row whose amax is below 2^-118 (an all-zero row too) gets scale 0 and codes 0.  A row
 * holding an infinity or a NaN gets scale NaN and codes 0; other rows are unaffected.
 * x      : rows x cols of `dt`, pitch ld_x elements; base and pitch 16-byte aligned.
 * codes  : out, rows x cols int8, pitch ld_codes bytes; base and pitch multiples of 16.
 * scales : out, float[rows].
 * cols % 16 == 0 (cols == 0 writes scales of 0).  Errors as for mxq_quantize_fp8.
 */
mxq_status mxq_quantize_int8(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                             int8_t* codes, int64_t ld_codes, float* scales, void* stream);

/*
 * mxq_dequantize_int8 -- 8-bit codes -> bf16: y = bf16_RNE( fl32( code * scale[row] ) ), the
 * quantize-dequantize (QDQ) emulation step.
 * codes : rows x cols int8, pitch ld_codes bytes (base and pitch multiples of 8);
 * scales: float[rows];  y : out, rows x cols bf16, pitch ld_y elements, base 16-byte
 * aligned, ld_y % 8 == 0.  cols % 8 == 0.
 */
mxq_status mxq_dequantize_int8(const int8_t* codes, int64_t ld_codes, const float* scales, int64_t rows,
                               int64_t cols, uint16_t* y, int64_t ld_y, void* stream);

/*
 * mxq_gemm_w8a8 -- 8-bit product with a scale for each token and each output channel:
 *   acc = sum_k a[m,k] * w[n,k] (int32, exact);  t = fl32( fl32(acc) * a_scales[m] );
 *   v = fl32( t * w_scales[n] ), or with a bias the fused multiply-add t * w_scales[n] + bias[n]
 *   rounded once;  out = v as binary32 (MXQ_F32) or bf16_RNE(v) (MXQ_BF16).
 * a : M x K int8, pitch ld_a bytes; w : N x K int8, pitch ld_w bytes.  Bases and pitches
 *     multiples of 16, pitches below 2^23 (fastest where both are multiples of 128).  Any int8
 *     codes, -128 included.
 * a_scales, w_scales : float, element m (n) at m * inc_as (n * inc_ws), increments >= 0 (0:
 *     one scale for all).  bias : float[N] or NULL.
 * out : M x N of out_dt, pitch ld_out elements (>= N), naturally aligned.
 * K % 16 == 0 and K < 2^17 (the sum then fits int32); K == 0 gives the bias, or zeros.
 * N <= 2^28, and M x N covered by at most 2^22 tiles of 256 x 256.
 * workspace, ws_bytes : NULL (0), or device memory of at least
 *     mxq_gemm_w8a8_workspace_bytes(M, N, K) bytes, 16-byte aligned, owned by the caller and
 *     not used by anything else until the call's work on `stream` is done.  With one, a
 *     long K over few output tiles is split over the GPU and summed in a second launch;
 *     the bits are the same either way.
 */
mxq_status mxq_gemm_w8a8(const int8_t* a, int64_t ld_a, const float* a_scales, int64_t inc_as,
                         const int8_t* w, int64_t ld_w, const float* w_scales, int64_t inc_ws,
                         const float* bias, int64_t M, int64_t N, int64_t K, void* out,
                         mxq_dtype out_dt, int64_t ld_out, void* workspace, size_t ws_bytes,
                         void* stream);

/*
 * mxq_gemm_w8a8_workspace_bytes -- workspace with which mxq_gemm_w8a8 splits K for a shape: 0
 * where it does not (or for an empty or invalid shape).  Host only; no device work.
 */
size_t mxq_gemm_w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * mxq_gemm_w8a8_fused -- mxq_gemm_w8a8 on unquantized activations, equal bit for bit to
 * mxq_quantize_int8(a) followed by mxq_gemm_w8a8 on the result.
 * a : M x K of `dt`, pitch ld_a elements; base and pitch (bytes) 16-byte aligned.
 * workspace, ws_bytes : device memory of at least mxq_gemm_w8a8_fused_workspace_bytes(M, N, K)
 *     bytes, 16-byte aligned (NULL where that is 0), owned by the caller and not used by
 *     anything else until the call's work on `stream` is done.
 * The other arguments and errors are those of mxq_quantize_int8 and mxq_gemm_w8a8;
 * MXQ_ERR_INVALID_ARG for a missing, misaligned or short workspace.
 */
mxq_status mxq_gemm_w8a8_fused(const void* a, mxq_dtype dt, int64_t ld_a, const int8_t* w, int64_t ld_w,
                               const float* w_scales, int64_t inc_ws, const float* bias, int64_t M,
                               int64_t N, int64_t K, void* out, mxq_dtype out_dt, int64_t ld_out,
                               void* workspace, size_t ws_bytes, void* stream);

/*
 * mxq_gemm_w8a8_fused_workspace_bytes -- workspace of mxq_gemm_w8a8_fused for a shape (0 for
 * an empty or invalid one).  Host only; no device work.
 */
size_t mxq_gemm_w8a8_fused_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* Which elements of a head turn together (mxq_qk_norm_rope), R the rotated width. */
typedef enum {
  MXQ_ROPE_INTERLEAVED = 0, /* (2i, 2i+1), i < R/2 */
  MXQ_ROPE_HALVES = 1,      /* (i, i + R/2), i < R/2 */
  MXQ_ROPE_STYLE_MAX_ENUM = 0x7FFFFFFF
} mxq_rope_style;

/*
 * mxq_qk_norm_rope -- root-mean-square norm of every query and key head with the position
 * rotation in the same pass (the step between the QKV projection and attention in blocks that
 * norm each head, as FLUX does; Wan norms the whole query and the whole key of a token before
 * the split into heads, with a weight of that width: another operator, which this is not).
 * For each token and head x of head_dim elements, in binary32:
 *   r = 1 / sqrt( sum x^2 / head_dim + eps );  y = (x * r) * w;
 *   pairs (a, b) of the first rot_dim elements -> (a c - b s, b c + a s), c and s from row
 *   p of cos and sin, column i (mxq_rope_style), p = positions[token] (token if NULL);
 * rounded to `dt` once.  The sum of squares is formed in binary32: a head where it
 * overflows comes out as zeros; with eps == 0 one whose mean of squares is 0 there (all
 * zeros, or elements of about 2^-75 and less) as NaN or infinities.  Other heads are
 * unaffected.  The rotated elements of a token whose position is outside [0, table_rows)
 * come out as NaN, and no memory outside the table is read for it.
 * q, k    : tokens x heads x head_dim of `dt`; element (t, h, d) at t * ld + h * hs + d.
 *           Either may have 0 heads (its other arguments are then ignored).
 * w_q, w_k: head_dim weights of w_dt each, or NULL for 1.
 * cos, sin: table_rows x rot_dim / 2 float, pitch ld_table; unused when rot_dim == 0.
 * out_q, out_k : like q and k, of `dt`, no two heads of an output on the same memory
 *           (MXQ_ERR_INVALID_ARG).  An output may be its input with the same pitches; no other
 *           overlap.
 * head_dim: a multiple of 8 up to 512; rot_dim: a multiple of 8 up to head_dim; heads up
 *           to 65536 each.  Bases 16-byte aligned; all pitches of q, k, out_q, out_k
 *           multiples of 16 bytes and not negative; ld_table % 4 == 0.  The heads of one
 *           token and 16 more at that pitch span less than 2^31 bytes.
 */
mxq_status mxq_qk_norm_rope(const void* q, int64_t heads_q, int64_t ld_q, int64_t hs_q, const void* k,
                            int64_t heads_k, int64_t ld_k, int64_t hs_k, mxq_dtype dt, int64_t tokens,
                            int64_t head_dim, const void* w_q, const void* w_k, mxq_dtype w_dt, float eps,
                            const float* cos, const float* sin, int64_t ld_table, int64_t table_rows,
                            int64_t rot_dim, const int64_t* positions, mxq_rope_style style, void* out_q,
                            int64_t ld_oq, int64_t hs_oq, void* out_k, int64_t ld_ok, int64_t hs_ok,
                            void* stream);

/*
 * mxq_quantize_qk_norm_rope -- the same, then the rule of mxq_quantize_int8 on the binary32
 * values of each token and head: codes int8 (pitches in bytes, bases and pitches multiples
 * of 8) and one scale for each, at t * ld_s + h.  With pitches that are multiples of 16 a head's codes are
 * operands of mxq_gemm_w8a8 (the 8-bit score product of a head).
 */
mxq_status mxq_quantize_qk_norm_rope(const void* q, int64_t heads_q, int64_t ld_q, int64_t hs_q, const void* k,
                                     int64_t heads_k, int64_t ld_k, int64_t hs_k, mxq_dtype dt, int64_t tokens,
                                     int64_t head_dim, const void* w_q, const void* w_k, mxq_dtype w_dt, float eps,
                                     const float* cos, const float* sin, int64_t ld_table, int64_t table_rows,
                                     int64_t rot_dim, const int64_t* positions, mxq_rope_style style,
                                     int8_t* codes_q, int64_t ld_cq, int64_t hs_cq, float* scales_q, int64_t ld_sq,
                                     int8_t* codes_k, int64_t ld_ck, int64_t hs_ck, float* scales_k, int64_t ld_sk,
                                     void* stream);

/*
 * Layer norm, and activations kept in 8 bits for the backward pass: what stands between the
 * 8-bit products of a transformer block, forward and backward.  The codes and row scales are
 * those of mxq_quantize_int8.
 *
 * mxq_layer_norm -- for each row x of cols elements, in binary32:
 *   mean = sum x / cols;  rstd = 1 / sqrt( sum (x - mean)^2 / cols + eps );
 *   y = (x - mean) * rstd * w + b,  rounded to `dt` once.
 * The deviations are taken from the mean itself (no difference of two squares), and a row of equal
 * finite values comes out as b.  A row with an infinity or a NaN comes out as NaN; a row whose squared
 * deviations overflow binary32 in their sum (a root mean square of 2^64 / sqrt(cols) and more) as b,
 * infinities or NaN.  With eps == 0 a row of equal values is NaN, and deviations that are all below 2^-60 lose
 * digits, for their squares leave binary32's normal numbers (all below 2^-75: infinities or NaN).
 * Other rows are unaffected.
 * x       : rows x cols of `dt`, pitch ld_x elements; base and pitch 16-byte aligned.
 * w, b    : cols weights and biases of w_dt, 16-byte aligned; either may be NULL (1, 0).
 * y       : out, rows x cols of `dt`, pitch ld_y elements; base and pitch 16-byte aligned.  May be
 *           x with the same pitch; no other overlap.
 * mean, rstd : out, float[rows] each, or both NULL.
 * x_codes, x_scales : out, the checkpoint mxq_quantize_int8(x), bit for bit (pitch ld_xc bytes, base
 *           and pitch multiples of 16), or x_codes NULL for none (ld_xc and x_scales are then ignored).
 *           Their step is 1/127 of the row's largest |x|: (x - mean) * rstd from them is off by up to x_scales / 2 *
 *           rstd, which is much for a row with an outlier or with a mean that is large beside its deviation.
 * cols    : a multiple of 8 (16 with x_codes), 8 to 16384.  eps finite and >= 0.
 */
mxq_status mxq_layer_norm(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x, const void* w,
                          const void* b, mxq_dtype w_dt, float eps, void* y, int64_t ld_y, float* mean,
                          float* rstd, int8_t* x_codes, int64_t ld_xc, float* x_scales, void* stream);

/*
 * mxq_quantize_layer_norm -- the same, then the rule of mxq_quantize_int8 on the binary32 values of
 * each row: codes (pitch ld_codes bytes; base and pitch multiples of 16) and float scales[rows],
 * operands of mxq_gemm_w8a8.  A row whose squares overflow, or with eps == 0 vanish, gets scale
 * NaN and codes 0.  cols: a multiple of 16.
 */
mxq_status mxq_quantize_layer_norm(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_x,
                                   const void* w, const void* b, mxq_dtype w_dt, float eps, int8_t* codes,
                                   int64_t ld_codes, float* scales, float* mean, float* rstd, int8_t* x_codes,
                                   int64_t ld_xc, float* x_scales, void* stream);

/*
 * mxq_layer_norm_backward -- with xh = (x - mean) * rstd and g = dy * w, in binary32:
 *   dx = rstd * ( g - sum g / cols - xh * sum (g xh) / cols ), rounded to `dt` once;
 *   dw = sum over rows of dy * xh;  db = sum over rows of dy.
 * The sums over rows are formed in an order that rows, cols and dt alone decide: the same inputs
 * give the same bits.
 * dy, dx  : rows x cols of `dt`; dx may be dy with the same pitch.
 * x       : with x_scales NULL the kept input, of `dt`; else its codes (int8, one float x_scales
 *           for each row; cols a multiple of 16), which stand for fl32(code * scale).
 * All bases and pitches 16-byte aligned.
 * mean, rstd : float[rows], as mxq_layer_norm left them.
 * w       : cols weights of w_dt, or NULL for 1.
 * dw, db  : out, float[cols] each, 16-byte aligned, or both NULL.  rows == 0 writes zeros.
 * workspace, ws_bytes : device memory of at least mxq_layer_norm_backward_workspace_bytes(rows, cols)
 *           bytes, 16-byte aligned (NULL where that is 0, or without dw and db), owned by the caller and
 *           not used by anything else until the call's work on `stream` is done.
 */
mxq_status mxq_layer_norm_backward(const void* dy, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_dy,
                                   const void* x, int64_t ld_x, const float* x_scales, const float* mean,
                                   const float* rstd, const void* w, mxq_dtype w_dt, void* dx, int64_t ld_dx,
                                   float* dw, float* db, void* workspace, size_t ws_bytes, void* stream);

/* Workspace of mxq_layer_norm_backward with dw and db (0 for an empty or invalid shape).  Host only. */
size_t mxq_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols);

/* Activation functions of a feed-forward layer (mxq_activation), s(z) = 1 / (1 + exp(-z)). */
typedef enum {
  MXQ_ACT_GELU_TANH = 0, /* u * s(2 sqrt(2 / pi) (u + 0.044715 u^3)): the tanh form of GELU */
  MXQ_ACT_SILU = 1,      /* u * s(u) */
  MXQ_ACTIVATION_MAX_ENUM = 0x7FFFFFFF
} mxq_activation_kind;

/*
 * mxq_activation -- y = f(u) element by element, in binary32, rounded to `dt` once, with an 8-bit
 * checkpoint of u for the backward pass.
 * u       : rows x cols of `dt`, pitch ld_u elements; base and pitch 16-byte aligned.
 * y       : out, rows x cols of `dt`, pitch ld_y elements; base and pitch 16-byte aligned.  May be u
 *           with the same pitch; no other overlap.
 * u_codes, u_scales : out, the checkpoint (pitch ld_uc bytes; base and pitch multiples of 16), or
 *           u_codes NULL for none (ld_uc and u_scales are then ignored).  It is the rule of
 *           mxq_quantize_int8 on u clamped to [-L, L], L = 4 for MXQ_ACT_GELU_TANH and 8 for MXQ_ACT_SILU:
 *           beyond L the derivative is within 4e-4 and 3e-3 of 0 or 1, and the step stays at most
 *           L / 127.  Infinities are clamped; a row with a NaN gets scale NaN and codes 0.
 * f(+inf) = +inf, f(-inf) = NaN.
 * cols    : a multiple of 8 (16 with u_codes), up to 65536.
 */
mxq_status mxq_activation(const void* u, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_u,
                          mxq_activation_kind act, void* y, int64_t ld_y, int8_t* u_codes, int64_t ld_uc,
                          float* u_scales, void* stream);

/*
 * mxq_quantize_activation -- the same, then the rule of mxq_quantize_int8 on the binary32 values
 * of each row: codes (pitch ld_codes bytes; base and pitch multiples of 16) and float scales[rows],
 * operands of mxq_gemm_w8a8.  cols: a multiple of 16.
 */
mxq_status mxq_quantize_activation(const void* u, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_u,
                                   mxq_activation_kind act, int8_t* codes, int64_t ld_codes, float* scales,
                                   int8_t* u_codes, int64_t ld_uc, float* u_scales, void* stream);

/*
 * mxq_activation_backward -- du = dy * f'(v) with v = fl32(code * scale) of the checkpoint, in
 * binary32, rounded to `dt` once.
 * dy, du  : rows x cols of `dt`, pitches in elements, 16-byte aligned; du may be dy with the same pitch.
 * u_codes, u_scales : the checkpoint of the same activation (or any other codes and scales; a row whose scale is
 *           not finite gives NaN).  cols: a multiple of 16.
 */
mxq_status mxq_activation_backward(const void* dy, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ld_dy,
                                   const int8_t* u_codes, int64_t ld_uc, const float* u_scales,
                                   mxq_activation_kind act, void* du, int64_t ld_du, void* stream);

/*
 * mxq_grad_weight_int8 -- the weight gradient of mxq_gemm_w8a8 from the codes that the forward
 * product took, N x K as the weights are:
 *   dW[n,k] = sum_m dy[m,n] * bf16_RNE( fl32( code[m,k] * scale[m] ) ), binary32 accumulation over
 * the values that mxq_dequantize_int8 gives, rounded to out_dt once; with `accumulate` not 0 that
 * sum is added to what `out` holds, in binary32, before the rounding.
 * The order of the sum is decided by M, N and K alone: the same inputs give the same bits.
 * dy      : M x N bf16, pitch ld_dy elements below 2^23; base and pitch 16-byte aligned.
 * codes   : M x K int8, pitch ld_codes bytes below 2^23; base and pitch multiples of 16.  scales : float[M].
 * out     : N x K of out_dt, pitch ld_out elements (>= K), naturally aligned (stored fastest on 16-byte
 *           boundaries).
 * N % 8 == 0, K % 16 == 0; N and K up to 2^22, N * K up to 2^36, M * K below 2^35.  M == 0 gives zeros
 * (with accumulate: leaves `out`).
 * workspace, ws_bytes : device memory of at least mxq_grad_weight_int8_workspace_bytes(M, N, K)
 *           bytes, 16-byte aligned (NULL where that is 0), owned by the caller and not used by anything
 *           else until the call's work on `stream` is done.
 */
mxq_status mxq_grad_weight_int8(const uint16_t* dy, int64_t ld_dy, const int8_t* codes, int64_t ld_codes,
                                const float* scales, int64_t M, int64_t N, int64_t K, void* out,
                                mxq_dtype out_dt, int64_t ld_out, int accumulate, void* workspace,
                                size_t ws_bytes, void* stream);

/* Workspace of mxq_grad_weight_int8 for a shape (0 for an empty or invalid one).  Host only. */
size_t mxq_grad_weight_int8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * Measurement aid (not part of the quantize / GEMM path).
 *
 * mxq_mfma_ceiling -- the MFMA throughput the chip sustains on the operand bits of a GEMM
 * call, with no memory traffic.  The MI355X holds its power under these GEMMs by lowering
 * its clock, and the energy of an MFMA grows with the operand bits that toggle, so this
 * ceiling (not the dense peak) bounds what a GEMM can reach on the same data.
 * Each lane of `waves` waves gathers 4 weight and 4 activation fragments (the bytes one
 * lane of the GEMM's MFMA holds) from pseudo-random rows and 32-element blocks of the
 * operand planes, with their scale bytes.  It then runs iters x 16 MFMAs of the GEMM's
 * instruction on them in registers: v_mfma_scale_f32_32x32x64_f8f6f4 (W4A4, W4A8) or
 * v_mfma_f32_16x16x32_bf16.
 * Work: waves * iters * 16 MFMAs of 2*32*32*64 FLOP (W4A4, W4A8) or 2*16*16*32 (bf16).
 * mode   : which GEMM's operands: W4A4 a = activation codes, a_scales; W4A8 a = FP8 bytes
 *          (a_scales unused); bf16 a = bf16 activations (no scales).  w / w_scales: the
 *          weight codes and scales (W4A4, W4A8) or bf16 weights.  Layouts as for the GEMMs:
 *          M x K activations and N x K weights, contiguous rows, bases 16-byte aligned.
 * K      : a positive multiple of 32; M, N >= 1.
 * waves  : a multiple of 4 in [4, 2^20]; iters in [1, 2^24].
 * sink   : device float[waves * 64], owned by the caller: one value per lane (keeps the
 *          work live; not a result).
 * Errors : MXQ_ERR_UNSUPPORTED for an unknown mode, MXQ_ERR_INVALID_ARG for bad sizes or
 *          pointers, checked before anything is enqueued.
 */
typedef enum {
  MXQ_GEMM_W4A4 = 0,
  MXQ_GEMM_W4A8 = 1,
  MXQ_GEMM_BF16 = 2,
  MXQ_GEMM_MODE_MAX_ENUM = 0x7FFFFFFF
} mxq_gemm_mode;
mxq_status mxq_mfma_ceiling(mxq_gemm_mode mode, const void* a, const uint8_t* a_scales,
                            const void* w, const uint8_t* w_scales, int64_t M, int64_t N,
                            int64_t K, int64_t waves, int64_t iters, float* sink, void* stream);

/* Thread-local message for the last failing call on this thread ("" if none). Valid
 * until the next mxq_* call on the same thread. */
const char* mxq_last_error(void);

/* MXQ_ABI_VERSION of the loaded library. */
int mxq_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_H */
