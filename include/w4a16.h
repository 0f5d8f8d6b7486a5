/*
 * libw4a16 -- asymmetric group-wise 4-bit weights (group 128) and fused
 * dequantizing matrix-vector / matrix-matrix products for AMD gfx950.
 *
 * Plain C ABI: every buffer is a raw device pointer owned by the caller, every
 * size is an integer, every call is asynchronous on the given HIP stream.
 * The library never allocates, frees or synchronizes device memory.
 *
 * Format (page "Weight quantization", sections "How it works" and "Code";
 * the affine map is also given on "LLM Quantization Architecture in Depth"
 * › "Number formats, scales and granularity"):
 *   - W is [N, K] row-major (N outputs, K inputs); groups are 128 consecutive
 *     inputs of one row, so K must be a multiple of 128.
 *   - per group: lo = min(min(w), 0), hi = max(max(w), 0);
 *     scale = (hi - lo) / 15 in binary32, or 1 when hi == lo;
 *     zero  = clamp(round(-lo / scale), 0, 15);
 *     code  = clamp(round(w / scale) + zero, 0, 15);
 *     round = nearest, halves away from zero; every step one IEEE binary32
 *     operation (true division, no fused multiply-add, subnormals kept).
 *   - canonical storage: packed [N, K/2] bytes, code of the even input index in
 *     the low nibble; scales [N, K/128] binary16 bit patterns (the binary32
 *     scale rounded to nearest even); zeros [N, K/128] bytes.
 *   - w_hat = (code - zero) * scale16 and the products use, per group,
 *     scale16 * sum (code - zero) * x: one multiply per group, with the exact
 *     difference code - zero as the operand of every product.
 *
 * Readings of points the pages leave open are fixed above: halves away from
 * zero, codes from the binary32 scale, fp16 stored scale, byte zero.
 *
 * Errors: the return value reports argument validation and launch failures
 * synchronously; W4_ERR_HIP carries the runtime's message in
 * w4_last_hip_error().  Data conditions found on the device are OR-ed into the
 * optional status word (see w4_quantize).  Nothing falls back to another code
 * path: an unsupported request is refused.
 *
 * Threading: no mutable global state except a per-device architecture check
 * done once; calls from several host threads are safe.  Calls that share an
 * output buffer must be ordered by the caller.
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define W4_GROUP 128
#define W4_FORMAT_VERSION 3
#define W4_GEMV_MAX_M 16
#define W4_GEMV_MAX_K 32768
#define W4_FP8_MAX_K 65536
#define W4_GEMM_MAX_K (1 << 20)
#define W4_ROWS_MAX_K 65536
#define W4_MAX_SEQUENCES 4096
#define W4_MAX_TOKENS (1 << 22)
#define W4_MAX_CONTEXT (1 << 30)

typedef enum {
    W4_OK = 0,
    W4_ERR_NULL = 1,         /* a required pointer is NULL */
    W4_ERR_SHAPE = 2,        /* N < 1, K < 128, K % 128 != 0, M out of range, size limit */
    W4_ERR_ALIGN = 3,        /* a pointer breaks its stated alignment */
    W4_ERR_DTYPE = 4,        /* dtype value not accepted by this call */
    W4_ERR_UNSUPPORTED = 5,  /* request outside the fixed format */
    W4_ERR_ARCH = 6,         /* current device is not gfx950 */
    W4_ERR_WORKSPACE = 7,    /* workspace missing or too small */
    W4_ERR_HIP = 8,          /* HIP runtime error; see w4_last_hip_error() */
    W4_ERR_BUFFER = 9,       /* destination buffer smaller than required */
    W4_ERR_VALUE = 10        /* a number outside its range (eps, a scale, a window, a rope record) */
} w4_status;

typedef enum { W4_F32 = 0, W4_BF16 = 1 } w4_dtype;

/* Device status word bits (OR-ed, never cleared): the first three written by w4_quantize, the first also
 * by the calls that quantize rows to 8 bits, the last three by the paged-cache calls. */
#define W4_STATUS_NONFINITE      1u  /* a weight or a value of a row was NaN or +-inf (outputs undefined) */
#define W4_STATUS_SCALE_OVERFLOW 2u  /* a binary32 scale rounded to binary16 infinity */
#define W4_STATUS_SCALE_ZERO     4u  /* a non-empty group's scale rounded to binary16 zero */
#define W4_STATUS_PAGE           8u  /* a page or slot number outside the cache */
#define W4_STATUS_LENGTH        16u  /* a negative length, or more new tokens than the arrays hold */
#define W4_STATUS_PAGES_SHORT   32u  /* a request found too few free pages or table entries */

/*
 * w4_quantize -- round-to-nearest quantization of W (page "Weight quantization",
 * "How it works": scale, zero and code formulas; "Code": range widened to 0,
 * f32 arithmetic, nibble packing with the even index low).
 *   W          [N, K] row-major, binary32 (wt = W4_F32) or bfloat16 (W4_BF16); 16-B aligned.
 *   packed     out [N, K/2] bytes; 16-B aligned.
 *   scales_f16 out [N, K/128] binary16 bit patterns; 2-B aligned.
 *   zeros      out [N, K/128] bytes.
 *   d_status   optional device word (may be NULL); W4_STATUS_* bits are OR-ed in.
 * Requires N >= 1, K >= 128, K % 128 == 0.  Deterministic; bit-exact with the
 * formulas above for finite input.
 */
w4_status w4_quantize(const void* W, w4_dtype wt, int64_t N, int64_t K,
                      uint8_t* packed, uint16_t* scales_f16, uint8_t* zeros,
                      uint32_t* d_status, hipStream_t stream);

/*
 * w4_quantize_symmetric -- the symmetric variant (page "Quantization" › "How it
 * really works" › "The mechanics: scale, round, clamp"): per group of 128 the step
 * is max|w| / 7 (1 for an all-zero group), each code is round(w / step) with halves
 * to even, clamped to [-8, 7]; one binary32 operation per step.  Written in the same
 * canonical arrays as w4_quantize: stored code = code + 8, every zero = 8, scale =
 * the step rounded to binary16 -- so w4_prepare, w4_gemv and w4_gemm take the result
 * unchanged ((stored - zero) * scale16 is the dequantized weight).
 * Arguments, alignment, errors and d_status bits as w4_quantize.
 */
w4_status w4_quantize_symmetric(const void* W, w4_dtype wt, int64_t N, int64_t K,
                                uint8_t* packed, uint16_t* scales_f16, uint8_t* zeros,
                                uint32_t* d_status, hipStream_t stream);

/*
 * Kernel layout ("pre-shuffled" weights with interleaved scale and zero: page
 * "LLM Quantization Architecture in Depth" › "Kernels and memory layout: the
 * format is a contract"; the stage list's "Memory Layout" on the
 * architecture page).  The prepared buffer is opaque; its size is
 * w4_prepared_bytes(N, K).  w4_prepare is a bijection of the canonical arrays
 * and w4_unprepare is its exact inverse.
 *   packed/scales_f16/zeros  canonical arrays as produced by w4_quantize
 *                            (packed 16-B aligned, scales 2-B aligned).
 *   prepared                 [w4_prepared_bytes(N, K)] bytes, 256-B aligned.
 * The products read zeros 0..15 (what w4_quantize writes); the round trip holds for
 * any byte.
 */
size_t w4_prepared_bytes(int64_t N, int64_t K);
w4_status w4_prepare(const uint8_t* packed, const uint16_t* scales_f16, const uint8_t* zeros,
                     int64_t N, int64_t K, void* prepared, size_t prepared_bytes,
                     hipStream_t stream);
w4_status w4_unprepare(const void* prepared, int64_t N, int64_t K,
                       uint8_t* packed, uint16_t* scales_f16, uint8_t* zeros,
                       hipStream_t stream);

/*
 * w4_gemv -- decode-sized product y[m, n] = sum_k w_hat[n, k] * x[m, k] for
 * 1 <= M <= 16, never forming w_hat in memory (page "Weight quantization",
 * "How it works": the per-group factored dot; architecture page stage "Fused
 * Kernels": dequantization inside the product).  Every product multiplies the exact
 * value q - zero of a code (a code equal to its zero adds exactly 0); bf16 x enters
 * the one-row kernel as binary16 x * 2^-E, E per wave of 2048 inputs (exact within 2^25
 * of the wave's largest value; a wave with a value outside that window, and binary32 x,
 * use one binary32 FMA per input instead), and the matrix-core kernels (2 <= M <= 16;
 * M = 2 stays on the one-row kernel unless the matrix has more than 16384 rows and
 * K <= 8192) as binary16 x * 2^-E with binary16 codes where x converts exactly (on
 * matrices with K <= 8192 and at least 48 rows per compute unit, E per wave; on the
 * others with M <= 4, E per wave and row of x), else as bf16 with bf16 q - zero codes.
 *   prepared  from w4_prepare (256-B aligned).
 *   x         [M, K] row-major, bfloat16 (xt = W4_BF16) or binary32 (W4_F32); 16-B aligned.
 *   y         [M, N] row-major, binary32 (yt = W4_F32) or bfloat16 (W4_BF16); must
 *             not overlap the inputs; 4-B aligned.
 * Requires K <= W4_GEMV_MAX_K.  Accumulates in binary32; deterministic (no atomics).
 */
w4_status w4_gemv(const void* prepared, int64_t N, int64_t K,
                  const void* x, w4_dtype xt, int64_t M,
                  void* y, w4_dtype yt, hipStream_t stream);

/*
 * Storage variants of the format (page "Quantization" › "Code": int4 groups of 128
 * and of 32; page "Weight quantization" › "Implementation notes": scales kept in fp16
 * or bf16; "Code" and "Complexity and constants": a 4-bit zero per group).
 *   group       32, 64 or 128 consecutive inputs of one row share a scale and a zero.
 *   scale_bf16  0: scales are binary16 bit patterns; 1: bfloat16 bit patterns.  Either
 *               is the binary32 step rounded to nearest even.
 *   zero_bits   8: zeros [N, K/group] bytes; 4: two zeros per byte over the flat
 *               [N, K/group] array (index i at byte i/2, even index in the low nibble),
 *               ceil(N*K/group / 2) bytes.
 *   symmetric   0: the asymmetric method of w4_quantize; 1: that of
 *               w4_quantize_symmetric (zero 8).
 * The codes and the binary32 step do not depend on the storage; {128, 0, 8, 0} is the
 * canonical format of w4_quantize and {128, 0, 8, 1} that of w4_quantize_symmetric.
 * The prepared layout of a format with group 128 and binary16 scales is the canonical
 * one (zeros are widened to the kernel's byte), so w4_gemv and w4_gemm take it; other
 * formats are read by w4_gemv_fmt only.  A format outside these values is refused with
 * W4_ERR_UNSUPPORTED.
 */
typedef struct {
    int32_t group;
    int32_t scale_bf16;
    int32_t zero_bits;
    int32_t symmetric;
} w4_format;

/* bytes of the zeros array of a format (0 for an invalid format or shape) */
size_t w4_zeros_bytes(int64_t N, int64_t K, const w4_format* fmt);

/*
 * w4_quantize_fmt -- w4_quantize / w4_quantize_symmetric in format *fmt.
 *   scales  out [N, K/group] 16-bit patterns of the format's scale type; 2-B aligned.
 *   zeros   out, w4_zeros_bytes(N, K, fmt) bytes.
 * Requires K % 128 == 0 (as every product does).  Other arguments, errors and d_status
 * bits as w4_quantize; with bfloat16 scales W4_STATUS_SCALE_OVERFLOW / _ZERO refer to
 * bfloat16 infinity / zero.
 */
w4_status w4_quantize_fmt(const void* W, w4_dtype wt, int64_t N, int64_t K,
                          const w4_format* fmt, uint8_t* packed, uint16_t* scales,
                          uint8_t* zeros, uint32_t* d_status, hipStream_t stream);

/*
 * w4_prepare_fmt / w4_unprepare_fmt -- the kernel layout of a format: the code region
 * of w4_prepare followed by one scale/zero word per row and group (four rows of one
 * group per 16 bytes).  Size w4_prepared_bytes_fmt(N, K, fmt); 256-B aligned.
 * w4_unprepare_fmt is the exact inverse.
 */
size_t w4_prepared_bytes_fmt(int64_t N, int64_t K, const w4_format* fmt);
w4_status w4_prepare_fmt(const uint8_t* packed, const uint16_t* scales, const uint8_t* zeros,
                         int64_t N, int64_t K, const w4_format* fmt, void* prepared,
                         size_t prepared_bytes, hipStream_t stream);
w4_status w4_unprepare_fmt(const void* prepared, int64_t N, int64_t K, const w4_format* fmt,
                           uint8_t* packed, uint16_t* scales, uint8_t* zeros,
                           hipStream_t stream);

/*
 * w4_gemv_fmt -- w4_gemv on the prepared layout of format *fmt (page "Weight
 * quantization", "How it works": scale * sum (code - zero) * x per group).  The
 * canonical-layout formats (group 128, binary16 scales) take w4_gemv's kernels; the
 * others run on its one-row (VALU) kernel at every M, in steps of up to four rows of x.
 * Arguments, limits and errors as w4_gemv.
 */
w4_status w4_gemv_fmt(const void* prepared, int64_t N, int64_t K, const w4_format* fmt,
                      const void* x, w4_dtype xt, int64_t M,
                      void* y, w4_dtype yt, hipStream_t stream);

/*
 * w4_gemm -- prefill-sized product Y[M, N] = X[M, K] * w_hat^T for any M >= 1
 * (page "LLM Quantization Architecture in Depth" › "Why fewer bits make
 * decoding faster": prefill is compute bound and weight-only formats must turn
 * weights back into 16-bit values before the matrix units).  The codes enter the
 * binary16 MFMA as the exact values q - zero and X as binary16 X * 2^-E[m] (E per
 * row, exact for every value within 2^28 of the row's largest); per group the f32
 * accumulator receives scale16 * P (page "Weight quantization", "How it works": the
 * dequantized weight (code - zero) * scale, one multiply per group), so no weight
 * and no activation is rounded.  Rows of X with a value outside that window are
 * recomputed by a fix-up pass with one binary32 FMA per weight.
 *   prepared  from w4_prepare.
 *   X         [M, K] bfloat16 row-major; 16-B aligned.
 *   Y         [M, N] row-major, binary32 or bfloat16; 4-B aligned.
 *   workspace device scratch of w4_gemm_workspace_bytes(M, N, K) bytes (the binary16
 *             copy of X, then per row its exponent and a window flag, each part
 *             256-B aligned), 16-B aligned; contents need no initialisation.  Calls
 *             sharing a workspace must be ordered.
 * Limits: N, K as w4_prepare and K <= W4_GEMM_MAX_K (the kernels address the operands of
 * a 128 x 256 tile with 32-bit offsets); 1 <= M <= 65535*128; at most 2^31 - 9 output
 * tiles of 128 x 256 (else W4_ERR_SHAPE; w4_gemm_workspace_bytes returns 0).
 */
size_t w4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
w4_status w4_gemm(const void* prepared, int64_t N, int64_t K,
                  const void* X, int64_t M, void* Y, w4_dtype yt,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * w4_gemm_noalloc -- w4_gemm for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc).  Same
 * product, same kernels, bit-identical Y; the workspace is a fixed array of
 * W4_GEMM_NOALLOC_MAX_WORKSPACE bytes in the library's device data, one copy per GPU,
 * held until the process ends.  The call allocates nothing (no hipMalloc, no allocating
 * library routine); its first call on a device looks up that device's copy once.
 *   Arguments, alignment and limits as w4_gemm, and in addition
 *   w4_gemm_workspace_bytes(M, N, K) <= W4_GEMM_NOALLOC_MAX_WORKSPACE, else
 *   W4_ERR_WORKSPACE before any device work (about M * K <= 8.3e6: M = 256 at
 *   K = 28672, M = 1024 at K = 8192).
 * Every call on one GPU shares that GPU's array, which keeps the last call's contents
 * (each call writes all it reads, nothing needs clearing): calls that may overlap on one
 * GPU -- on different streams without ordering, or from several threads -- race and give
 * undefined Y.  Order them on one stream, or use w4_gemm with workspaces of their own.
 */
#define W4_GEMM_NOALLOC_MAX_WORKSPACE (16u << 20)
w4_status w4_gemm_noalloc(const void* prepared, int64_t N, int64_t K,
                          const void* X, int64_t M, void* Y, w4_dtype yt, hipStream_t stream);

/*
 * W8A8 in FP8 E4M3 for prefill (page "LLM Quantization Architecture in Depth" › "Why fewer
 * bits make decoding faster": prefill is compute bound, so its arithmetic must be narrower,
 * with activations quantized too; › "Number formats, scales and granularity": E4M3, largest
 * value 448, dynamic per-token activation scales; page "Quantization" › "Code": FP8 E4M3
 * per-channel scaling, rounding to 3 mantissa bits with subnormals).
 *
 * w4_fp8_quantize_rows -- per-row E4M3 quantization of A [rows, K] (weights: one row per
 * output channel; activations: one row per token, at run time).
 *   scale[r] = max_k |A[r, k]| / 448 in binary64 (1 for an all-zero row), stored rounded to
 *   binary32; code = E4M3 byte of A[r, k] / scale[r] (binary64 quotient, magnitude capped at
 *   448, rounded halves-to-even on the grid of 3 mantissa bits of its binary exponent,
 *   exponents below -6 on the grid of -6).  Bytes are OCP E4M3: sign bit 7, exponent bits
 *   6..3 with bias 7, mantissa bits 2..0; 0x7E = 448; a value that rounds to zero keeps its
 *   sign (0x80); 0x7F/0xFF (NaN) are never written.
 *   A       [rows, K] row-major, binary32 (at = W4_F32) or bfloat16 (W4_BF16); 16-B aligned.
 *   codes   [rows, K] bytes, 16-B aligned.   scales  [rows] binary32, 4-B aligned.
 *   d_status  optional device word: bit 0 is OR-ed in if a row holds a non-finite value
 *             (its codes are then undefined).
 * Requires K a multiple of 128, 128 <= K <= W4_FP8_MAX_K.
 *
 * w4_fp8_gemm -- Y[m, n] = sx[m] * sw[n] * sum_k value(xq[m, k]) * value(wq[n, k]) on the
 * FP8 matrix cores with binary32 accumulation (each product of two E4M3 values is exact).
 *   xq, sx   [M, K] codes and [M] scales of the activations (w4_fp8_quantize_rows).
 *   wq, sw   [N, K] codes and [N] scales of the weights.
 *   Y        [M, N] row-major, binary32 (yt = W4_F32) or bfloat16 (W4_BF16); must not
 *            overlap the inputs.  Codes 16-B aligned, scales 4-B, Y 4-B (2-B for bf16).
 * Requires K a multiple of 128, 128 <= K <= W4_FP8_MAX_K.  Deterministic (no atomics).
 */
w4_status w4_fp8_quantize_rows(const void* A, w4_dtype at, int64_t rows, int64_t K,
                               uint8_t* codes, float* scales, uint32_t* d_status,
                               hipStream_t stream);
w4_status w4_fp8_gemm(const uint8_t* xq, const float* sx, int64_t M, const uint8_t* wq,
                      const float* sw, int64_t N, int64_t K, void* Y, w4_dtype yt,
                      hipStream_t stream);

/*
 * W8A8 in INT8 (page "Quantization" › "How it really works" and "Code": symmetric 8-bit
 * codes with one absmax scale per block; the architecture page names INT8 beside FP8 for
 * W8A8 prefill).
 *
 * w4_int8_quantize_rows -- per-row symmetric INT8: step[r] = max_k |A[r, k]| / 127 in
 *   binary64 (1 for an all-zero row), stored rounded to binary32; code = A[r, k] / step[r]
 *   in binary64, rounded to the nearest integer with halves to even, clamped to
 *   [-128, 127].  Arguments, alignment, limits and status as w4_fp8_quantize_rows, with
 *   codes [rows, K] int8.
 * w4_int8_gemm -- Y[m, n] = sx[m] * sw[n] * sum_k xq[m, k] * wq[n, k] on the INT8 matrix
 *   cores; the sums are exact int32 (|sum| <= K * 128 * 128 < 2^31 for K <= W4_FP8_MAX_K),
 *   then converted to binary32 and scaled.  Arguments, alignment and limits as
 *   w4_fp8_gemm.  Deterministic.
 */
w4_status w4_int8_quantize_rows(const void* A, w4_dtype at, int64_t rows, int64_t K,
                                int8_t* codes, float* scales, uint32_t* d_status,
                                hipStream_t stream);
w4_status w4_int8_gemm(const int8_t* xq, const float* sx, int64_t M, const int8_t* wq,
                       const float* sw, int64_t N, int64_t K, void* Y, w4_dtype yt,
                       hipStream_t stream);

/*
 * Operators between the products of a decoder layer.  They take what the products write and
 * write what the products take: binary32 or bfloat16 rows, or 8-bit codes with row scales.
 *
 * w4_rmsnorm -- root-mean-square norm of rows, with the residual's addition.
 *   h = x + residual, rounded to the residual's type and written to residual_out;
 *   y[i] = h[i] * s * weight[i], s = 1 / sqrt(mean(h^2) + eps) (sum in binary64, s and the
 *   products in binary32).  Without a residual h = x.
 *   x             [rows, K] binary32 or bfloat16.   weight  [K] binary32 or bfloat16.
 *   residual      [rows, K] binary32 or bfloat16, or NULL.
 *   residual_out  [rows, K] of the residual's type; may be residual itself (in place); NULL
 *                 with residual, and only then.
 *   y             [rows, K] binary32 or bfloat16.
 * w4_rmsnorm_fp8, w4_rmsnorm_int8 -- the same y, quantized per row without being stored: codes
 *   [rows, K] and scales [rows] as w4_fp8_quantize_rows / w4_int8_quantize_rows write them for
 *   the binary32 y, bit for bit; d_status (optional) receives W4_STATUS_NONFINITE where a row
 *   holds a value that is not finite (the row's codes say nothing then; 0x7F is not among them).
 * Requires rows >= 1, K a multiple of 128, 128 <= K <= W4_ROWS_MAX_K, eps finite and > 0
 * (W4_ERR_VALUE).  All arrays 16-B aligned (scales, d_status 4-B); outputs must not overlap
 * inputs except residual_out as stated.  Deterministic.
 */
w4_status w4_rmsnorm(const void* x, w4_dtype xt, const void* residual, void* residual_out,
                     w4_dtype rt, const void* weight, w4_dtype wt, float eps, int64_t rows,
                     int64_t K, void* y, w4_dtype yt, hipStream_t stream);
w4_status w4_rmsnorm_fp8(const void* x, w4_dtype xt, const void* residual, void* residual_out,
                         w4_dtype rt, const void* weight, w4_dtype wt, float eps, int64_t rows,
                         int64_t K, uint8_t* codes, float* scales, uint32_t* d_status,
                         hipStream_t stream);
w4_status w4_rmsnorm_int8(const void* x, w4_dtype xt, const void* residual, void* residual_out,
                          w4_dtype rt, const void* weight, w4_dtype wt, float eps, int64_t rows,
                          int64_t K, int8_t* codes, float* scales, uint32_t* d_status,
                          hipStream_t stream);

/*
 * w4_silu_mul -- the gate between the fused gate|up product and the down product:
 *   y[r, i] = g / (1 + exp(-g)) * u in binary32, g = gate_up[r, i], u = gate_up[r, F + i].
 *   gate_up  [rows, 2F] binary32 or bfloat16.   y  [rows, F] binary32 or bfloat16.
 * w4_silu_mul_fp8, w4_silu_mul_int8 -- the same y as codes [rows, F] and scales [rows], as above.
 * Requires F a multiple of 128, 128 <= F <= W4_ROWS_MAX_K.  Alignment, errors as w4_rmsnorm.
 */
w4_status w4_silu_mul(const void* gate_up, w4_dtype gt, int64_t rows, int64_t F, void* y,
                      w4_dtype yt, hipStream_t stream);
w4_status w4_silu_mul_fp8(const void* gate_up, w4_dtype gt, int64_t rows, int64_t F,
                          uint8_t* codes, float* scales, uint32_t* d_status, hipStream_t stream);
w4_status w4_silu_mul_int8(const void* gate_up, w4_dtype gt, int64_t rows, int64_t F,
                           int8_t* codes, float* scales, uint32_t* d_status, hipStream_t stream);

/*
 * A paged cache of keys and values.  Row j of page p and kv head h is row
 * (p * kv_heads + h) * page_size + j of k and v, head_dim elements; a slot is
 * p * page_size + j.
 *   type       W4_CACHE_BF16: bfloat16 rows; W4_CACHE_FP8: E4M3 codes, one binary32 scale per
 *              row in k_scales and v_scales [pages, kv_heads, page_size] (NULL otherwise).
 *   page_size  a power of two, 16 to 4096.   head_dim  64 or 128.   kv_heads  1 to 1024.
 * k and v 16-B aligned, scales 4-B.  W4_ERR_UNSUPPORTED for another type, page size or head
 * dimension.  pages >= 1; kv_heads * page_size * pages < 2^40.
 */
typedef enum { W4_CACHE_BF16 = 0, W4_CACHE_FP8 = 1 } w4_cache_type;
typedef struct {
    void* k;
    void* v;
    float* k_scales;
    float* v_scales;
    int64_t pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t type;
} w4_kv_cache;

/*
 * Rotary positions.  Pair i (0 <= i < rotary_dim / 2) of a head turns by position * f[i], with
 * f[i] = base^(-2 i / rotary_dim) and, for contexts longer than the original_positions trained:
 *   W4_ROPE_NONE    f as it is.
 *   W4_ROPE_LINEAR  f / factor.
 *   W4_ROPE_BANDS   by the turns t = original_positions * f / (2 pi): f / factor where t <= low,
 *                   f where t >= high, between them f * (k + (1 - k) / factor) with
 *                   k = (t - low) / (high - low).
 *   W4_ROPE_RAMP    f * (1 - r + r / factor), r rising from 0 to 1 between the pairs
 *                   floor(c(high)) (at least 0) and ceil(c(low)) (at most rotary_dim - 1;
 *                   0.001 more if both are the same), c(t) = rotary_dim *
 *                   ln(original_positions / (2 pi t)) / (2 ln base); r is 1 for all pairs where
 *                   ceil(c(low)) < 0 and 0 where floor(c(high)) > rotary_dim - 1; cosines and
 *                   sines are multiplied by the amplitude 1 + 0.1 ln(factor).
 *   rotary_dim   elements of a head that turn: a multiple of 16 (the rest stays as it is).
 *   interleaved  0: pairs (i, i + rotary_dim / 2); 1: pairs (2i, 2i + 1).
 * Requires base > 1, factor >= 1 (but for NONE), and for BANDS and RAMP 0 < low < high and
 * original_positions >= 1; all finite (W4_ERR_VALUE).
 *
 * w4_rope_frequencies -- f on the host, binary64: freqs [rotary_dim / 2]; *amplitude (may be
 *   NULL) is 1 except for RAMP.  No device work.
 *
 * w4_rope_cache -- rotates the rows of the fused q|k|v product and stores K and V in the cache.
 *   qkv        [T, (heads + 2 kv_heads) * head_dim] binary32 or bfloat16: the query heads, the
 *              key heads, the value heads; 16-B aligned.
 *   positions  [T] device.   slots  [T] device: where the token's K and V go.  A token with a
 *              negative slot is padding: neither its q nor the cache is written; one with a slot
 *              past the cache is skipped too and sets W4_STATUS_PAGE.  Slots must differ from
 *              each other (two tokens with one slot leave either's values, element by element).
 *   d_freqs    [rotary_dim / 2] device binary64 from w4_rope_frequencies; 8-B aligned.
 *   q          out [T, heads, head_dim] bfloat16; 16-B aligned; must not overlap qkv.
 * Angles are formed in binary64, rotations in binary32, results rounded once: q and a bfloat16
 * cache to nearest even, rows of an E4M3 cache as w4_fp8_quantize_rows with K = head_dim would
 * the binary32 row (d_status: W4_STATUS_NONFINITE).  Requires 1 <= T <= W4_MAX_TOKENS,
 * heads a multiple of kv_heads, at most 65536, T * heads < 2^26, rotary_dim <= head_dim.
 */
typedef enum { W4_ROPE_NONE = 0, W4_ROPE_LINEAR = 1, W4_ROPE_BANDS = 2, W4_ROPE_RAMP = 3 } w4_rope_scaling;
typedef struct {
    int32_t rotary_dim;
    int32_t interleaved;
    int32_t scaling;
    int32_t reserved;            /* 0 */
    double base;
    double factor;
    double low;
    double high;
    int64_t original_positions;
} w4_rope;
w4_status w4_rope_frequencies(const w4_rope* rope, double* freqs, double* amplitude);
w4_status w4_rope_cache(const void* qkv, w4_dtype xt, int64_t T, int64_t heads,
                        const w4_kv_cache* cache, const int32_t* positions, const int64_t* slots,
                        const w4_rope* rope, const double* d_freqs, void* q, uint32_t* d_status,
                        hipStream_t stream);

/*
 * w4_block_tables -- places the new tokens of a batch of requests in pages, on the device.
 * Request b has lens_in[b] cached tokens in the pages that row b of block_table names, and
 * new_lens[b] tokens more in this step; the batch packs the new tokens request by request.
 *   free_pages   [free_capacity] page numbers, of which the first *free_count_in are free; pages
 *                are taken from the end.
 *   lens_out     [B] lens_in + new_lens (may be lens_in).
 *   free_count_out  pages left (may be free_count_in).
 *   block_table  [B, max_pages], in and out: entries of newly taken pages are written.
 *   cu_q         out [B + 1]: first new token of each request in the batch; cu_q[B] their number.
 *   positions, slots  out [T]: of each new token; 0 and -1 behind the last one.
 * A request whose length is negative or whose tokens do not end within T (W4_STATUS_LENGTH), or
 * whose pages do not fit its table row, or are not there once the requests ahead of it are
 * served (W4_STATUS_PAGES_SHORT), is left as it is: it takes no page, its length stays and its
 * tokens get position 0 and slot -1; cu_q still counts them, the requests behind it are served.  A negative new length counts as
 * none, a taken page with a negative number gives slot -1.
 * Requires 1 <= B <= W4_MAX_SEQUENCES, 1 <= T <= W4_MAX_TOKENS, page_size as in w4_kv_cache,
 * max_pages * page_size <= W4_MAX_CONTEXT, free_capacity >= 0; int32 arrays 4-B aligned, slots
 * 8-B.  Outputs must not overlap inputs except as stated.  Deterministic.
 */
w4_status w4_block_tables(const int32_t* new_lens, const int32_t* lens_in, int64_t B,
                          const int32_t* free_pages, int64_t free_capacity,
                          const int32_t* free_count_in, int32_t* lens_out,
                          int32_t* free_count_out, int32_t* block_table, int64_t max_pages,
                          int32_t page_size, int32_t* cu_q, int32_t* positions, int64_t* slots,
                          int64_t T, uint32_t* d_status, hipStream_t stream);

/*
 * w4_paged_attention -- attention of the new tokens of each request over its cached tokens, the
 * new ones among them (w4_rope_cache has stored them):
 *   o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale * q . k_j), over the keys j <= position, with
 *   a window the last `window` of them.
 * Token t of request b (rows cu_q[b] .. cu_q[b+1] of the batch) has position
 * lens[b] - (cu_q[b+1] - cu_q[b]) + t.  Query head h reads kv head h / (heads / kv_heads).
 *   q            [T, heads, head_dim] bfloat16; 16-B aligned.
 *   block_table  [B, max_pages] device; cu_q [B + 1], lens [B] device (as w4_block_tables
 *                writes them: lens counts the new tokens; one past the table counts as its end).
 *   scale        finite, > 0.   window  0 (none) or >= 1.   (else W4_ERR_VALUE)
 *   o            out [T, heads, head_dim] bfloat16; 16-B aligned; must not overlap q.  Rows that
 *                belong to no request stay as they are; a row that sees no key gets zeros.
 *   workspace    w4_paged_attention_workspace_bytes(...) bytes of device scratch (may be 0),
 *                16-B aligned; contents need no initialisation.  Calls (and captured graphs)
 *                sharing a workspace must be ordered.
 * A key that a row sees in a page that the cache does not have reads as zeros (K and V) and sets
 * W4_STATUS_PAGE in d_status (optional).  Table entries of pages that lie wholly before every row's
 * window, or behind a request's keys, are not looked at: such pages may have been given back.
 * What lies in the cache behind a request's keys, and at keys that a row does not see, does not
 * reach the row, NaN and infinities included.
 * Scores, softmax sums and outputs are formed in binary32 and o is rounded once.  V is multiplied by
 * weights held in two bfloat16 parts (2^-16) for every request where T = B or all rows together
 * (T times heads / kv_heads) are at most 32, else for requests of at most 32 rows, 64 with an E4M3
 * cache or where 2 * B * kv_heads <= 256; for the others by weights rounded to bfloat16 (2^-8).  A
 * request's last bits may so depend on the batch that it is in.
 * T = B is taken for one token a request: any lengths give right results, but a long prompt there
 * reads its keys once for every 16 rows.  Where prompts and idle places may add up to T = B, one
 * padding row more (T = B + 1) avoids that.
 * Deterministic; the split of the work depends on the arguments and lengths only.
 * Requires 1 <= T <= W4_MAX_TOKENS, 1 <= B <= W4_MAX_SEQUENCES, heads a multiple of kv_heads, at
 * most 65536, T * heads < 2^26, 1 <= max_pages, max_pages * page_size <= W4_MAX_CONTEXT.
 */
size_t w4_paged_attention_workspace_bytes(int64_t T, int64_t heads, const w4_kv_cache* cache,
                                          int64_t B, int64_t max_pages);
w4_status w4_paged_attention(const void* q, int64_t T, int64_t heads, const w4_kv_cache* cache,
                             const int32_t* block_table, int64_t max_pages, const int32_t* cu_q,
                             const int32_t* lens, int64_t B, float scale, int64_t window, void* o,
                             void* workspace, size_t workspace_bytes, uint32_t* d_status,
                             hipStream_t stream);

/*
 * w4_stream_read -- measurement probe, not part of the method: reads `bytes` bytes of
 * device memory at `buf` once with plain streaming loads (8192 workgroups, each a
 * contiguous share, non-temporal 16-byte loads) and discards them, so a product's rate
 * can be compared with a kernel that only reads the same bytes in the same launch
 * pattern (page "Weight quantization", "Complexity and constants": decode time is bytes
 * read / bandwidth).
 *   buf   device memory, 16-B aligned; bytes a non-zero multiple of 16.
 *   sink  a device word the kernel may overwrite (it almost never does); 4-B aligned.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_ARCH, W4_ERR_HIP.
 */
w4_status w4_stream_read(const void* buf, size_t bytes, uint32_t* sink, hipStream_t stream);

/* Text of a status code (static storage). */
const char* w4_status_string(w4_status s);
/* Message of the last W4_ERR_HIP on the calling thread ("" if none). */
const char* w4_last_hip_error(void);
/* W4_FORMAT_VERSION of the library (prepared-layout version). */
int w4_format_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */
