/*
 * qlin.h -- C ABI of libqlin.so, the MI355X (gfx950) quantized linear layer.
 *
 * A linear layer computes Y = X W^T with X [m, k] (activations, row-major,
 * k contiguous) and W [n, k] (weights, row-major).  Two phases use two
 * weight formats, as in Disaggregated Quantization (singularity-lens: the
 * format-disaggregated variant runs prefill with NVFP4 compute and decode on
 * a weight-only path) and Mix-Quant (gist.science, section 2 "Method":
 * NVFP4 W4A4 prefill):
 *
 *   prefill  quantize_nvfp4(X) -> gemm_w4a4(codes, scales, s_t, W packed NVFP4)
 *   decode   gemm_w4a16(X bf16, W packed INT4 group-128)
 *            gemm_lut2 (X bf16, W packed 2-bit codebook)
 *
 * Offline weight preparation (not timed; the Disaggregated Quantization page
 * notes that its LUT speed comparison leaves out weight-format conversion):
 *   NVFP4: quantize_nvfp4(W fp32) then repack_weights(QL_NVFP4, ...)
 *   INT4 : quantize_int4_g128(W)  then repack_weights(QL_INT4_G128, ...)
 *   LUT2 : fit_lut2(W)            then repack_weights(QL_LUT2, ...)
 * The MARLIN article (abeam.tech, "オフラインで並べ替えておく") motivates
 * repacking weights and scales offline into the order the kernel reads.
 *
 * Conventions for every call
 *   - Pointers are DEVICE pointers unless stated otherwise; `stream` is a
 *     hipStream_t passed as void* (NULL = the default stream).
 *   - Every call is asynchronous on `stream`.  No call allocates, frees or
 *     synchronises; the caller owns every buffer and keeps it alive until the
 *     stream work that uses it has completed.
 *   - Argument errors are reported synchronously, before any launch, as a
 *     ql_status; a failed launch returns QL_EHIP.  No call aborts and no C++
 *     exception crosses this interface.
 *   - m == 0 (or n == 0 for weight preparation) returns QL_OK and does nothing.
 *   - Buffers must be 16-byte aligned and contiguous.
 *   - Results are deterministic: fixed reduction order, no floating-point
 *     atomics, so repeated runs are bitwise identical.
 *   - Inputs must be finite (NaN/Inf are outside the method's domain).
 *   - Calls are stateless and may be issued from several host threads.
 */
#ifndef QLIN_H
#define QLIN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QL_OK = 0,
  QL_EINVAL = 1,     /* null pointer, negative size or unknown flag          */
  QL_ESHAPE = 2,     /* shape constraint violated (see each call)            */
  QL_EALIGN = 3,     /* pointer not 16-byte aligned                          */
  QL_EDTYPE = 4,     /* unknown or unsupported dtype                         */
  QL_EWORKSPACE = 5, /* workspace or output buffer too small                 */
  QL_EHIP = 6,       /* a HIP launch failed                                  */
  QL_EFORMAT = 7     /* unknown weight format                                */
} ql_status;

typedef enum { QL_F32 = 0, QL_BF16 = 1 } ql_dtype;
typedef enum { QL_NVFP4 = 0, QL_INT4_G128 = 1, QL_LUT2 = 2, QL_INT4_SP24 = 3 } ql_format;

/* quantize_nvfp4 flag: read *tensor_scale as the (calibrated) tensor scale
 * instead of computing it from the tensor's absolute maximum. */
#define QL_STATIC_SCALE 1u

/* Human-readable name of a status code (static string; never NULL). */
const char *ql_status_str(int status);

/* Layout version of packed weight blobs produced by this library. */
int ql_version(void);

/* ------------------------------------------------------------------------
 * NVFP4 quantization, round to nearest (Mix-Quant, section 2: NVFP4 keeps a
 * local scale per 16-element group plus a tensor-level scale, and plain RTN
 * is enough for the format).  Element codes are E2M1, group scales E4M3
 * (OCP E4M3FN), the tensor scale fp32.  Operation order, all binary32 and
 * correctly rounded:
 *   amax = max|x|;  s_t = amax / 2688;  d = 6 * s_t
 *   per 16-group: s_g = E4M3(max|x_g| / d)   (RNE, saturating at 448; 0 if d == 0)
 *   p = s_g * s_t;  p == 0 -> codes are the sign bits alone
 *   else inv = 1 / p;  code = E2M1(x * inv)  (RNE, ties to even, saturating at 6)
 *
 * x            [rows, cols], dtype QL_F32 or QL_BF16.
 * codes        out [rows, cols/2]  : byte j holds column 2j (low nibble) and 2j+1.
 * scales       out [rows, cols/16] : E4M3 bit patterns.
 * tensor_scale device fp32 scalar: out (s_t) by default; in when
 *              flags & QL_STATIC_SCALE.
 * workspace    >= quantize_nvfp4_workspace(rows, cols) bytes of device memory
 *              (per-block partial maxima; may be NULL when that size is 0).
 * Shapes: cols % 16 == 0.  Errors: QL_EINVAL, QL_ESHAPE, QL_EALIGN,
 * QL_EDTYPE, QL_EWORKSPACE, QL_EHIP.
 * ---------------------------------------------------------------------- */
size_t quantize_nvfp4_workspace(int64_t rows, int64_t cols);
int quantize_nvfp4(const void *x, int x_dtype, int64_t rows, int64_t cols,
                   uint8_t *codes, uint8_t *scales, float *tensor_scale,
                   unsigned flags, void *workspace, size_t workspace_bytes,
                   void *stream);

/* ------------------------------------------------------------------------
 * quantize_nvfp4 for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation):
 * the same computation, arguments, outputs and errors as quantize_nvfp4,
 * without the workspace.  The per-block partial maxima go to a 4 KiB array
 * (1024 x uint32) that the library keeps in each GPU's memory for the life of
 * the process; its device address is looked up once per device, at the first
 * call on that device (with that device current).  The call allocates and
 * frees nothing.  Nothing in the array needs clearing: every partial a call
 * reads is written by that call's own first pass.
 *
 * Every call on one GPU shares that GPU's array, which keeps the last call's
 * contents: calls that may overlap on one GPU (issued to different streams
 * without an ordering between them) race on it and may compute a wrong
 * tensor scale.  Calls on one stream are ordered and safe.
 *
 * Errors: as quantize_nvfp4 (no QL_EWORKSPACE for a missing workspace);
 * QL_EWORKSPACE if the input would need more than 1024 partial maxima (the
 * first pass never runs more than 1024 blocks, so no shape the other checks
 * accept does); QL_EHIP if the array's address cannot be looked up.
 * ---------------------------------------------------------------------- */
int quantize_nvfp4_noalloc(const void *x, int x_dtype, int64_t rows, int64_t cols,
                           uint8_t *codes, uint8_t *scales, float *tensor_scale,
                           unsigned flags, void *stream);

/* ------------------------------------------------------------------------
 * Symmetric INT4 weight quantization with groups of 128 along k (MARLIN
 * article, "データの扱い方": 4-bit weights, group size 128).  Per row and
 * group: a = max|w|; s = bf16(a / 7) (binary32 division, then RNE to bf16);
 * q = clamp(rne(w / s), -7, 7) (binary32 division by the stored scale);
 * q = 0 when s == 0.
 *
 * w       [n, k] fp32.
 * codes   out [n, k/2]   : u = q + 8 (1..15), column 2j in the low nibble.
 * scales  out [n, k/128] : bf16 bit patterns.
 * Shapes: k % 128 == 0.  Errors: QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EHIP.
 * ---------------------------------------------------------------------- */
int quantize_int4_g128(const float *w, int64_t n, int64_t k, uint8_t *codes,
                       uint16_t *scales, void *stream);

/* ------------------------------------------------------------------------
 * 2:4 structured-sparse INT4 group-128 quantization (MARLIN article,
 * "データの扱い方" and "実験と結果": Sparse-MARLIN combines the group-128
 * INT4 format with 2:4 structured sparsity).  The pages do not say how the
 * pattern is chosen; here: in every run of four consecutive columns of a row
 * the two entries of largest |w| are kept (ties to the lower column) and the
 * other two are set to zero, then the row is quantized exactly as by
 * quantize_int4_g128 (so pruned entries have q = 0, u = 8).
 *
 * Arguments, outputs, shapes and errors as quantize_int4_g128; the codes are
 * in the same dense canonical layout, with at most two nonzero q per quad.
 * ---------------------------------------------------------------------- */
int quantize_int4_g128_sp24(const float *w, int64_t n, int64_t k, uint8_t *codes,
                            uint16_t *scales, void *stream);

/* ------------------------------------------------------------------------
 * 2-bit codebook (LUT2) fit: per weight row, 4 centroids by 10 Lloyd
 * K-means iterations (KLLM article, aibr.jp, sections 1 and 3: K-means
 * quantization into centroids plus an index matrix; Disaggregated
 * Quantization: 2-bit LUT decode weights).  Centroids start at the
 * quantiles sorted(w)[floor((2j+1) k / 8)]; each iteration assigns every
 * weight to the nearest centroid in fp64 (ties to the lower index) and moves
 * each non-empty centroid to the fp64 mean of its weights, summed in
 * ascending column order.  Centroids are then rounded to bf16 (via binary32)
 * and every weight is re-assigned to the nearest rounded centroid.
 *
 * w          [n, k] fp32.
 * idx        out [n, k/4] : column 4b+i in bits 2i..2i+1 of byte b.
 * centroids  out [n, 4]   : bf16 bit patterns, ascending.
 * workspace  >= fit_lut2_workspace(n, k) bytes.
 * Shapes: k % 128 == 0, k <= 32768.  Errors: QL_EINVAL, QL_ESHAPE,
 * QL_EALIGN, QL_EWORKSPACE, QL_EHIP.
 * ---------------------------------------------------------------------- */
size_t fit_lut2_workspace(int64_t n, int64_t k);
int fit_lut2(const float *w, int64_t n, int64_t k, uint8_t *idx,
             uint16_t *centroids, void *workspace, size_t workspace_bytes,
             void *stream);

/* ------------------------------------------------------------------------
 * Offline repack of canonical quantized weights into the private gfx950
 * operand order read by the GEMM kernels (an opaque, versioned blob with a
 * header).  Pure data movement: values are not changed.
 *
 * fmt            QL_NVFP4 | QL_INT4_G128 | QL_LUT2 | QL_INT4_SP24.
 * codes          canonical codes as produced by quantize_nvfp4 (NVFP4, from
 *                W [n,k]), quantize_int4_g128 / quantize_int4_g128_sp24, or
 *                fit_lut2.  QL_INT4_SP24 keeps, in each run of four
 *                consecutive columns, the two codes of largest |q| (ties to
 *                the lower column) with their positions: every nonzero code
 *                when the codes come from quantize_int4_g128_sp24.
 * scales_or_lut  E4M3 [n, k/16] | bf16 [n, k/128] (INT4 and INT4_SP24) |
 *                bf16 centroids [n, 4].
 * tensor_scale   device fp32 s_t of the weights (NVFP4 only, else NULL);
 *                copied into the blob.
 * packed         out, >= repack_weights_bytes(fmt, n, k) bytes.
 * Shapes: n % 16 == 0, k % 128 == 0.  Errors: QL_EINVAL, QL_ESHAPE,
 * QL_EALIGN, QL_EFORMAT, QL_EWORKSPACE, QL_EHIP.
 * ---------------------------------------------------------------------- */
size_t repack_weights_bytes(int fmt, int64_t n, int64_t k);
int repack_weights(int fmt, int64_t n, int64_t k, const uint8_t *codes,
                   const void *scales_or_lut, const float *tensor_scale,
                   void *packed, size_t packed_bytes, void *stream);

/* ------------------------------------------------------------------------
 * W4A4 prefill GEMM (Mix-Quant, section 2, system-level deployment: the
 * prefill worker runs the NVFP4 W4A4 path):
 *   Y[m,n] = s_tA s_tW sum_g sA[m,g] sW[n,g] sum_{k in g} E2M1(a[m,k]) E2M1(w[n,k])
 * computed with exact fp16 dequantized operands on gfx950 MFMA and fp32
 * accumulation.
 *
 * a_codes, a_scales, a_tensor_scale : output of quantize_nvfp4 on X [m, k].
 * w_packed  NVFP4 blob of W [n, k] from repack_weights.
 * y         out [m, n], y_dtype QL_F32 or QL_BF16 (RNE).
 * Shapes: n % 16 == 0, k % 128 == 0, m >= 0.  n and k must be the values the
 * blob was packed with: the kernels read the blob header first, and a blob
 * that is not an NVFP4 blob of this (n, k) is not read further and leaves y
 * untouched (the host cannot detect it without synchronising, so no status
 * reports it).  Errors: QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EDTYPE,
 * QL_EHIP.
 * ---------------------------------------------------------------------- */
int gemm_w4a4(const uint8_t *a_codes, const uint8_t *a_scales,
              const float *a_tensor_scale, const void *w_packed, int64_t m,
              int64_t n, int64_t k, void *y, int y_dtype, void *stream);

/* ------------------------------------------------------------------------
 * gemm_w4a4 with a caller-provided workspace that lets the last, partly
 * filled round of 256 x 256 output tiles (one tile per compute unit and
 * round), or a whole problem of at most half a round, be split along k over
 * the idle compute units: fp32 partial tiles go to the workspace and a
 * second launch adds them in a fixed order (so results stay deterministic;
 * they differ from gemm_w4a4's in fp32 rounding only).  Same arithmetic
 * definition and arguments as gemm_w4a4, plus:
 *
 * workspace        device memory of at least gemm_w4a4_workspace(m, n, k)
 *                  bytes, 16-byte aligned, not read before it is written;
 *                  may be NULL (then the call is gemm_w4a4).  Calls that
 *                  share one workspace must be ordered (same stream).
 * gemm_w4a4_workspace returns 0 when no split applies to the shape (the
 * tiles fill whole rounds, the last round is more than half full, or k is
 * too short for two slices), and depends on the current device's
 * compute-unit count.
 * Errors: as gemm_w4a4, and QL_EWORKSPACE when workspace is non-NULL and
 * smaller than gemm_w4a4_workspace(m, n, k).
 * ---------------------------------------------------------------------- */
size_t gemm_w4a4_workspace(int64_t m, int64_t n, int64_t k);
int gemm_w4a4_ws(const uint8_t *a_codes, const uint8_t *a_scales,
                 const float *a_tensor_scale, const void *w_packed, int64_t m,
                 int64_t n, int64_t k, void *y, int y_dtype, void *workspace,
                 size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Quantize folded into the W4A4 GEMM (Mix-Quant technical summary, section 2,
 * system-level deployment: the prefill path quantizes activations to NVFP4
 * and runs the W4A4 product): the result of quantize_nvfp4 on bf16 X followed
 * by gemm_w4a4 on its outputs, without materialising the activation codes.
 * The GEMM kernel quantizes each activation tile as it loads it, with the
 * quantizer's own operation order (quantize_nvfp4 above), so the codes, the
 * tensor scale and y are bit-identical to that pair of calls wherever
 * gemm_w4a4 runs its small-batch kernel (m <= 32) or its 128-row-tile kernel
 * (m <= 128, or few 256 x 256 tiles), whose quantizing variants this call
 * runs; gemm_w4a4's 256 x 256 kernel accumulates in another k order and
 * agrees in fp32 rounding only.  Every block that uses an activation group
 * quantizes it again (once per block of output columns): at m <= 32 this
 * costs about as much as the pair of calls (less on narrow layers), above
 * that about twice as much.  It is for callers that want no activation
 * codes in memory, or a single launch with a static tensor scale.  Two
 * launches (the amax pass, then the GEMM), or one with a static tensor
 * scale.
 *
 * x_bf16          [m, k] bf16, 16-byte aligned.
 * a_tensor_scale  device fp32 s_t of X: out by default; in when
 *                 flags & QL_STATIC_SCALE (as quantize_nvfp4).
 * w_packed        NVFP4 blob of W [n, k] from repack_weights.
 * y               out [m, n], y_dtype QL_F32 or QL_BF16 (RNE).
 * workspace       >= quantize_gemm_w4a4_workspace(m, k) bytes of device
 *                 memory (the amax pass's partial maxima), 16-byte aligned;
 *                 unused (may be NULL) with QL_STATIC_SCALE.  Calls sharing a
 *                 workspace must be ordered (same stream).
 * Shapes: n % 16 == 0, k % 128 == 0, m >= 0.  A blob that is not an NVFP4
 * blob of this (n, k) leaves y and the tensor scale untouched (as gemm_w4a4).
 * Errors: QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EDTYPE, QL_EWORKSPACE, QL_EHIP.
 * ---------------------------------------------------------------------- */
size_t quantize_gemm_w4a4_workspace(int64_t m, int64_t k);
int quantize_gemm_w4a4(const void *x_bf16, int64_t m, int64_t k, float *a_tensor_scale,
                       unsigned flags, const void *w_packed, int64_t n, void *y,
                       int y_dtype, void *workspace, size_t workspace_bytes,
                       void *stream);

/* ------------------------------------------------------------------------
 * W4A16 decode GEMV / skinny GEMM (weight-only decode: Disaggregated
 * Quantization; MARLIN article, "どんな技術か": 16-bit activations times
 * INT4 weights, dequantized in registers):
 *   Y[m,n] = sum_g s[n,g] sum_{k in g} x[m,k] q[n,k]   (fp32 accumulation)
 * x        [m, k] bf16.   w_packed: INT4 blob from repack_weights.
 * y        out [m, n], QL_F32 or QL_BF16.
 * Tuned for m <= 32 (decode batches); any m >= 0 is accepted.
 * Shapes: n % 16 == 0, k % 128 == 0.  Errors as gemm_w4a4.
 * The kernels read the blob header together with their first weight loads
 * and test it (magic, version, format, n, k) before their first store: a blob
 * that is not one of this format packed for this (n, k) leaves y untouched
 * (the host cannot detect it without synchronising, so no status reports
 * it).  It is read as a blob of this format and shape first, so the buffer
 * must hold at least repack_weights_bytes(format, n, k) bytes.
 * ---------------------------------------------------------------------- */
int gemm_w4a16(const void *x_bf16, const void *w_packed, int64_t m, int64_t n,
               int64_t k, void *y, int y_dtype, void *stream);

/* ------------------------------------------------------------------------
 * gemm_w4a16 with a caller-provided workspace that lets the k dimension be
 * split over blocks: each block takes one k slice of several 16-row weight
 * tiles, so the activation fragments it loads serve all of them (without a
 * split, narrow-n shapes run one row tile per block, and every block loads
 * the whole activation), and a second launch adds the slices' fp32 partial
 * sums in slice order (deterministic; results differ from gemm_w4a16's in
 * fp32 rounding only).  Same arithmetic definition and arguments as
 * gemm_w4a16, plus:
 *
 * workspace        device memory of at least gemm_w4a16_workspace(m, n, k)
 *                  bytes, 16-byte aligned, not read before it is written;
 *                  may be NULL (then the call is gemm_w4a16).  Calls that
 *                  share one workspace must be ordered (same stream).
 * gemm_w4a16_workspace returns 0 when no split applies to the shape (it
 * applies to 8 < m <= 32 with k > 4096, where it was measured faster), and
 * depends on the current device's compute-unit count.
 * Errors: as gemm_w4a16, and QL_EWORKSPACE when workspace is non-NULL and
 * smaller than gemm_w4a16_workspace(m, n, k).
 * ---------------------------------------------------------------------- */
size_t gemm_w4a16_workspace(int64_t m, int64_t n, int64_t k);
int gemm_w4a16_ws(const void *x_bf16, const void *w_packed, int64_t m, int64_t n,
                  int64_t k, void *y, int y_dtype, void *workspace,
                  size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * LUT2 decode GEMV (2-bit codebook weights; KLLM article section 3 and
 * Disaggregated Quantization's LUT2 decode):
 *   Y[m,n] = sum_k x[m,k] C[n, idx[n,k]]   (fp32 accumulation)
 * x        [m, k] bf16.   w_packed: LUT2 blob from repack_weights.
 * y        out [m, n], QL_F32 or QL_BF16.
 * Shapes: n % 16 == 0, k % 128 == 0.  Errors as gemm_w4a4.
 * The kernels read the blob header together with their first weight loads
 * and test it (magic, version, format, n, k) before their first store: a blob
 * that is not one of this format packed for this (n, k) leaves y untouched
 * (the host cannot detect it without synchronising, so no status reports
 * it).  It is read as a blob of this format and shape first, so the buffer
 * must hold at least repack_weights_bytes(format, n, k) bytes.
 * ---------------------------------------------------------------------- */
int gemm_lut2(const void *x_bf16, const void *w_packed, int64_t m, int64_t n,
              int64_t k, void *y, int y_dtype, void *stream);

/* ------------------------------------------------------------------------
 * gemm_lut2 with a caller-provided workspace for a k split over blocks, as
 * gemm_w4a16_ws: same arithmetic definition and arguments as gemm_lut2, plus
 * the workspace (at least gemm_lut2_workspace(m, n, k) bytes, 16-byte
 * aligned, not read before it is written; NULL makes the call gemm_lut2;
 * calls sharing a workspace must be ordered).  gemm_lut2_workspace returns 0
 * when no split applies.  Errors: as gemm_lut2, and QL_EWORKSPACE when the
 * workspace is non-NULL and too small.
 * ---------------------------------------------------------------------- */
size_t gemm_lut2_workspace(int64_t m, int64_t n, int64_t k);
int gemm_lut2_ws(const void *x_bf16, const void *w_packed, int64_t m, int64_t n,
                 int64_t k, void *y, int y_dtype, void *workspace,
                 size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * 2:4 sparse W4A16 decode GEMV / skinny GEMM (MARLIN article, "実験と結果":
 * Sparse-MARLIN), on gfx950's 2:4 sparse MFMA:
 *   Y[m,n] = sum_g s[n,g] sum_{k in g, kept} x[m,k] q[n,k]   (fp32 accumulation)
 * x        [m, k] bf16.   w_packed: QL_INT4_SP24 blob from repack_weights.
 * y        out [m, n], QL_F32 or QL_BF16.
 * Tuned for m <= 32; any m >= 0 is accepted.
 * Shapes: n % 16 == 0, k % 128 == 0.  Errors as gemm_w4a4.
 * The kernels read the blob header together with their first weight loads
 * and test it (magic, version, format, n, k) before their first store: a blob
 * that is not one of this format packed for this (n, k) leaves y untouched
 * (the host cannot detect it without synchronising, so no status reports
 * it).  It is read as a blob of this format and shape first, so the buffer
 * must hold at least repack_weights_bytes(format, n, k) bytes.
 * ---------------------------------------------------------------------- */
int gemm_w4a16_sp24(const void *x_bf16, const void *w_packed, int64_t m, int64_t n,
                    int64_t k, void *y, int y_dtype, void *stream);

/* ------------------------------------------------------------------------
 * gemm_w4a16_sp24 with a caller-provided workspace for a k split over
 * blocks, as gemm_w4a16_ws: each block takes one k slice of several 16-row
 * weight tiles, and a second launch adds the slices' fp32 partial sums in
 * slice order (deterministic; results differ from gemm_w4a16_sp24's in fp32
 * rounding only).  Same arithmetic definition and arguments as
 * gemm_w4a16_sp24, plus the workspace (at least
 * gemm_w4a16_sp24_workspace(m, n, k) bytes, 16-byte aligned, not read before
 * it is written; NULL makes the call gemm_w4a16_sp24; calls sharing a
 * workspace must be ordered).  gemm_w4a16_sp24_workspace returns 0 when no
 * split applies (it applies to 8 < m <= 32 with k > 4096) and depends on the
 * current device's compute-unit count.  Errors: as gemm_w4a16_sp24, and
 * QL_EWORKSPACE when the workspace is non-NULL and too small.
 * ---------------------------------------------------------------------- */
size_t gemm_w4a16_sp24_workspace(int64_t m, int64_t n, int64_t k);
int gemm_w4a16_sp24_ws(const void *x_bf16, const void *w_packed, int64_t m,
                       int64_t n, int64_t k, void *y, int y_dtype, void *workspace,
                       size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Paged key/value cache.  Between a layer's qkv and output projections stand
 * the head norms, the rotation of queries and keys by their positions, the
 * cache of keys and values and the attention over it:
 *
 *   qkv_norm_rope_append(qkv) -> q, and K, V rows written to the cache
 *   kv_attention(q, cache)    -> y, the input of the output projection
 *   kv_commit                 -> after speculative decoding: the accepted
 *                                drafts' rows move behind the context
 *   kv_append, kv_gather         write and read rows without the norms
 *
 * The reference pages hand this cache from the prefill half to the decode
 * half (Disaggregated Quantization; Mix-Quant, system-level deployment) and
 * measure 8-bit against 16-bit caches (the qiita article on f16 and q8_0).
 *
 * A cache is one buffer of pages.  A page holds page_size consecutive tokens
 * of one sequence for all n_kv heads; a slot is page * page_size + offset.
 * Formats of one row (the K or V vector of one token and head):
 *   QL_KV_BF16   the values, rounded to nearest even
 *   QL_KV_E4M3   E4M3 codes of x / 2^e; e is the smallest integer >= -100 with
 *                max|x| <= 448 * 2^e (-100 for a row of zeros)
 *   QL_KV_NVFP4  as quantize_nvfp4 with the row's own tensor scale 2^e: groups
 *                of 16, s_g = E4M3(max|x_g| / 2^e / 6), code =
 *                E2M1(x / 2^e * (1 / s_g)), each binary32 step rounded once;
 *                e as above with 2688 = 6 * 448 in the place of 448
 * In the two quantized formats an infinity takes the largest code, counted as
 * 2^128 for e, and reads back as an infinity (finite elements beside it lose
 * their bits to that e); a NaN stays a NaN (QL_KV_NVFP4: its whole group of 16
 * reads back as NaN).
 *
 * Layout: blocks of 16 tokens of one kv head, [n_pages][n_kv][page_size / 16].
 * All blocks' codes come first, each block's 16 K rows and then its 16 V rows
 * of R bytes (R = 2 d, d, d / 2); then, in the same order, all blocks' scales
 * (0, 32, 2 d + 32 bytes).  Token t of a block, C = min(16, R / 4):
 *   K codes        byte b of the row at (b / C) 16 C + t C + b % C
 *   V codes        element u (QL_KV_NVFP4: byte u, a pair of elements) at
 *                  (u / S) 16 S + (t / 4) 4 S + (u % S) 4 + t % 4, counted in
 *                  elements (bytes); S = 32, 64, min(d, 128) / 2
 *   NVFP4 scales   K group g at (g / P) 16 P + t P + g % P with P = C / 8;
 *                  V group g at d + 16 g + t
 *   row exponents  e + 127 in one byte, in the last 32 bytes of a block's
 *                  scales: K at (t / 4) 8 + t % 4, V four bytes after it
 *
 * format     QL_KV_BF16, QL_KV_E4M3 or QL_KV_NVFP4.
 * n_kv       key/value heads, 1..1024.
 * head_dim   64, 128 or 256.
 * page_size  a power of two, 16..4096.
 * data       device buffer of at least kv_cache_bytes(...) bytes, 16-byte
 *            aligned.  It needs no initialisation: only rows that were
 *            written are ever used.
 * The struct is read during the call only.  kv_cache_bytes returns 0 for
 * arguments outside these ranges (or more than 2^40 blocks).
 * Errors of every call that takes one: QL_EINVAL (null), QL_EFORMAT (format),
 * QL_ESHAPE (sizes), QL_EWORKSPACE (bytes), QL_EALIGN (data).
 * ---------------------------------------------------------------------- */
typedef enum { QL_KV_BF16 = 0, QL_KV_E4M3 = 1, QL_KV_NVFP4 = 2 } ql_kv_format;

typedef struct {
  int32_t format;
  int32_t n_kv;
  int32_t head_dim;
  int32_t page_size;
  int64_t n_pages;
  void *data;
  size_t bytes;
} ql_kv_cache;

size_t kv_cache_bytes(int format, int64_t n_pages, int64_t page_size, int64_t n_kv,
                      int64_t head_dim);

/* ------------------------------------------------------------------------
 * Write K and V rows to their slots, in the cache's format.
 *
 * k, v       [tokens, n_kv, head_dim], x_dtype QL_F32 or QL_BF16; a token's
 *            heads are contiguous, tokens are k_stride / v_stride elements
 *            apart (slices of a fused qkv buffer will do).  Rows start on 16
 *            bytes: both strides and the pointers are multiples of 16 bytes.
 * slots      int64 [tokens].  A slot outside the cache (any negative number)
 *            is skipped; two tokens of one call must not share a slot.
 * Errors: the cache's, QL_EINVAL, QL_ESHAPE (tokens < 0 is QL_EINVAL, more
 * than 2^31 - 1, or a stride shorter than a token's heads), QL_EDTYPE,
 * QL_EALIGN, QL_EHIP.
 * ---------------------------------------------------------------------- */
int kv_append(const ql_kv_cache *cache, const void *k, const void *v, int x_dtype,
              int64_t tokens, int64_t k_stride, int64_t v_stride, const int64_t *slots,
              void *stream);

/* ------------------------------------------------------------------------
 * Read rows back: k, v out [tokens, n_kv, head_dim] contiguous, the values
 * the cached rows stand for, y_dtype QL_F32 or QL_BF16 (both exact: a code
 * times its scales has at most 6 significant bits; rows of exponents near the
 * end of the type's range excepted).  A slot outside the cache gives zeros.
 * Errors: as kv_append.
 * ---------------------------------------------------------------------- */
int kv_gather(const ql_kv_cache *cache, const int64_t *slots, int64_t tokens, void *k, void *v,
              int y_dtype, void *stream);

/* ------------------------------------------------------------------------
 * The step between the qkv projection and the attention, in one pass over
 * the projection's output: RMS norm of every query and key head, rotation of
 * both by the token's position, queries out, K and V written to the cache
 * (as kv_append).  Queries are computed in binary32 (their squares' sum must
 * lie in its range: values from 1e-18 to 1e17, or any small ones with an eps
 * that is not), keys in binary64 up to the roundings of the row's format.
 *   norm      x <- x / sqrt(mean(x^2) + eps) * weight
 *   rotation  (a, b) <- (a c - b s, b c + a s) for rot / 2 pairs of a head,
 *             a = x[i], b = x[i + rot / 2], or x[2 i], x[2 i + 1] with
 *             QL_ROPE_INTERLEAVED; elements from rot on are left as they are
 *
 * qkv        [tokens, (n_q + 2 n_kv) * head_dim], QL_F32 or QL_BF16: queries,
 *            keys, values; rows row_stride elements apart, 16-byte aligned.
 * n_q        query heads, 1..65536.
 * q_weight,  fp32 [head_dim] norm weights of queries and keys; NULL: no norm
 * k_weight   of that kind.
 * positions  int32 [tokens]; a position outside [0, max_pos) takes the
 *            nearest row of the table.  May be NULL when rot == 0.
 * rope       fp32 [max_pos, rot]: c[0..rot/2), then s[0..rot/2) of a position.
 *            May be NULL when rot == 0.
 * rot        0 (no rotation) or an even number up to head_dim.
 * flags      0 or QL_ROPE_INTERLEAVED.
 * q_out      out [tokens, n_q, head_dim] bf16 (RNE), for every token, also
 *            one whose slot is skipped.
 * Errors: the cache's, QL_EINVAL, QL_ESHAPE, QL_EDTYPE, QL_EALIGN, QL_EHIP.
 * ---------------------------------------------------------------------- */
#define QL_ROPE_INTERLEAVED 1u
int qkv_norm_rope_append(const ql_kv_cache *cache, const void *qkv, int x_dtype, int64_t tokens,
                         int64_t row_stride, int64_t n_q, const float *q_weight,
                         const float *k_weight, float eps, const int32_t *positions,
                         const float *rope, int64_t max_pos, int64_t rot, unsigned flags,
                         void *q_out, const int64_t *slots, void *stream);

/* ------------------------------------------------------------------------
 * Attention of each sequence's newest tokens over its cached context and
 * over themselves.  Sequence b has n_b = cu_q[b + 1] - cu_q[b] queries; its
 * keys are the first kv_lens[b] positions of its pages, the last n_b of which
 * are the rows of those same tokens (written beforehand).  Query i sees the
 * context (every position before the last n_b) and, of the n_b new tokens,
 *   tree != NULL  token j where bit j of tree[cu_q[b] + i] is set (a tree of
 *                 drafted tokens: the bits of the path from the root to i,
 *                 itself included), n_b <= 64
 *   tree == NULL  tokens j <= i: one token is ordinary decoding, several are
 *                 a chain of drafts or a chunk of a prompt
 * and of those only positions whose page is in the cache: a block-table entry
 * outside [0, n_pages) hides its page's tokens.
 *   y = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale q.k_p - max_p scale q.k_p)
 * A query that sees nothing gives zeros.  Rows that no query of a sequence
 * sees do not matter, whatever they hold; a NaN or infinity in a row hidden
 * from one query does not reach it.  A NaN that a query sees makes its result
 * NaN, in V's element at least and possibly in all.  An infinity that it sees
 * in V makes the result infinite or NaN likewise; in a quantized cache it counts
 * as its code's value, 1.75 2^128 (QL_KV_E4M3) or 1.3125 2^128, times its
 * weight.  One in K gives an infinite score: a result of NaN, or no weight.
 *
 * Sums are binary32.  Keys, values and queries enter exactly (queries over
 * QL_KV_NVFP4 rounded to a multiple of 2^-38 of their row's largest value).
 * Weights are rounded to 16 bits (QL_KV_BF16; those below 2^-120 of the largest
 * lose bits, below 2^-133 all of them), or to 11 bits, those below
 * 2^-21 of the largest w_p 2^e_p (e_p: the exponent of V's row) to a multiple
 * of at most 2^-31 of it.  Weights below 2^-70 of the largest, or 2^(e - 130)
 * where a V row's exponent e is above 60, may be missing from their sum.
 *
 * q            bf16 [tokens, n_q, head_dim]; a token's heads are contiguous,
 *              tokens q_stride elements apart; 16-byte aligned rows.
 * tokens       rows of q and y; cu_q[n_seqs] <= tokens.
 * n_q          query heads, a multiple of n_kv; heads h n_q / n_kv .. + n_q /
 *              n_kv - 1 share kv head h.
 * cu_q         int32 [n_seqs + 1], ascending from 0; kv_lens int32 [n_seqs].
 * block_table  int32 [n_seqs, table_cols], rows table_stride elements apart:
 *              the page of positions page_size * j .. of each sequence.
 *              Positions past the table's last column are not read: they are
 *              hidden, like those of a page that is not in the cache.
 * max_q        at least every n_b (queries past it are not computed).
 * max_kv       about the largest kv_lens[b]; whether and into how many parts
 *              keys are split goes by it, where goes by the lengths
 *              themselves.  The result is right for any value.
 * y            out bf16 [tokens, n_q, head_dim] contiguous (RNE).
 * workspace    >= kv_attention_workspace(...) bytes, 16-byte aligned (NULL when
 *              that is 0).  Calls that share one must be ordered.
 * Errors: the cache's, QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EWORKSPACE,
 * QL_EHIP.  tokens == 0, n_seqs == 0 or max_q == 0: QL_OK, nothing is done.
 * ---------------------------------------------------------------------- */
size_t kv_attention_workspace(const ql_kv_cache *cache, int64_t tokens, int64_t n_q,
                              int64_t n_seqs, int64_t max_q, int64_t max_kv);
int kv_attention(const ql_kv_cache *cache, const void *q_bf16, int64_t q_stride, int64_t tokens,
                 int64_t n_q, int64_t n_seqs, const int32_t *cu_q, const int32_t *kv_lens,
                 const int32_t *block_table, int64_t table_stride, int64_t table_cols,
                 int64_t max_q, int64_t max_kv, const uint64_t *tree, float scale, void *y,
                 void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * After a tree of drafted tokens was verified: the rows of the accepted path
 * move right behind the context, as they are (no requantization).  With ctx =
 * kv_lens[b] - n_b, row ctx + path[b][j] goes to ctx + j, for every j at
 * once: sources are read before targets are written.  The caller's new length
 * is ctx plus the accepted count; cu_q and kv_lens are those of the
 * verification.
 *
 * path  int32 [n_seqs, max_path]: accepted draft indices, root first; an
 *       entry outside [0, n_b) moves nothing (pad with -1), nor does one of
 *       whose two rows the page is not in the cache.  max_path <= 64.
 * Errors: as kv_attention.
 * ---------------------------------------------------------------------- */
int kv_commit(const ql_kv_cache *cache, int64_t n_seqs, const int32_t *cu_q,
              const int32_t *kv_lens, const int32_t *block_table, int64_t table_stride,
              int64_t table_cols, const int32_t *path, int64_t max_path, void *stream);

/* ========================================================================
 * Linear layers whose rows choose their own weights: mixtures of experts
 * (each token meets the weights of its top_k experts) and low-rank adapters
 * (each request has its own).  The calls run over a PLAN, the rows of a batch
 * in the order of the weights they meet:
 *
 *   order   [rows]        the row at each place of that order
 *   where   [rows]        the place of each row (the inverse)
 *   offsets [groups + 1]  group g's run is the places offsets[g] ..
 *                         offsets[g + 1] - 1, its rows in ascending order
 *
 * Rows of no group come last, from offsets[groups] on.  For a mixture the
 * rows of a plan are the pairs (token, choice), pair = token * top_k + choice.
 * Everything stays on the device: no call needs to know a group's size, and a
 * captured graph may be replayed on other choices.  The arrays are as one of
 * the two calls below wrote them; entries outside of the batch are held to it
 * (no call reads or writes out of bounds for any contents), with results that
 * mean nothing.
 *
 * At most 1024 groups, 2^24 - 1 rows, top_k <= 64.
 * ===================================================================== */

/* ------------------------------------------------------------------------
 * The plan of given choices (the adapter of each row).
 * ids   [rows]: the row's group; outside of 0 .. groups - 1: none.
 * The plan's arrays share no bytes with ids (QL_EINVAL).
 * rows == 0 writes offsets of zero.  workspace: group_rows_workspace(rows,
 * groups) bytes, 16-byte aligned (0: may be NULL), not read before it is
 * written; calls that share one must be ordered.
 * Errors: QL_EINVAL, QL_ESHAPE, QL_EALIGN (int32 pointers: 4 bytes),
 * QL_EWORKSPACE, QL_EHIP.
 * ---------------------------------------------------------------------- */
size_t group_rows_workspace(int64_t rows, int64_t groups);
int group_rows(const int32_t *ids, int64_t rows, int64_t groups, int32_t *order, int32_t *where,
               int32_t *offsets, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * A router's choice: for each token the top_k experts of largest logit (of
 * equal ones the lowest expert first), their weights, and the plan of the
 * pairs.
 *   weight = exp(l - max) / sum exp(l' - max), in binary32, the sum over all
 *   experts or, with QL_ROUTE_RENORMALIZE, over the chosen ones.
 * An expert whose logit is -infinity or NaN is not chosen and takes no part in
 * the sum: where fewer than top_k are left, the other choices are -1 with
 * weight 0 and belong to no group.  Experts at +infinity share the weight.
 *
 * logits   [tokens, experts] QL_F32 or QL_BF16, rows row_stride elements apart.
 * ids, weights  out [tokens, top_k].
 * order, where, offsets  out: the plan of tokens * top_k pairs.  No output shares
 *          bytes with the logits (QL_EINVAL).
 * workspace as group_rows.  Errors: as group_rows, and QL_EDTYPE.
 * ---------------------------------------------------------------------- */
#define QL_ROUTE_RENORMALIZE 1u
size_t moe_route_workspace(int64_t tokens, int64_t experts, int64_t top_k);
int moe_route(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t row_stride,
              int64_t top_k, unsigned flags, int32_t *ids, float *weights, int32_t *order,
              int32_t *where, int32_t *offsets, void *workspace, size_t workspace_bytes,
              void *stream);

/* ------------------------------------------------------------------------
 * The pairs' products with their experts' weights: for place p of expert e
 *   y[p, :] = x[row(p), :] W_e^T
 * W4A16 (decoding; bf16 x, INT4 blobs) and W4A4 (prompts; x as quantize_nvfp4
 * leaves it, under one tensor scale, NVFP4 blobs).
 *
 * row(p)   order[p] / top_k with QL_ROWS_GATHER (x holds a row for each token),
 *          else p (x is in the plan's order; order may be NULL).
 * experts  n_experts blobs of W_e [n, k] from repack_weights, expert_bytes
 *          apart (a multiple of 16, at least repack_weights_bytes(...)).
 * y        out [pairs, n] in the plan's order, QL_F32 or QL_BF16; shares no
 *          bytes with x (QL_EINVAL).
 * QL_ROWS_SILU_MUL: the first n / 2 rows of W_e are a gate g, the others u,
 *          and y [pairs, n / 2] = silu(g) * u, silu(g) = g / (1 + exp(-g)), in
 *          binary32, rounded once.
 * Rows of y of pairs without an expert are set to zero.
 * Shapes: n % 16 == 0 (n % 32 with QL_ROWS_SILU_MUL), k % 128 == 0, n * k <=
 * 2^31; W4A4: fewer than 2^32 / k rows of x, and (pairs / T + n_experts + 1)
 * (n / 256, rounded up) at most 2^23 - 4096, T = 64 up to 256 pairs an expert
 * (pairs <= 256 n_experts), else 256; W4A16: (pairs / 32 + n_experts + 1)
 * (n / 512, rounded up) below 2^22.  A blob that is not of this
 * format and (n, k) leaves its expert's rows untouched.
 * Errors: QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EDTYPE, QL_EWORKSPACE
 * (expert_bytes too small), QL_EHIP.
 * ---------------------------------------------------------------------- */
#define QL_ROWS_GATHER 1u
#define QL_ROWS_SILU_MUL 2u
int moe_gemm_w4a16(const void *x_bf16, const void *experts, int64_t n_experts, int64_t expert_bytes,
                   const int32_t *order, const int32_t *offsets, int64_t pairs, int64_t top_k,
                   int64_t n, int64_t k, unsigned flags, void *y, int y_dtype, void *stream);
int moe_gemm_w4a4(const uint8_t *a_codes, const uint8_t *a_scales, const float *a_tensor_scale,
                  const void *experts, int64_t n_experts, int64_t expert_bytes,
                  const int32_t *order, const int32_t *offsets, int64_t pairs, int64_t top_k,
                  int64_t n, int64_t k, unsigned flags, void *y, int y_dtype, void *stream);

/* ------------------------------------------------------------------------
 * Back to the tokens: out[t, :] = sum_j weights[t, j] rows[where[t, j], :], in
 * binary32 and in the order of the choices.  Places from offsets[n_experts] on
 * (pairs without an expert) are not read and add nothing.
 * rows  [tokens * top_k, n] and out [tokens, n], each QL_F32 or QL_BF16, out
 *       sharing no bytes with rows (QL_EINVAL).
 * Shapes: n % 8 == 0.  Errors: as the products.
 * ---------------------------------------------------------------------- */
int moe_combine(const void *rows, int x_dtype, const int32_t *where, const int32_t *offsets,
                int64_t n_experts, const float *weights, int64_t tokens, int64_t top_k, int64_t n,
                void *out, int out_dtype, void *stream);

/* ------------------------------------------------------------------------
 * Low-rank adapters beside a projection that all rows share:
 *   out[t, :] = y[t, :] + scale[i] B_i (A_i x[t, :]),  i the adapter of row t
 * binary32 accumulation; A x is kept in 16 bits of mantissa or more (all 24
 * where y is binary32), and out is rounded once.  Rows without an adapter: out =
 * y.
 *
 * y, out   [rows, n] QL_F32 or QL_BF16 (y_dtype for both), rows y_stride and
 *          out_stride elements apart (slices of a fused projection will do).
 *          out may be y; otherwise they share no bytes, and out none with x
 *          (QL_EINVAL; slices side by side of rows of one stride will do).
 * x        [rows, k] bf16, rows x_stride apart.
 * a, b     [adapters, rank, k] and [adapters, n, rank] bf16, contiguous.
 * scale    [adapters] or NULL (1).
 * order, offsets  the plan of the rows' adapters (group_rows).
 * workspace  lora_add_workspace(rows, adapters, rank, k) bytes, 16-byte
 *          aligned, not read before it is written; calls that share one must be
 *          ordered.
 * Shapes: n % 16 == 0, k % 128 == 0, rank a multiple of 8 up to 128 (smaller
 * ranks: padded with zeros).  Row strides are multiples of 16 bytes; rows times
 * a stride is at most 2^47 bytes.
 * Errors: QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EDTYPE, QL_EWORKSPACE, QL_EHIP.
 * ---------------------------------------------------------------------- */
size_t lora_add_workspace(int64_t rows, int64_t adapters, int64_t rank, int64_t k);
int lora_add(const void *y, int64_t y_stride, const void *x_bf16, int64_t x_stride,
             const void *a_bf16, const void *b_bf16, const float *scale, int64_t adapters,
             int64_t rank, const int32_t *order, const int32_t *offsets, int64_t rows, int64_t n,
             int64_t k, void *out, int64_t out_stride, int y_dtype, void *workspace,
             size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_H */
