/*
 * metis_fp4.h -- C ABI of libmetis_fp4.so: the spectral-domain FP4 linear
 * layer (randomized split + block FP4 quantization + W4A4G4 GEMMs) for
 * AMD Instinct MI355X (gfx950).
 *
 * Method: "Metis: Training LLMs with FP4 Quantization" (arXiv 2509.00404),
 * abstract; SII open-source-week post on Metis, §2.3-§2.4. A matrix is split
 * into a dominant low-rank part U_k diag(S_k) V_k^T, found by a random
 * projection or by sparse column sampling, and a long-tail residual R; each
 * part is quantized to FP4 separately and the linear layer's three GEMMs run
 * on the quantized parts.
 *
 * Conventions for every call
 *  - Array pointers are DEVICE pointers owned by the caller. The library never
 *    allocates or frees memory, never synchronizes the device and keeps no
 *    global state: calls are re-entrant and may run on any stream. (The one
 *    exception, spectral_fp4_linear_fwd_noalloc, uses a static per-GPU
 *    scratch array instead of a workspace argument.)
 *  - All work is enqueued on `stream` (asynchronous). Outputs are valid once
 *    the stream reaches that point.
 *  - Arguments are validated on the host before any HIP call; a failed check
 *    returns METIS_ERR_INVALID / METIS_ERR_UNSUPPORTED / METIS_ERR_WORKSPACE
 *    and enqueues nothing. A failed launch returns METIS_ERR_HIP.
 *  - Matrices are row-major with an explicit leading dimension (elements).
 *  - FP4 blocks always run along the last (contiguous) axis of the stored
 *    matrix; for a GEMM operand that is the contraction axis.
 *  - Inputs containing NaN or Inf give undefined (but memory-safe) results,
 *    where a call does not say otherwise.
 *  - Empty matrices (a zero dimension) are valid and enqueue nothing, where a
 *    call does not say otherwise.
 */
#ifndef METIS_FP4_H
#define METIS_FP4_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  METIS_OK = 0,
  METIS_ERR_INVALID = 1,     /* bad pointer, shape, leading dimension or missing operand */
  METIS_ERR_UNSUPPORTED = 2, /* a valid request this build does not implement */
  METIS_ERR_WORKSPACE = 3,   /* ws == NULL or ws_bytes below the matching *_workspace_bytes() */
  METIS_ERR_HIP = 4,         /* a HIP launch failed */
  METIS_ERR_TOO_LARGE = 5    /* the request needs more than a fixed-size static scratch */
} metis_status_t;

/* FP4 block formats (the pages name MXFP4 and NVFP4: SII post, project
 * highlights and §2.2). Bit layouts: OCP Microscaling Formats v1.0 (E2M1
 * elements, E8M0 scale per 32) and NVIDIA's NVFP4 (E2M1, E4M3 scale per 16,
 * one fp32 scale per tensor). */
typedef enum { METIS_MXFP4 = 0, METIS_NVFP4 = 1 } metis_fmt_t;

/* Storage type of a dense input. */
typedef enum { METIS_F32 = 0, METIS_BF16 = 1 } metis_dtype_t;

/* How the dominant subspace is sketched ("Metis" abstract: preservation via
 * random projection, and via sparse random sampling). */
typedef enum {
  METIS_OMEGA_GAUSSIAN = 0, /* omega: n x l bf16 row-major Gaussian test matrix */
  METIS_OMEGA_COLUMNS = 1   /* omega: int32 J[l], distinct column ids in [0, n) */
} metis_omega_t;

/* One FP4 matrix (rows x cols), blocks along cols.
 *  codes:        rows * cols / 2 bytes, row-major; element 2j of a row sits in
 *                the low nibble of byte j, element 2j+1 in the high nibble.
 *                Nibble = E2M1 code: bit 3 sign, bits 2-1 exponent, bit 0 mantissa.
 *  scales:       rows * (cols / B) bytes row-major, B = 32 (MXFP4, E8M0 byte e
 *                means 2^(e-127)) or 16 (NVFP4, E4M3 byte).
 *  tensor_scale: NVFP4 only: one fp32 on the device; NULL for MXFP4.
 * Element value: e2m1(code) * scale (* tensor_scale for NVFP4). */
typedef struct {
  int32_t fmt; /* metis_fmt_t */
  int32_t reserved;
  int64_t rows, cols;
  uint8_t *codes;
  uint8_t *scales;
  float *tensor_scale;
} metis_fp4_t;

/* Quantized split of one m x n tensor A = U diag(S) V^T + R.
 * k == 0 marks an operand that is not split: R_q / Rt_q then hold the
 * quantized tensor itself and U, S, V, Ut_q, Vt_q are unused.
 *  U (m x k), S (k, descending), V (n x k): fp32 row-major factors. Each column
 *      of U has its largest-magnitude entry positive (lowest row on ties).
 *  Ut_q: U^T (k x m) blocked along m;  Vt_q: V^T (k x n) blocked along n.
 *      (Each singular vector is quantized along its length; S stays fp32.)
 *  R_q:  R (m x n) blocked along n -- the operand of a GEMM contracting over n.
 *  Rt_q: R^T (n x m) blocked along m -- the operand of a GEMM contracting over m.
 *      Either residual orientation may be absent (codes == NULL). */
typedef struct {
  int64_t m, n;
  int32_t k;
  int32_t reserved;
  float *U;
  float *S;
  float *V;
  metis_fp4_t Ut_q;
  metis_fp4_t Vt_q;
  metis_fp4_t R_q;
  metis_fp4_t Rt_q;
} metis_split_t;

/* Human-readable name of a status code (static string, never NULL). */
const char *metis_status_str(metis_status_t status);

/* ABI revision of this header (bumped on any incompatible change). */
int32_t metis_abi_version(void);

/* ------------------------------------------------------------------------
 * Block FP4 quantization of a dense matrix (OCP MX v1.0 §6.3 scale rule for
 * MXFP4: shared exponent floor(log2 amax) - 2, clamped to [-127, 127];
 * NVFP4: s_t = max(amax_tensor / 2688, 2^-126), block scale
 * e4m3(amax_block / (6 s_t)), element x / (e4m3 * s_t), each step a correctly
 * rounded fp32 operation). Elements round to nearest E2M1 value, ties to the
 * even code, saturating at +-6; an all-zero block gets scale 0 and +-0 codes.
 *
 *  x:         rows x cols, leading dimension ldx >= cols, type dt.
 *  transpose: 0 -> out is rows x cols blocked along cols;
 *             1 -> out is x^T (cols x rows) blocked along rows.
 *  out:       caller sets fmt, codes, scales (and tensor_scale for NVFP4);
 *             the library writes out->rows and out->cols.
 *  ws:        scratch of fp4_block_quant_workspace_bytes() bytes (0 for MXFP4:
 *             ws may then be NULL).
 * The blocked axis must be a multiple of the block size (32 or 16). */
size_t fp4_block_quant_workspace_bytes(int64_t rows, int64_t cols, metis_fmt_t fmt);
metis_status_t fp4_block_quant(const void *x, metis_dtype_t dt, int64_t rows, int64_t cols, int64_t ldx,
                               int32_t transpose, metis_fp4_t *out, void *ws, size_t ws_bytes,
                               hipStream_t stream);

/* Exact dequantization to fp32: y (in->rows x in->cols, leading dimension
 * ldy >= in->cols) = e2m1(code) * scale (* tensor_scale). */
metis_status_t fp4_block_dequant(const metis_fp4_t *in, float *y, int64_t ldy, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Randomized spectral split (SII post on Metis §2.4 item 1: dominant part and
 * long-tail residual, quantized separately, decomposition done in a
 * low-dimensional space; steps as in Halko-Martinsson-Tropp 2011, Alg. 4.1
 * without power iterations and Alg. 5.1):
 *   Y = A Omega (or A[:, J]);  Q = orth(Y);  B = Q^T A;  B = Ub diag(sigma) W^T;
 *   U = Q Ub[:, :k], S = sigma[:k], V = W[:, :k], column signs fixed as above;
 *   R = A - U diag(S) V^T, quantized in the orientations whose codes != NULL;
 *   U^T and V^T quantized along their length.
 *
 *  A:     m x n (lda >= n) of type dt.
 *  omega: METIS_OMEGA_GAUSSIAN: n x l bf16 row-major (the bits of bfloat16
 *         values); METIS_OMEGA_COLUMNS: int32[l] distinct ids in [0, n)
 *         (ids out of range give undefined values, never an out-of-bounds read).
 *  1 <= k <= l <= min(m, n); k <= 96 and l <= 512 (beyond: METIS_ERR_UNSUPPORTED).
 *  Sketches with l <= 96 keep the l x l problems in LDS; wider ones keep
 *  them in global memory (their Cholesky and tridiagonal reduction take one
 *  launch per 16 pivots or per reflector, so they are launch-bound). m and n
 *  multiples of 32; A
 *  16-byte aligned and lda * sizeof(element) a multiple of 16.
 *  out:   caller provides U, S, V (fp32) and the codes/scales (/tensor_scale)
 *         buffers of Ut_q, Vt_q, R_q and/or Rt_q (each fp4 member's fmt must
 *         equal `fmt`); the library writes m, n, k and the rows/cols fields.
 *  info:  optional device int32 (may be NULL), written with 0 on success or
 *         i > 0 when the sketch is rank deficient (the i-th pivot of its
 *         Cholesky factor broke down); the columns of U from that rank on
 *         then carry S = 0. Read it after synchronizing the stream.
 *  ws:    scratch of metis_split_workspace_bytes() bytes, 256-byte aligned.
 * Results are bitwise reproducible run to run (no atomics in reductions). */
size_t metis_split_workspace_bytes(int64_t m, int64_t n, int32_t l, int32_t k, metis_omega_t kind,
                                   metis_fmt_t fmt);
metis_status_t metis_split(const void *A, metis_dtype_t dt, int64_t m, int64_t n, int64_t lda,
                           const void *omega, metis_omega_t kind, int32_t l, int32_t k, metis_fmt_t fmt,
                           metis_split_t *out, int32_t *info, void *ws, size_t ws_bytes,
                           hipStream_t stream);

/* The same split with q power (subspace) iterations after the sketch
 * (Halko-Martinsson-Tropp 2011, Alg. 4.4): with Q = orth(Y), each iteration
 * forms Z = orth(A^T Q) and Y = A Z, Q = orth(Y), every orthonormalization a
 * CholeskyQR2 in fp64 and Z applied as bf16 hi + lo (fp32-accurate). Each
 * iteration adds two passes over A. metis_split is q = 0.
 *  q: 0 <= q <= 16 (beyond: METIS_ERR_UNSUPPORTED); q > 0 needs l <= 96
 *     (beyond: METIS_ERR_UNSUPPORTED); q < 0: METIS_ERR_INVALID.
 *  info: the rank status of the last sketch's Cholesky factor.
 *  ws: metis_split_power_workspace_bytes() bytes (it grows with q > 0).
 * Everything else as for metis_split. */
size_t metis_split_power_workspace_bytes(int64_t m, int64_t n, int32_t l, int32_t k, metis_omega_t kind,
                                         int32_t q, metis_fmt_t fmt);
metis_status_t metis_split_power(const void *A, metis_dtype_t dt, int64_t m, int64_t n, int64_t lda,
                                 const void *omega, metis_omega_t kind, int32_t l, int32_t k, int32_t q,
                                 metis_fmt_t fmt, metis_split_t *out, int32_t *info, void *ws, size_t ws_bytes,
                                 hipStream_t stream);

/* ------------------------------------------------------------------------
 * Mean-residual split (Averis, "Averaging-Induced Residual Splitting", as
 * retold on the zhu318.com page, method paragraphs): the mean over all rows,
 * mu (one value per column), and the residual A - mu broadcast over the rows
 * are quantized separately. The result is the rank-1 split record
 *   U = 1 (m x 1), S = {1}, V = mu (n x 1),  R = A - 1 mu^T,
 * so it enters spectral_fp4_linear_fwd/_bwd and metis_gemm_nt_* like any
 * split operand (the all-ones U is exact in both FP4 formats).
 *  A, dt, m, n, lda, fmt, out, ws, stream: as for metis_split, with k = 1
 *  (out->U holds m floats, S one, V n). mu is summed in fp64 over rows in a
 *  fixed order and rounded once to fp32; R = A - mu is one fp32 subtraction
 *  per element. ws: metis_mean_split_workspace_bytes() bytes, 256-byte
 *  aligned. Errors as for metis_split; bitwise reproducible. */
size_t metis_mean_split_workspace_bytes(int64_t m, int64_t n, metis_fmt_t fmt);
metis_status_t metis_mean_split(const void *A, metis_dtype_t dt, int64_t m, int64_t n, int64_t lda,
                                metis_fmt_t fmt, metis_split_t *out, void *ws, size_t ws_bytes,
                                hipStream_t stream);

/* ------------------------------------------------------------------------
 * W4A4G4 linear layer ("Metis" abstract: FP4 weights, activations and
 * gradients). Each GEMM is C = A_hat B_hat^T with, for a split operand,
 * A_hat = R_hat + U_hat diag(S) V_hat^T in the orientation it is used in
 * (R_q for contraction over n, Rt_q for contraction over m). The product runs
 * as the FP4 GEMM of the residuals plus a low-rank correction; outputs are
 * fp32. Shapes: X is M x K (tokens x in), W is N x K (out x in), dY is M x N.
 *   fwd:  Y  = X W^T    (M x N)   needs X.R_q,  W.R_q
 *   bwd:  dX = dY W     (M x K)   needs dY.R_q, W.Rt_q
 *         dW = dY^T X   (N x K)   needs dY.Rt_q, X.Rt_q
 * All operands must share one format. ws: metis_linear_workspace_bytes()
 * bytes (256-byte aligned); dY may be NULL in the query for fwd only. */
size_t metis_linear_workspace_bytes(const metis_split_t *X, const metis_split_t *W, const metis_split_t *dY);
metis_status_t spectral_fp4_linear_fwd(const metis_split_t *X, const metis_split_t *W, float *Y, int64_t ldy,
                                       void *ws, size_t ws_bytes, hipStream_t stream);
/* The forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * spectral_fp4_linear_fwd with its workspace taken from a static device array
 * of METIS_NOALLOC_SCRATCH_BYTES in the library instead of a ws argument. The
 * call itself allocates nothing; each GPU the library runs on holds its own
 * copy of the array from the library's load until the process ends. Inputs
 * and Y are the caller's, as for spectral_fp4_linear_fwd, and the result is
 * the same bit for bit.
 *  - Work is enqueued on `stream`, which must belong to the current device.
 *  - A forward whose metis_linear_workspace_bytes(X, W, NULL) exceeds
 *    METIS_NOALLOC_SCRATCH_BYTES returns METIS_ERR_TOO_LARGE and enqueues
 *    nothing (64 MiB covers 8192 tokens x 4096 x 14336 at k = 64).
 *  - Every call on one GPU shares that GPU's array, and the array keeps the
 *    last call's contents (nothing in it needs to start at zero). Calls that
 *    overlap on one GPU (concurrent streams, or host threads without
 *    ordering) race on it: serialize them.
 * Other errors as for spectral_fp4_linear_fwd; METIS_ERR_HIP also when the
 * array's device address cannot be looked up. */
#define METIS_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
metis_status_t spectral_fp4_linear_fwd_noalloc(const metis_split_t *X, const metis_split_t *W, float *Y,
                                               int64_t ldy, hipStream_t stream);

/* dX or dW may be NULL to skip that product. */
metis_status_t spectral_fp4_linear_bwd(const metis_split_t *dY, const metis_split_t *X, const metis_split_t *W,
                                       float *dX, int64_t lddx, float *dW, int64_t lddw, void *ws,
                                       size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * The two halves of one GEMM C = A_hat B_hat^T (rows of C from operand a,
 * columns from operand b; a_trans / b_trans select the orientation each
 * operand is used in: 0 -> R_q, contraction over its n; 1 -> Rt_q,
 * contraction over its m). spectral_fp4_linear_fwd/bwd are prepare + main.
 *  prepare: the skinny FP4 products R_a F_b, R_b F_a, F_a^T F_b and the bf16
 *           correction panels, written into ws;
 *  main:    the FP4 GEMM of the residuals plus the low-rank correction read
 *           from ws (left there by prepare on the same stream), fp32 output.
 * Splitting them lets a caller run the next prepare (in another workspace)
 * while a main runs, or time the main kernel alone. ws holds
 * metis_gemm_nt_workspace_bytes() bytes, 256-byte aligned. */
size_t metis_gemm_nt_workspace_bytes(const metis_split_t *a, int32_t a_trans, const metis_split_t *b,
                                     int32_t b_trans);
metis_status_t metis_gemm_nt_prepare(const metis_split_t *a, int32_t a_trans, const metis_split_t *b,
                                     int32_t b_trans, void *ws, size_t ws_bytes, hipStream_t stream);
metis_status_t metis_gemm_nt_main(const metis_split_t *a, int32_t a_trans, const metis_split_t *b, int32_t b_trans,
                                  float *C, int64_t ldc, const void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Adaptive spectral learning rate (SII post on Metis, §2.4 item 2; the
 * earlier version's abstract, chatpaper.ai page, item (ii)): the gradient
 * along a split's mid and low singular directions is scaled up by the
 * inverse of its normalized singular value, the dominant directions and the
 * unresolved tail R left as they are. With the split G = U diag(S) V^T + R of
 * the gradient (metis_split of G):
 *   gamma_i = min(gamma_max, max(1, S[r_ref] / S_i))  (1 where S_i = 0),
 *   G <- G + U diag(S (gamma - 1)) V^T,   in place.
 *  G:  m x n fp32, leading dimension ldg >= n (device).
 *  U (m x k), S (k, descending), V (n x k): fp32 row-major, as in a split
 *      record of G (device).
 *  1 <= k <= 96, 0 <= r_ref < k, gamma_max >= 1 (else METIS_ERR_INVALID;
 *  k > 96: METIS_ERR_UNSUPPORTED).
 * The rank-k term is summed in fp32 in ascending i and added to G once. */
metis_status_t metis_spectral_lr_rescale(float *G, int64_t m, int64_t n, int64_t ldg, const float *U,
                                         const float *S, const float *V, int32_t k, int32_t r_ref, float gamma_max,
                                         hipStream_t stream);

/* ------------------------------------------------------------------------
 * Dual-range regularizer (SII post on Metis, §2.4 item 3; chatpaper.ai
 * abstract, item (iii)): a penalty that restrains oversized values and
 * suppresses near-zero ones, compressing a parameter tensor's range. Two-sided
 * hinge on each element w of W:
 *   loss = lam_hi sum relu(|w| - tau_hi)^2 + lam_lo sum_{w != 0} relu(tau_lo - |w|)^2,
 *   dloss/dw = 2 lam_hi relu(|w| - tau_hi) sign(w) - 2 lam_lo relu(tau_lo - |w|) sign(w).
 *  W:     rows x cols of type dt (leading dimension ldw >= cols; cols % 8 == 0;
 *         16-byte aligned rows).
 *  grad:  optional fp32 rows x cols (ldg >= cols, 16-byte aligned rows): the
 *         gradient, stored (accumulate == 0) or added to what is there
 *         (accumulate != 0). Each gradient value is formed in fp64 and rounded
 *         once to fp32 (after the addition when accumulating).
 *  loss:  optional device fp64 scalar; needs ws of
 *         metis_dual_range_workspace_bytes() bytes (8-byte aligned), and is
 *         summed in a fixed order (bitwise reproducible).
 *  0 <= tau_lo <= tau_hi, lam_lo, lam_hi >= 0 (else METIS_ERR_INVALID). */
size_t metis_dual_range_workspace_bytes(void);
metis_status_t metis_dual_range_reg(const void *W, metis_dtype_t dt, int64_t rows, int64_t cols, int64_t ldw,
                                    float tau_lo, float tau_hi, float lam_lo, float lam_hi, float *grad, int64_t ldg,
                                    int32_t accumulate, double *loss, void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * 8-bit storage of activations between the forward and the backward pass
 * (what the backward pass reads again beside the FP4 operands: norm inputs,
 * gate inputs). Formats: OCP Microscaling v1.0 §5.3, one E8M0 scale per 32
 * elements along a row, the last block of a row possibly shorter.
 *  METIS_MXFP8:  E4M3 elements (at most 448; relative half step 2^-4 down to
 *                2^-6 of the scale, spacing 2^-9 below).
 *  METIS_MXINT8: two's complement elements in units of 1/64 (at most 127/64;
 *                half step 2^-7 of the scale everywhere).
 * Scale 2^e: the smallest e >= -127 with which no element of the block exceeds
 * the largest representable one (so nothing is clipped; only an MXINT8 block
 * above 127/64 * 2^127 is held at that value). Elements x / 2^e round to
 * nearest even; an MXFP8 zero keeps its sign. A block that holds an infinity
 * or a NaN is stored with scale byte 255 and reads back as NaN throughout; an
 * all-zero block has scale byte 0. */
typedef enum { METIS_MXFP8 = 2, METIS_MXINT8 = 3 } metis_fmt8_t;

/* One matrix (rows x cols) in 8 bits, blocks along cols.
 *  codes:  rows * cols bytes, row-major, rows tightly packed.
 *  scales: rows * ceil(cols / 32) bytes, row-major; byte e means 2^(e-127). */
typedef struct {
  int32_t fmt; /* metis_fmt8_t */
  int32_t reserved;
  int64_t rows, cols;
  uint8_t *codes;
  uint8_t *scales;
} metis_act8_t;

/* x (rows x cols of type dt, ldx >= cols, aligned to its element type; any
 * width) into out, whose fmt, codes and scales the caller sets; the library
 * writes out->rows and out->cols. Beyond 2^31 - 1 rows or 2^30 columns:
 * METIS_ERR_UNSUPPORTED, here and in the calls below. In these calls no output
 * (nor the workspace) may share memory with an input or another output, else
 * METIS_ERR_INVALID; the two halves of one matrix share none. (Two matrices of
 * different leading dimension are taken to share memory where their address
 * ranges meet.) */
metis_status_t act8_block_quant(const void *x, metis_dtype_t dt, int64_t rows, int64_t cols, int64_t ldx,
                                metis_act8_t *out, hipStream_t stream);
/* The stored values as type dt, exact in both types (no element has more than
 * 8 significant bits), but for subnormals in bf16 and for 2^128, which MXFP8
 * rounds magnitudes from 1.9375 * 2^127 on to: it reads back as infinity. */
metis_status_t act8_block_dequant(const metis_act8_t *in, void *y, metis_dtype_t dt, int64_t ldy, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Layer norm and RMS norm of the rows of x (n = cols), the input of an FP4
 * projection:
 *   LAYER: mean = sum(x) / n,  rstd = (sum((x - mean)^2) / n + eps)^(-1/2)
 *   RMS:   mean = 0,           rstd = (sum(x^2) / n + eps)^(-1/2)
 *   y = (x - mean) rstd w + b.
 *  x:      rows x cols of type dt, ldx >= cols, aligned to its element type.
 *  w, b:   cols elements of type wdt; either may be NULL (w = 1, b = 0).
 *  y:      rows x cols of type ydt, rounded once from fp32.
 *  mean, rstd: optional fp32 outputs, one per row (mean: LAYER only, not
 *          written for RMS; neither with cols = 0); the backward pass needs
 *          them.
 *  stored: optional: x in 8 bits as act8_block_quant writes it (fmt, codes and
 *          scales set by the caller), from the same read of x.
 *  eps >= 0 (else METIS_ERR_INVALID). Sums in fp32; the deviation is summed
 * around the mean, in a second pass over the row on chip. A finite row has a
 * finite mean. Where the sum of squares passes fp32's largest number (n
 * elements 1.8e19 / sqrt(n) from the mean; from 0 for RMS) rstd is 0: y is b,
 * dx is 0 and the row adds nothing to dw (an element farther from the mean than
 * that number gives NaN). At the other end, squares below 1e-38 lose bits,
 * which shows where eps is no larger; with eps = 0 a row whose squares are all
 * 0 has rstd = infinity and y = NaN. */
typedef enum {
  METIS_NORM_LAYER = 0,
  METIS_NORM_RMS = 1,
  METIS_NORM_NONE = 2 /* metis_qk_norm_rope_* only */
} metis_norm_t;
metis_status_t metis_norm_fwd(const void *x, metis_dtype_t dt, int64_t rows, int64_t cols, int64_t ldx, const void *w,
                              const void *b, metis_dtype_t wdt, metis_norm_t kind, float eps, void *y,
                              metis_dtype_t ydt, int64_t ldy, float *mean, float *rstd, metis_act8_t *stored,
                              hipStream_t stream);

/* Its gradients. With xh = (x - mean) rstd and g = dy w:
 *   dx = rstd (g - [LAYER: sum(g) / n] - xh sum(g xh) / n),
 *   dw = sum over rows of dy xh,  db = sum over rows of dy.
 *  dy:     rows x cols of type dydt. x: dense, type xdt; or NULL with `stored`
 *          the 8-bit form of x (its rows and cols set): then xh is formed from
 *          the stored values with the mean and rstd given, and off by up to
 *          |x| rstd / 16 (MXFP8) or max |x of its block| rstd / 127 (MXINT8).
 *          For a row whose mean is m deviations that is about m / 16 or
 *          (m + 3) / 127 in an xh of order 1: beyond m of a few (MXFP8) or a
 *          few tens (MXINT8) keep x dense.
 *  mean, rstd: as written by metis_norm_fwd (mean may be NULL for RMS).
 *  dx:     rows x cols of type dxdt, rounded once from fp32.
 *  dw, db: optional fp32 of cols elements, stored (accumulate == 0) or added
 *          to what is there (accumulate != 0). With no rows they are zero
 *          (stored) or kept (added).
 *  ws:     metis_norm_bwd_workspace_bytes() bytes, 256-byte aligned; may be
 *          NULL without dw and db. Sums over rows run in a fixed order (no
 *          atomics): bitwise reproducible. xh, dy w, rstd dy, their
 *          products and the sums have to stay in fp32's range. A NaN or an infinity in dy spoils its row of
 *          dx and its column of dw and db; one in x, through the row's
 *          statistics, its row of dx and all of dw. */
size_t metis_norm_bwd_workspace_bytes(int64_t rows, int64_t cols);
metis_status_t metis_norm_bwd(const void *dy, metis_dtype_t dydt, int64_t lddy, const void *x, metis_dtype_t xdt,
                              int64_t ldx, const metis_act8_t *stored, const void *w, metis_dtype_t wdt,
                              metis_norm_t kind, const float *mean, const float *rstd, int64_t rows, int64_t cols,
                              void *dx, metis_dtype_t dxdt, int64_t lddx, float *dw, float *db, int32_t accumulate,
                              void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * SwiGLU gate between an FFN's up and down projections:
 *   h = silu(a) b,  silu(a) = a / (1 + exp(-a)).
 *  a, b:   rows x cols of type dt, leading dimensions lda, ldb >= cols (the
 *          two halves of one fused projection's output, or two matrices).
 *  h:      rows x cols of type hdt, rounded once from fp32.
 *  qa, qb: optional, both or neither and of one format: a and b in 8 bits as
 *          act8_block_quant writes them, from the same read.
 * A NaN or an infinity reaches the outputs of its own element only (a = -inf
 * gives NaN, as a / (1 + exp(-a)) does). Below a = -86.6 the sigmoid is taken
 * as 0, so that h is 0 where it should be up to 2^-118 |b|. */
metis_status_t metis_swiglu_fwd(const void *a, int64_t lda, const void *b, int64_t ldb, metis_dtype_t dt, int64_t rows,
                                int64_t cols, void *h, metis_dtype_t hdt, int64_t ldh, metis_act8_t *qa,
                                metis_act8_t *qb, hipStream_t stream);

/* Its gradients. With s = 1 / (1 + exp(-a)):
 *   da = dh b s (1 + a (1 - s)),  db = dh a s.
 *  dh:     rows x cols of type dhdt.
 *  a, b:   dense, type dt; or both NULL with qa and qb their 8-bit forms.
 *  da, db: rows x cols of type odt, rounded once from fp32.
 *          Below a = -86.6 both are 0 (off by up to 2^-118 |dh b| and 2^-118
 *          |dh|); above a = 87.3 the slope in da is 1. dh b has to stay in
 *          fp32's range. An infinite a gives infinity or NaN.
 *  h:      optional, type odt: silu(a) b again, from the a and b given (the
 *          weight gradient of the down projection reads it). */
metis_status_t metis_swiglu_bwd(const void *dh, metis_dtype_t dhdt, int64_t lddh, const void *a, int64_t lda,
                                const void *b, int64_t ldb, metis_dtype_t dt, const metis_act8_t *qa,
                                const metis_act8_t *qb, int64_t rows, int64_t cols, void *da, int64_t ldda, void *db,
                                int64_t lddb, void *h, int64_t ldh, metis_dtype_t odt, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Norms of queries and keys for each head with the position rotation in the
 * same pass: what stands between the query / key projection and attention.
 * A token's row of q holds q_heads heads of head_dim elements side by side, a
 * row of k k_heads of them. For each head x of n = head_dim elements
 *   LAYER: xh = (x - mean) rstd,  RMS: xh = x rstd  (as metis_norm_fwd, no
 *   bias),  NONE: xh = x,
 *   u = xh w  (w = wq or wk, shared by the heads; NULL: 1),
 * and of the first rot_dim elements each pair (a, b) is turned by its angle:
 *   y_a = u_a cos - u_b sin,  y_b = u_b cos + u_a sin.
 * Pair i (of rot_dim / 2) is (i, i + rot_dim / 2) with METIS_ROPE_HALVES and
 * (2 i, 2 i + 1) with METIS_ROPE_NEIGHBOURS; the elements behind rot_dim are
 * left as they are.
 *  q, k:      tokens x (heads * head_dim) of type dt, ldq / ldk at least that
 *             wide (also parts of one matrix). k_heads = 0: no k, wk, ko.
 *  positions: int32 of tokens elements: the row of `rope` for each token.
 *  rope:      fp32, rope_rows x rot_dim, tightly packed: the cosines of a
 *             position's rot_dim / 2 angles, then their sines. A position
 *             outside [0, rope_rows) makes the token's rotated elements NaN
 *             (its gradient and dw too), never an out-of-bounds read. rot_dim = 0:
 *             positions and rope are not read.
 *  qo, ko:    tokens x (heads * head_dim) of type odt, rounded once from fp32.
 *  1 <= head_dim <= 512, 0 <= rot_dim <= head_dim, rot_dim even, at most 65536
 * heads (head_dim or heads beyond: METIS_ERR_UNSUPPORTED). No output may share
 * memory with an input or another output; the sums' range is as for
 * metis_norm_fwd. */
typedef enum { METIS_ROPE_HALVES = 0, METIS_ROPE_NEIGHBOURS = 1 } metis_rope_t;
metis_status_t metis_qk_norm_rope_fwd(const void *q, int64_t ldq, int32_t q_heads, const void *k, int64_t ldk,
                                      int32_t k_heads, metis_dtype_t dt, int64_t tokens, int32_t head_dim,
                                      const void *wq, const void *wk, metis_dtype_t wdt, metis_norm_t kind, float eps,
                                      const int32_t *positions, const float *rope, int64_t rope_rows, int32_t rot_dim,
                                      metis_rope_t pairs, void *qo, int64_t ldqo, void *ko, int64_t ldko,
                                      metis_dtype_t odt, hipStream_t stream);

/* Its gradients. With g = dy turned back by the same angles and u = g w:
 *   dx = rstd (u - [LAYER: sum(u) / n] - xh sum(u xh) / n),  NONE: dx = u,
 *   dw = sum over tokens and heads of g xh.
 *  dq, dk: tokens x (heads * head_dim) of type dydt: the gradients of qo, ko.
 *  q, k:   the forward's inputs (xh is formed again from them, nothing is
 *          kept); not read with METIS_NORM_NONE, where they may be NULL.
 *  dqi, dki: gradients of q and k, type dxdt, rounded once from fp32.
 *  dwq, dwk: optional fp32 of head_dim elements, stored (accumulate == 0) or
 *          added to what is there (accumulate != 0); NULL with NONE. With no
 *          tokens they are zero (stored) or kept (added).
 *  ws:     metis_qk_norm_rope_bwd_workspace_bytes() bytes, 256-byte aligned;
 *          may be NULL without dwq and dwk.
 *  tokens times half the heads of q or k, rounded up, has to be below 2^29
 *  (beyond: METIS_ERR_UNSUPPORTED; parts of the tokens can be added up with
 *  accumulate). Sums run in a fixed order: bitwise reproducible. */
size_t metis_qk_norm_rope_bwd_workspace_bytes(int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim);
metis_status_t metis_qk_norm_rope_bwd(const void *dq, int64_t lddq, const void *dk, int64_t lddk, metis_dtype_t dydt,
                                      const void *q, int64_t ldq, int32_t q_heads, const void *k, int64_t ldk,
                                      int32_t k_heads, metis_dtype_t dt, int64_t tokens, int32_t head_dim,
                                      const void *wq, const void *wk, metis_dtype_t wdt, metis_norm_t kind, float eps,
                                      const int32_t *positions, const float *rope, int64_t rope_rows, int32_t rot_dim,
                                      metis_rope_t pairs, void *dqi, int64_t lddqi, void *dki, int64_t lddki,
                                      metis_dtype_t dxdt, float *dwq, float *dwk, int32_t accumulate, void *ws,
                                      size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * The linear layer for a few tokens: y = x W_hat^T with x dense (not
 * quantized) and W_hat the FP4 weight of spectral_fp4_linear_fwd,
 *   y[t, i] = sum_j R_hat[i, j] x[t, j]
 *           + sum_r U_hat[i, r] S_r sum_j V_hat[j, r] x[t, j],
 * each codes-times-scales value exact, products and sums in fp32.
 *  x:  tokens x W->n of type dt, ldx >= W->n >= 1.
 *  W:  R_q set (codes and scales 4-byte aligned), with k > 0 also S, Ut_q and
 *      Vt_q; U, V and Rt_q are not read. Unsplit (k == 0) weights may have any
 *      number of rows and any multiple of the block (32 or 16) of columns.
 *  y:  tokens x W->m of type ydt, rounded once from fp32.
 *  ws: metis_fp4_gemv_workspace_bytes() bytes, 256-byte aligned; NULL is fine
 *      where that is 0 (bf16 x and k == 0).
 * Any number of tokens is taken, 64 at a time (21 where x is fp32), and W is
 * read once for each of these, so that beyond a few hundred tokens quantizing x
 * for spectral_fp4_linear_fwd is faster. Values below 2^-126 may be taken as 0. A NaN or an infinity in x
 * spoils its own token. Bitwise reproducible. */
size_t metis_fp4_gemv_workspace_bytes(int64_t tokens, metis_dtype_t dt, const metis_split_t *W);
metis_status_t metis_fp4_gemv(const void *x, metis_dtype_t dt, int64_t tokens, int64_t ldx, const metis_split_t *W,
                              void *y, metis_dtype_t ydt, int64_t ldy, void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Paged FP4 cache of keys and values. k and v are two FP4 matrices of
 * pages * heads * page_size rows and head_dim columns (k.cols == v.cols): the
 * row of place s in page p for head h is (p * heads + h) * page_size + s.
 *  head_dim: a multiple of 32, at most 256 (beyond: METIS_ERR_UNSUPPORTED), in
 *      both formats; at most 2^31 - 1 rows. page_size may be any number >= 1.
 *  NVFP4: the tensor scales are the caller's and are read only: tensor_scale
 *      of k and v has to be set to a positive normal number before anything is
 *      stored (largest magnitude expected / 2688); larger values saturate. */
typedef struct {
  int64_t pages;
  int32_t page_size, heads;
  metis_fp4_t k, v;
} metis_kv_cache_t;

/* A batch of sequences that new tokens belong to (device arrays).
 *  table:   int32, seqs x max_pages, leading dimension ldt: the pages of each
 *           sequence in order; entries behind its last page are not read.
 *  lengths: int32[seqs]: tokens of each sequence with its new ones. 0 or less:
 *           the sequence is not in use.
 *  starts:  int32[seqs + 1]: the new tokens of sequence s are the rows
 *           starts[s] .. starts[s + 1] - 1, its last ones in order; NULL: one
 *           new token each, row s of sequence s. Rows outside belong to none.
 *           starts should not decrease. Where they do, a row that several
 *           sequences claim is one and the same sequence's in all calls, or
 *           none's: the s that a bisection finds for starts[s + 1] > row.
 * A new token i of n of a sequence of length L is at position L - n + i;
 * negative positions are no tokens. A sequence whose rows reach outside the
 * call's tokens is left out. max_pages * page_size <= 2^28. */
typedef struct {
  const int32_t *table, *lengths, *starts;
  int64_t ldt;
  int32_t seqs, max_pages;
} metis_kv_batch_t;

/* Stores new tokens' keys and values into the cache, the keys turned by the
 * angles of their positions on the way.
 *  k, v:  tokens x (heads * head_dim) of type dt.
 *  rope, rope_rows, rot_dim, pairs: as for metis_qk_norm_rope_fwd; NULL with
 *         rot_dim = 0 stores the keys as they are. The rotation is formed in
 *         fp64 and rounded once to fp32.
 * Each row of a head is then quantized as fp4_block_quant does with the
 * cache's tensor scale. A row that belongs to no sequence, and a token whose
 * position is outside the table or the rope, or whose page is outside
 * [0, pages), is not stored; nothing else in the cache changes. A page that a
 * call writes to may stand only once in the tables: in one sequence's, in one
 * place of it. */
metis_status_t metis_kv_append(const void *k, int64_t ldk, const void *v, int64_t ldv, metis_dtype_t dt,
                               int64_t tokens, const metis_kv_batch_t *batch, const float *rope, int64_t rope_rows,
                               int32_t rot_dim, metis_rope_t pairs, const metis_kv_cache_t *cache, hipStream_t stream);

/* Attention of the new tokens over the cache (their own keys and values
 * stored already): for the query at position p of a sequence
 *   o = sum_t softmax_t(scale q . k_t) v_t,  t in (p - window, p]  (window 0:
 *   all t <= p).
 *  q:      tokens x (heads * head_dim) of type dt, tokens * heads < 2^24;
 *          heads a multiple of the cache's: query head h reads head h / (heads / cache->heads).
 *  o:      tokens x (heads * head_dim) of type odt, rounded once from fp32. A
 *          new token that sees nothing (a sequence not in use, a negative
 *          position) gives zeros; rows that belong to no sequence are left as
 *          they were. A page outside [0, pages) below a query's position, or a
 *          length beyond the table, makes its output NaN, never an
 *          out-of-bounds read.
 *  lse:    optional fp32, tokens x heads: log sum_t exp(scale q . k_t), -inf
 *          where nothing is seen (to join with attention over other tokens).
 *  max_new: an upper bound of the new tokens of any sequence (1 without
 *          starts); those beyond it are left as they were.
 *  max_length: about the most tokens that a query sees, the largest length or
 *          with a window the window, which the work is divided by (any value
 *          >= 1 gives the same result but for rounding; the true one the best
 *          speed). The lengths themselves stay on the device.
 *  ws:     metis_kv_attention_workspace_bytes() bytes, 256-byte aligned.
 * Queries and keys enter the products as they are (fp32 queries as three bf16
 * parts), the weights exp(score - max) as three bf16 parts, all of their bits;
 * scores, sums and o in fp32. Bitwise reproducible. A NaN or an infinity in q
 * makes its own row's o and lse NaN, as do scores that are all -inf by overflow;
 * one in the cache spoils every new token's of its sequence and head, in the rows
 * that the kernel works on with it. */
size_t metis_kv_attention_workspace_bytes(int64_t tokens, int32_t heads, int32_t max_new, int64_t max_length,
                                          const metis_kv_batch_t *batch, const metis_kv_cache_t *cache);
metis_status_t metis_kv_attention(const void *q, metis_dtype_t dt, int64_t tokens, int64_t ldq, int32_t heads,
                                  const metis_kv_batch_t *batch, const metis_kv_cache_t *cache, int32_t max_new,
                                  int64_t max_length, float scale, int64_t window, void *o, metis_dtype_t odt,
                                  int64_t ldo, float *lse, void *ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* METIS_FP4_H */
