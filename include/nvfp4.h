/*
 * nvfp4.h -- C ABI of the MI355X (gfx950) NVFP4 W4A4 library.
 *
 * The library implements the data-parallel hot path of NVFP4 W4A4 inference of linear
 * layers:
 *   1. activation quantization: per 16-element block a max-abs, an E4M3 block scale under
 *      an FP32 global scale, round-to-nearest-even to E2M1 codes packed two per byte;
 *   2. the block-scaled 4-bit x 4-bit GEMM Y = A . W^T with FP32 accumulation;
 *   3. the fused-module GEMM in which several separately calibrated modules share one
 *      launch and each column segment keeps its own weight global scale (the repair of the
 *      global-scale mismatch);
 *   4. the GEMM whose output leaves already quantized to NVFP4 for the next linear layer;
 *   5. the FP8 (E4M3) key-value cache codec with calibrated per-tensor scales;
 *   6. the fused Gated DeltaNet input projection whose two gate segments leave as the
 *      write strength and the log-space decay, in the same launch;
 *   7. a lossy variant: NVFP4 re-encoded to MXFP4 and multiplied with gfx950's native scaled
 *      FP4 matrix instructions;
 *   8. the gated MLP input projection: the fused gate+up GEMM with its SwiGLU activation in
 *      the same launch, the result optionally leaving as NVFP4 for the down projection;
 *   9. batch-1 decode of one linear layer in one launch: 1 and 2 with the token's quantization
 *      inside the GEMM kernel;
 *  10. the attention half of the hybrid model around the key-value cache: per-head norms of
 *      queries and keys with the position rotation, appending keys and values to a paged cache
 *      (FP8 as in 5, or bf16), and attention of new tokens over that cache.
 *
 * Sources: the element format (E2M1 values, one E4M3 scale per 16-element block) is from
 * "NVFP4 W4A4 Quantization Compresses 27B Hybrid Models" (thevalue.engineering), section
 * "Challenging the Recurrence Fragility Assumption"; W4A4 on every linear layer and the
 * 16-element block from "Why Gated DeltaNet Survives 4-Bit Quantization" (kipquest),
 * "The deep dive"; the global-scale mismatch (modules calibrated one by one, run as one
 * fused GEMM under a single scale) and its repair from the paper's abstract (Lattice and
 * kipquest pages).  Each declaration below names the passage its operation follows.
 *
 * Data format (identical for activations and weights):
 *   codes [rows, cols/2]  uint8, row-major, contiguous; two 4-bit E2M1 codes per byte, the
 *                         even column in the low nibble.  Code = sign<<3 | magnitude index,
 *                         magnitudes {0, 0.5, 1, 1.5, 2, 3, 4, 6}.
 *   scales [rows, cols/16] uint8, row-major, contiguous; OCP E4M3FN bytes (bias 7,
 *                         max 448, never NaN), one per 16 consecutive elements of a row.
 *   global scale          float32 on the device: one per tensor, or one per row.
 *   value = E2M1(code) * E4M3(scale) * global_scale.
 *   The dynamic global scale is s_g = fl32(max|x| / 2688), 2688 = 6 * 448.
 *
 * Conventions of every entry point:
 *   * Pointers are DEVICE pointers unless marked (host).  The caller owns all memory; the
 *     library never allocates device memory and never synchronises.  Its only state is set up
 *     once per device by the first call that launches work there (kernel limits, the compute-
 *     unit count, the address of nvfp4_quantize_no_alloc's static array), under std::call_once,
 *     for the device the call's stream belongs to: first calls from several host threads at
 *     once are safe.
 *   * Work is enqueued on `stream` (a hipStream_t passed as void*; NULL = default stream)
 *     and is stream-ordered; the global scales never travel to the host.
 *   * Return value: an nvfp4_status.  Argument errors are detected on the host before any
 *     launch and leave every output untouched.  A failed launch returns NVFP4_ERR_HIP.
 *   * Non-finite input is reported in band: the affected global scale (of the tensor, or of
 *     the row in per-row mode) becomes NaN or infinite and the codes and scales it governs
 *     are unspecified.
 *   * Calls on different streams may run concurrently if their outputs and workspaces do
 *     not overlap.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_INVALID_ARG = 1, /* null pointer, bad size, misalignment, bad enum */
  NVFP4_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. too many segments) */
  NVFP4_ERR_WORKSPACE = 3,   /* workspace missing or smaller than the *_workspace_size */
  NVFP4_ERR_HIP = 4          /* a HIP runtime call or kernel launch failed */
} nvfp4_status;

/* NVFP4_E4M3 (OCP E4M3FN bytes under a calibrated scale) is a type of paged caches only. */
typedef enum { NVFP4_F32 = 0, NVFP4_BF16 = 1, NVFP4_E4M3 = 2 } nvfp4_dtype;

typedef enum {
  NVFP4_SCALE_PER_TENSOR = 0, /* s_g = max|x| over the tensor / 2688, written to [1]    */
  NVFP4_SCALE_PER_ROW = 1,    /* s_g[r] = max|x[r,:]| / 2688, written to [rows]         */
  NVFP4_SCALE_GIVEN = 2       /* s_g read from global_scale[0] (a calibrated scale)     */
} nvfp4_scale_mode;

#define NVFP4_MAX_SEGMENTS 64

/*
 * Quantize X[rows, cols] to NVFP4 (format above).  The element format -- E2M1 values with one
 * E4M3 scale per 16-element block -- is the one "NVFP4 W4A4 Quantization Compresses 27B Hybrid
 * Models" describes ("Challenging the Recurrence Fragility Assumption"); "Why Gated DeltaNet
 * Survives 4-Bit Quantization" ("The deep dive") quantizes activations this way at every
 * linear layer, the block of sixteen confining an outlier channel's damage to its own block.
 * The pages imply an FP32 per-module global scale (the mismatch in the paper abstract) without
 * its formula: s_g = fl32(max|x| / 2688) is this library's reading.
 *   x             [rows, ldx] of x_dtype (NVFP4_BF16 or NVFP4_F32); 16-byte aligned, and
 *                 ldx * element size a multiple of 16 bytes; ldx >= cols.
 *   rows >= 0     rows == 0 is a no-op except that PER_TENSOR writes s_g = 0.
 *   cols > 0      multiple of 16.
 *   codes         out [rows, cols/2], 8-byte aligned.
 *   scales        out [rows, cols/16].
 *   global_scale  PER_TENSOR: out [1]; PER_ROW: out [rows]; GIVEN: in [1].  A given scale
 *                 must be finite and > 0 (otherwise the output is unspecified); a zero
 *                 scale (all-zero input) gives all-zero scale bytes and sign-only codes.
 *   workspace     device scratch of nvfp4_quantize_workspace_size() bytes (may be NULL if
 *                 that is 0); contents need no initialisation and are clobbered.
 * Follows: block max -> E4M3 scale -> E2M1 round-to-nearest-even, two codes per byte.
 */
int nvfp4_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                   uint8_t* codes, uint8_t* scales, float* global_scale, int mode,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace nvfp4_quantize needs for this shape and mode (4 KB per tensor, 0
 * per row or given); 0 for a bad shape. */
size_t nvfp4_quantize_workspace_size(int64_t rows, int64_t cols, int mode);

/*
 * nvfp4_quantize for callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc.  Same arguments, results and errors as
 * nvfp4_quantize, without the workspace: the per-tensor mode's partial maxima go to a static
 * device array of the library (4 KB per GPU, held until the process ends) instead.  Allocates
 * nothing, on the host or the device.
 *   Every call on one GPU shares that GPU's array, so calls that overlap in time on one GPU
 *   (different streams, or threads without ordering) race and may return wrong results;
 *   serialise them.  Calls on one stream are ordered and safe.
 *   A shape whose workspace need exceeds the array returns NVFP4_ERR_WORKSPACE (no shape
 *   does at present: the need is at most 4 KB).
 */
int nvfp4_quantize_no_alloc(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                            uint8_t* codes, uint8_t* scales, float* global_scale, int mode, void* stream);

/*
 * The W4A4 linear layer: weights and activations both in the 4-bit block format, as "Why Gated
 * DeltaNet Survives 4-Bit Quantization" ("The deep dive") runs every linear layer of the hybrid
 * model; the paper abstract credits this recipe with the fastest prefill of those compared.
 * Y[M, N] = A . W^T with A = NVFP4 [M, K] activations and W = NVFP4 [N, K] weights, both
 * K-major; FP32 accumulation of the exactly dequantized operands, then
 * y = (acc * a_global[m or 0]) * w_global[0], stored as y_dtype (bf16: round to nearest
 * even).
 *   M >= 0, N >= 0 (zero is a no-op), K > 0 and a multiple of 16.
 *   a_codes, a_scales, w_codes, w_scales 16-byte aligned.
 *   a_global      device [1] (a_global_per_row == 0) or [M] (== 1).
 *   w_global      device [1].
 *   y             [M, ldy] of y_dtype, ldy >= N.
 *   workspace     nvfp4_gemm_workspace_size(M, N, K) bytes (may be NULL if 0; every
 *                 shape needs 0 bytes at present, the argument keeps the ABI stable).
 */
int nvfp4_gemm(int64_t M, int64_t N, int64_t K,
               const uint8_t* a_codes, const uint8_t* a_scales, const float* a_global,
               int a_global_per_row,
               const uint8_t* w_codes, const uint8_t* w_scales, const float* w_global,
               void* y, int y_dtype, int64_t ldy,
               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Batch-1 decode of one W4A4 linear layer in one call: the token's activation row is quantized
 * to the 4-bit block format and multiplied with W, as every linear layer of the hybrid model
 * runs at decode ("Why Gated DeltaNet Survives 4-Bit Quantization", "The deep dive": 4-bit
 * weights and activations).  The result is that of
 *   nvfp4_quantize(x, x_dtype, 1, K, K, a_codes, a_scales, a_global, mode, ...)
 *   nvfp4_gemm(1, N, K, a_codes, a_scales, a_global, 0, w_codes, w_scales, w_global, y, y_dtype, N, ...)
 * on the same stream: the token's NVFP4 bytes are written to a_codes / a_scales (and its global
 * scale to a_global, except in NVFP4_SCALE_GIVEN mode, where a_global is read), bit for bit those
 * of nvfp4_quantize, and Y[1, N] to y.  Y is bit for bit that of nvfp4_gemm except where the one
 * launch below runs and nvfp4_gemm takes an MFMA kernel for the shape (bf16 input, K a multiple
 * of 256, N above 32 x the CU count): there both are within nvfp4_gemm's rounding bound of the
 * exact product, accumulated in a different order.
 * With one row NVFP4_SCALE_PER_TENSOR and NVFP4_SCALE_PER_ROW are the same scale; neither needs a
 * workspace here.  For bf16 input with K a multiple of 64 whose working set fits the kernel's
 * 160 KB of LDS (the token twice, as bf16 and as fp16 values, plus the weight copy rings: K up to
 * 18432 for N up to 32512 on 256 CUs) it is one launch that quantizes the token inside the GEMM
 * kernel, with no separate quantize launch; other inputs run the two calls above internally.
 *   N >= 0 (zero: only the quantization), K > 0 and a multiple of 16.
 *   x             device [K] of x_dtype, 16-byte aligned.
 *   a_codes       out [K/2], a_scales out [K/16], both 16-byte aligned; a_global device [1].
 *   w_codes, w_scales, w_global, y_dtype as in nvfp4_gemm; y device [N] of y_dtype.
 */
int nvfp4_decode_linear(int64_t N, int64_t K, const void* x, int x_dtype, int mode,
                        uint8_t* a_codes, uint8_t* a_scales, float* a_global,
                        const uint8_t* w_codes, const uint8_t* w_scales, const float* w_global,
                        void* y, int y_dtype, void* stream);

/*
 * The fused-module GEMM, the repair of the global-scale mismatch the paper abstract reports
 * (modules calibrated one by one, each with its own global scale, served by a kernel that fuses
 * them into one GEMM); "Quantizing All Layers Reveals Recurrent Memory Is Robust" ("Block
 * Scaling and the Geography of Outliers") describes the bug as a single scale applied to every
 * fused module.  W is the concatenation along N of num_segments separately
 * quantized modules (codes [sum N_i, K/2], scales [sum N_i, K/16]); output column n of
 * segment i is scaled by that module's own global scale w_globals[i]:
 *   Y[:, off_i : off_i + N_i] = A . W_i^T,  off_i = N_0 + ... + N_{i-1}.
 * One launch; one shared activation quantization.  This is the repair of the global-scale
 * mismatch: a kernel that applied one scale to every segment would mis-scale segment i by
 * w_globals[0] / w_globals[i].
 *   1 <= num_segments <= NVFP4_MAX_SEGMENTS; seg_n (host) widths, each > 0.
 *   w_globals     device [num_segments].
 *   Other arguments as in nvfp4_gemm, with N = sum of seg_n.
 */
int nvfp4_gemm_fused_segments(int64_t M, int64_t K,
                              const uint8_t* a_codes, const uint8_t* a_scales,
                              const float* a_global, int a_global_per_row,
                              int num_segments, const int64_t* seg_n,
                              const uint8_t* w_codes, const uint8_t* w_scales,
                              const float* w_globals,
                              void* y, int y_dtype, int64_t ldy,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * The (fused-module) GEMM with its output quantized to NVFP4 for the next linear layer, in
 * the same launch: Y is never written in bf16 or fp32.  Every linear layer takes 4-bit
 * activations ("Why Gated DeltaNet Survives 4-Bit Quantization", "The deep dive"), so a layer
 * whose output feeds another linear layer can hand it over already quantized.  For every output element the fp32
 * value y = (acc * a_global[m or 0]) * w_globals[seg(n)] is the one nvfp4_gemm_fused_segments
 * would store as fp32 for the same shape; each 16-column block of an output row is then
 * encoded exactly as nvfp4_quantize in NVFP4_SCALE_GIVEN mode encodes it under
 * y_global[0] (block max -> E4M3 scale -> E2M1 round-to-nearest-even).  The output global
 * scale is given (a calibrated, static scale): a dynamic per-tensor scale would need the
 * whole output before the first block could be encoded.  Format and encoding as for
 * nvfp4_quantize (sources in the file header).
 *   N = sum of seg_n, a multiple of 16; K a multiple of 128 below 2^24, and for M > 16 a
 *   multiple of 256 (other shapes: NVFP4_ERR_UNSUPPORTED).
 *   y_global      device [1], in: finite and > 0.
 *   y_codes       out [M, N/2], 16-byte aligned; y_scales out [M, N/16], 16-byte aligned.
 *   Other arguments as in nvfp4_gemm_fused_segments (one segment: a plain GEMM).
 */
int nvfp4_gemm_nvfp4_out(int64_t M, int64_t K,
                         const uint8_t* a_codes, const uint8_t* a_scales,
                         const float* a_global, int a_global_per_row,
                         int num_segments, const int64_t* seg_n,
                         const uint8_t* w_codes, const uint8_t* w_scales,
                         const float* w_globals,
                         const float* y_global, uint8_t* y_codes, uint8_t* y_scales,
                         void* stream);

/*
 * The fused Gated DeltaNet (GDN) input projection with its gate epilogue, in one launch.  The
 * GDN block has two gate projections, one setting how strongly the recurrent state is written
 * and one how much of it decays per step; the write strength goes through a sigmoid and the
 * decay is parameterized in log space through softplus and exponential ("Why Gated DeltaNet
 * Survives 4-Bit Quantization" (kipquest), "The deep dive", incl. its scope paragraph;
 * "Quantizing All Layers Reveals Recurrent Memory Is Robust" (freegardner), "The Gates That
 * Were Supposed to Break").  The pages print no formula; this is the standard GDN gate
 * parameterization that matches their description.
 * The last two segments are the gate projections, of equal width H (one column per value
 * head): the write-strength projection b, then the decay projection a.  Y is written exactly
 * as nvfp4_gemm_fused_segments writes it (all N columns, gate pre-activations included); in
 * addition, from each gate column's fp32 value y (before any rounding to y_dtype), for row m
 * and head j:
 *   beta[m, j] = 1 / (1 + exp(-y_b[m, j]))                           (write strength)
 *   g[m, j]    = -exp(a_log[j]) * softplus(y_a[m, j] + dt_bias[j])   (log decay; decay = e^g)
 * with softplus(z) = ln(1 + e^z), evaluated in fp32 without overflow.
 *   2 <= num_segments <= NVFP4_MAX_SEGMENTS, seg_n[num_segments-2] == seg_n[num_segments-1] = H.
 *   a_log, dt_bias  device [H] fp32, 4-byte aligned (per-head parameters).
 *   g, beta         device out [M, H] fp32, row-major, contiguous, 4-byte aligned.
 *   Other arguments as in nvfp4_gemm_fused_segments.
 */
int nvfp4_gemm_fused_gdn_gates(int64_t M, int64_t K,
                               const uint8_t* a_codes, const uint8_t* a_scales,
                               const float* a_global, int a_global_per_row,
                               int num_segments, const int64_t* seg_n,
                               const uint8_t* w_codes, const uint8_t* w_scales,
                               const float* w_globals,
                               void* y, int y_dtype, int64_t ldy,
                               const float* a_log, const float* dt_bias, float* g, float* beta,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace the GEMM entry points need for this shape: 0 for every shape at
 * present (decode reduces K inside the workgroup); kept so the ABI need not change. */
size_t nvfp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * Lossy re-encoding of an NVFP4 tensor to MXFP4, the block-scaled 4-bit format that gfx950's
 * scaled FP4 matrix instructions take: E2M1 codes with one E8M0 scale (a power of two,
 * 2^(byte - 127)) per 32 consecutive elements of a row (OCP Microscaling (MX) specification
 * v1.0).  Each 32-element block (two NVFP4 blocks) is re-encoded from its exact NVFP4 values
 * v = E2M1 * E4M3 (the NVFP4 element format: "NVFP4 W4A4 Quantization Compresses 27B Hybrid
 * Models", "Challenging the Recurrence Fragility Assumption"), leaving the tensor's global
 * scale aside (it stays the multiplier of the MXFP4 tensor, unchanged):
 *   e = floor(log2(max |v|)) - 2 (the MX specification's shared exponent for E2M1),
 *   mx_scales byte = e + 127,  magnitude = E2M1_RNE_SAT(|v| / 2^e),  sign bit kept;
 *   a block of zeros gets byte 0 and magnitude 0.
 * Lossy by design: the E4M3 mantissa of each block scale is dropped and both 16-element halves
 * share one power-of-two scale.
 *   cols > 0 and a multiple of 32; rows >= 0 (0 is a no-op).
 *   codes     [rows, cols/2] NVFP4 codes, 16-byte aligned;  scales [rows, cols/16] E4M3, 2-byte aligned.
 *   mx_codes  out [rows, cols/2], 16-byte aligned (may be codes itself: in place);
 *   mx_scales out [rows, cols/32] E8M0 bytes.
 */
int nvfp4_to_mxfp4(int64_t rows, int64_t cols, const uint8_t* codes, const uint8_t* scales,
                   uint8_t* mx_codes, uint8_t* mx_scales, void* stream);

/*
 * The (fused-module) GEMM on MXFP4 operands with the scaled FP4 MFMA (fp32 accumulation):
 *   Y[m, n] = (sum_k E2M1(a_mk) 2^(sa_m,k/32 - 127) E2M1(w_nk) 2^(sw_n,k/32 - 127))
 *             * a_global[m or 0] * w_globals[seg(n)],
 * stored as fp32 or bf16 (round to nearest even).  Operands as nvfp4_to_mxfp4 writes them;
 * the global scales are the NVFP4 tensors' own.  With the operands re-encoded from NVFP4 this
 * is a lossy variant of nvfp4_gemm_fused_segments.
 *   K a multiple of 256 below 2^24 (other K: NVFP4_ERR_UNSUPPORTED); any M >= 0 (M <= 16 runs
 *   a decode kernel that streams W).  a_scales [M, K/32], w_scales [N, K/32], 16-byte aligned.
 *   Other arguments as in nvfp4_gemm_fused_segments (one segment: a plain GEMM).
 */
int nvfp4_mxfp4_gemm(int64_t M, int64_t K,
                     const uint8_t* a_codes, const uint8_t* a_scales,
                     const float* a_global, int a_global_per_row,
                     int num_segments, const int64_t* seg_n,
                     const uint8_t* w_codes, const uint8_t* w_scales,
                     const float* w_globals,
                     void* y, int y_dtype, int64_t ldy, void* stream);

/*
 * Interleave the gate and up projections of a gated (SwiGLU) MLP into the weight layout
 * nvfp4_gemm_swiglu takes: rows 32p .. 32p+15 of w are gate rows 16p .. 16p+15 and rows
 * 32p+16 .. 32p+31 the up rows 16p .. 16p+15 (codes and scale bytes alike), so that each
 * 32-row group holds both projections of 16 hidden units.  A one-time weight preparation (a
 * pure row permutation, stream-ordered device-to-device copies); the two projections keep
 * their own global scales, passed to nvfp4_gemm_swiglu as {gate, up}.
 *   F > 0 and a multiple of 16 (hidden width); K > 0 and a multiple of 16.
 *   gate_codes, up_codes    [F, K/2];  gate_scales, up_scales [F, K/16]   (device, contiguous).
 *   w_codes  out [2F, K/2];  w_scales out [2F, K/16]  (device, contiguous; must not overlap
 *   the inputs).
 */
int nvfp4_interleave_gate_up(int64_t F, int64_t K,
                             const uint8_t* gate_codes, const uint8_t* gate_scales,
                             const uint8_t* up_codes, const uint8_t* up_scales,
                             uint8_t* w_codes, uint8_t* w_scales, void* stream);

/*
 * The gated MLP input projection in one launch: the fused gate+up GEMM of the quantized
 * feed-forward block (paper abstract: NVFP4 W4A4 on all linear layers; "Why Gated DeltaNet
 * Survives 4-Bit Quantization", "The deep dive") with its SwiGLU activation and, optionally,
 * the NVFP4 encoding of the result for the down projection.  The pages do not name the MLP's
 * activation; this is the gated SiLU (SwiGLU) block of the Qwen family:
 *   y_gate[m, j], y_up[m, j] = the fp32 GEMM outputs (acc * a_global[m or 0]) * w_globals[0
 *   or 1] of hidden unit j, as nvfp4_gemm_fused_segments computes them for the segments
 *   [gate, up];
 *   h[m, j] = silu(y_gate) * y_up,  silu(y) = y * sigmoid(y) = y / (1 + e^-y)  (fp32).
 * h is stored as fp32 or bf16 (round to nearest even) when h is given, and as NVFP4 when
 * h_codes is given: each 16-element block of a row encoded exactly as nvfp4_quantize in
 * NVFP4_SCALE_GIVEN mode encodes it under h_global[0] (a calibrated, static scale).  At least
 * one of the two outputs is required.
 *   F > 0, a multiple of 16 (hidden width); K a multiple of 128 below 2^24, and for M > 16 a
 *   multiple of 256 (other shapes: NVFP4_ERR_UNSUPPORTED); M * F < 2^31.
 *   w_codes [2F, K/2], w_scales [2F, K/16]: the interleaved layout of nvfp4_interleave_gate_up.
 *   w_globals device [2] = {gate, up}.
 *   h       out [M, F] of h_dtype, row pitch ldh >= F elements, or NULL.
 *   h_global device [1], finite and > 0; h_codes out [M, F/2], h_scales out [M, F/16], both
 *   16-byte aligned; all three NULL when no NVFP4 output is wanted.
 *   Other arguments as in nvfp4_gemm.
 */
int nvfp4_gemm_swiglu(int64_t M, int64_t F, int64_t K,
                      const uint8_t* a_codes, const uint8_t* a_scales,
                      const float* a_global, int a_global_per_row,
                      const uint8_t* w_codes, const uint8_t* w_scales, const float* w_globals,
                      void* h, int h_dtype, int64_t ldh,
                      const float* h_global, uint8_t* h_codes, uint8_t* h_scales, void* stream);

/*
 * FP8 key-value cache codec with a calibrated per-tensor scale (the pages' second serving
 * finding: calibrated FP8 KV-cache scales are performance-free -- paper abstract;
 * "Quantizing All Layers Reveals Recurrent Memory Is Robust", "The Calibrated Cache That
 * Ships for Free"; "NVFP4 W4A4 Quantization Compresses 27B Hybrid Models", "Efficiency Gains
 * and Serving Optimization").  FP8 is the OCP E4M3FN byte of the file header; the tensor is
 * treated as n contiguous elements (e.g. a K or V cache flattened).
 *   quantize:   q[i] = sign | E4M3_RNE_SAT(fl32(|x[i]| / scale[0])) (round to nearest even,
 *               saturating at 448; +-inf -> +-448; NaN -> 0x7F).
 *   dequantize: y[i] = fl32(E4M3(q[i]) * scale[0]) as y_dtype (bf16: round to nearest even);
 *               0x7F / 0xFF -> NaN.
 *   x             [n] of x_dtype, 16-byte aligned.   q   [n] bytes, 8-byte aligned.
 *   y             [n] of y_dtype, 16-byte aligned.   scale device [1], finite and > 0.
 *   n >= 0        n == 0 is a no-op.
 */
int nvfp4_fp8_kv_quantize(const void* x, int x_dtype, int64_t n, const float* scale, uint8_t* q,
                          void* stream);
int nvfp4_fp8_kv_dequantize(const uint8_t* q, int64_t n, const float* scale, void* y, int y_dtype,
                            void* stream);

/*
 * Operators of the attention layers around a paged key-value cache (the calibrated FP8 cache of
 * the codec above, or bf16).  A cache is a pool of pages; each sequence owns the pages its row of
 * the page table lists, in order.
 */

/* Head vectors x[t, h, 0 .. dim-1]: rows of `dim` contiguous elements at t * token_stride + h *
 * head_stride (elements), so that q, k and v may be column ranges of one fused projection.
 * data 16-byte aligned; both strides (of a dimension longer than one) times the element size a
 * multiple of 16 bytes, head_stride >= dim, token_stride >= 0; an output's rows must not overlap. */
typedef struct {
  void* data;
  int64_t heads;
  int64_t token_stride;
  int64_t head_stride;
} nvfp4_heads;

/* A paged cache and the batch of sequences it serves (host struct; pointers are device pointers).
 *   k, v         page p is [kv_heads, page_size, head_dim] contiguous at p * page_stride
 *                elements; NVFP4_E4M3 or NVFP4_BF16; 16-byte aligned, page strides times the element
 *                size multiples of 16 bytes (k and v may be interleaved in one allocation).
 *   page_size    tokens per page: a power of two, 16 to 1024.
 *   num_pages    at least 1, below 2^31.
 *   page_table   int32 [num_seqs, table_width], row pitch table_stride: token position t of
 *                sequence s lies in page page_table[s][t / page_size], row t % page_size.  An entry
 *                outside [0, num_pages) stands for no page: appends to it are dropped, its keys are
 *                attended by nobody (entries past a sequence's length are never read).
 *   k_scale, v_scale  device fp32, the calibrated scales of an E4M3 cache (finite and > 0, value =
 *                E4M3(byte) * scale): one, or one per key-value head (scale_count = 1 or kv_heads).
 *                Ignored for bf16.
 *   cu_q         int32 [num_seqs + 1]: the new tokens of sequence s are rows cu_q[s] ..
 *                cu_q[s+1] - 1 of q, k and v (non-decreasing; rows before cu_q[0] or from
 *                cu_q[num_seqs] on belong to nobody and their outputs are left as they were).
 *   kv_len       int32 [num_seqs]: tokens of the sequence in the cache, new ones included, at most
 *                table_width * page_size: new token i of n has position kv_len - n + i.
 * cu_q, kv_len and the page table are read on the device by the kernels, so a captured graph
 * follows their contents.  A value out of range never makes a kernel access memory outside the
 * operands: attention clamps cu_q to the call's rows and kv_len to what the table holds, appending
 * drops the tokens whose place is outside. */
typedef struct {
  void* k;
  void* v;
  int64_t num_pages;
  int64_t k_page_stride;
  int64_t v_page_stride;
  const int32_t* page_table;
  int64_t table_stride;
  const float* k_scale;
  const float* v_scale;
  const int32_t* cu_q;
  const int32_t* kv_len;
  int32_t dtype;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_seqs;
  int32_t table_width;
  int32_t scale_count;
} nvfp4_paged_kv;

/* The position rotation: channel pairs of the first `dim` channels of each head are turned by the
 * angles of the token's position, read from a table of cos (dim/2 values) then sin (dim/2) per
 * position, fp32 [rows, dim] contiguous, 16-byte aligned:
 *   y[a] = x[a] cos_i - x[b] sin_i,  y[b] = x[b] cos_i + x[a] sin_i,  i < dim/2,
 * (a, b) = (i, i + dim/2), or (2i, 2i + 1) with interleaved = 1.  dim is a multiple of 16, at most
 * the head dimension; the other channels pass through.
 *   positions    device int32, one per token (NULL: see the entry point).  A position outside
 *                [0, rows) has no angles: the rotated channels of that token become NaN. */
typedef struct {
  const float* table;
  int64_t rows;
  const int32_t* positions;
  int32_t dim;
  int32_t interleaved;
} nvfp4_rope;

/*
 * Norms of queries and keys for each head and the position rotation, in one pass: the input side
 * of the hybrid model's attention layers.  Per head vector, in fp32 and rounded once on the way out:
 *   x <- x * w / sqrt(mean(x^2) + eps)   (when that tensor's weight is given)
 *   x <- rotation of x                     (when rope is given; rope->positions required)
 *   tokens >= 0 (0 is a no-op), head_dim a multiple of 16, 16 to 512.
 *   q, k         inputs of x_dtype (NVFP4_BF16 or NVFP4_F32); k may be NULL.
 *   q_weight, k_weight  device fp32 [head_dim], 16-byte aligned, or NULL; eps >= 0.
 *   q_out, k_out outputs of out_dtype (NVFP4_BF16: round to nearest even, or NVFP4_F32), heads as
 *                the inputs'; may be the inputs themselves if type and layout are equal, and must
 *                not overlap them otherwise.  k_out NULL exactly when k is.
 */
int nvfp4_qk_norm_rope(int64_t tokens, int64_t head_dim, int x_dtype, const nvfp4_heads* q, const nvfp4_heads* k,
                       const float* q_weight, const float* k_weight, float eps, const nvfp4_rope* rope, int out_dtype,
                       const nvfp4_heads* q_out, const nvfp4_heads* k_out, void* stream);

/*
 * Append the new tokens' keys and values to the cache, keys normed and rotated on the way, in one
 * launch; with q given, the queries leave normed and rotated in the same launch.
 *   k: norm (k_weight not NULL) and rotation (rope not NULL) as nvfp4_qk_norm_rope, v as it is; both
 *      stored at the token's position: E4M3 as nvfp4_fp8_kv_quantize encodes the fp32 value under the
 *      head's scale, or bf16 rounded to nearest even.
 *   rope->positions NULL: a token's position is its place in its sequence.
 *   Tokens at a negative place, past the page table or on an invalid page are not stored.  Two tokens
 *   that share a place (sequences that share a page) leave either one's bytes.
 *   tokens >= 0 (0 is a no-op): rows of q, k, v.  kv->head_dim a multiple of 16, 16 to 512.
 *   k, v         of x_dtype, kv->kv_heads heads.
 *   q, q_out     both NULL, or q of x_dtype and q_out of q_out_dtype as in nvfp4_qk_norm_rope.
 */
int nvfp4_kv_append(const nvfp4_paged_kv* kv, int64_t tokens, int x_dtype, const nvfp4_heads* k, const nvfp4_heads* v,
                    const float* k_weight, float eps, const nvfp4_rope* rope, const nvfp4_heads* q,
                    const float* q_weight, int q_out_dtype, const nvfp4_heads* q_out, void* stream);

/*
 * Attention of new tokens over the paged cache (their own keys and values appended before):
 *   out[t, h] = sum_j p_j v_j,  p = softmax_j(scale * q[t, h] . k_j),  key-value head h / (q heads /
 * kv heads), over the keys j the token sees: with causal = 1 those at positions up to its own,
 * and with window > 0 only the last `window` of them; with causal = 0 all kv_len (window must be 0).
 * One call takes any mix of single tokens and chunks.  A token that sees no key (an empty
 * sequence, a position below 0, no valid page), or whose every score is -inf, gets zeros and lse =
 * -inf.  Keys a token does not see have no influence, whatever their bytes hold (NaN, infinities).  An infinite or
 * NaN value at a key it does see reaches its output however small the probability.
 *   q            bf16, heads a multiple of kv->kv_heads, at most 256 per key-value head.
 *   head_dim     64, 128 or 256 (others: NVFP4_ERR_UNSUPPORTED).
 *   table_width * page_size  at most 2^30 (more: NVFP4_ERR_UNSUPPORTED).
 *   scale        > 0 and finite, usually head_dim^-0.5.
 *   max_q        the largest number of new tokens of one sequence, or 0 if not known: a hint that
 *                picks kernels.  Results do not depend on its truth beyond rounding (the order of sums), speed does.
 *   out          bf16 (round to nearest even), heads as q; must not overlap the inputs.
 *   lse          device fp32 [tokens, q heads] contiguous, or NULL: ln sum_j exp(scale q.k_j).
 *   workspace    device, 16-byte aligned, nvfp4_paged_attention_workspace_size() bytes for the same
 *                arguments; contents need no initialisation and are clobbered.
 * Scores, softmax statistics and sums are fp32; probabilities are rounded for their product with V: to fp16 beside an
 * E4M3 cache (2^-11 relative, at most 2^-32 of the row's sum absolute), to bf16 beside a bf16 cache (2^-8
 * relative), whose values may exceed fp16's range.  Deterministic: the same inputs and arguments give the same bits.
 */
int nvfp4_paged_attention(const nvfp4_paged_kv* kv, int64_t tokens, int64_t max_q, const nvfp4_heads* q, float scale,
                          int causal, int64_t window, const nvfp4_heads* out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Bytes of workspace nvfp4_paged_attention needs for these sizes, whatever the lengths: partial
 * results of a key axis split over workgroups.  0 for bad sizes. */
size_t nvfp4_paged_attention_workspace_size(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t q_heads,
                                            int64_t kv_heads, int64_t head_dim, int dtype);

/* Static description of a status code. */
const char* nvfp4_status_string(int status);

/* Library version: major * 10000 + minor * 100 + patch. */
int nvfp4_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H */
