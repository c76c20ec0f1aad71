/*
 * bsq.h -- C ABI of libbsq.so: block-scaled low-precision quantization (MXFP8, NVFP4,
 * MXFP4) and the block-scaled GEMM with a fused bias + bf16 epilogue, for GB300 (sm_103a).
 *
 * The method: the linear layers of a ViT block (qkv, proj, fc1, fc2) run as block-scaled
 * low-precision GEMMs ("lightly-train - DINOv3 + EoMT on RTX 5090" README, section 2 number
 * formats table; sections 4.3 and 5.3 name the quantized GEMMs). A layer is two steps:
 *   1. per-block quantization of a bf16 (or fp32) matrix along its K dimension;
 *   2. out = bf16(alpha * sum_k Ahat[m,k] * Bhat[n,k] + bias[n]), fp32 accumulation.
 *
 * Conventions shared by every entry point
 *   - All buffer pointers are DEVICE pointers, 16-byte aligned (the block norms, expert rows and
 *     gradient norms: element aligned, where not said otherwise), allocated by the caller;
 *     the library allocates no memory and keeps no per-call state. Its only state is one
 *     status word per device (see bsq_get_device_status) and a thread-local last error.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream) and
 *     returns without synchronising, except bsq_get_device_status.
 *   - Matrices are row-major. Quantized operands are "K-major": element (r, k) of a
 *     rows x cols matrix is at r * cols + k (the "TN" GEMM of section 5.5 of the README).
 *   - Return value 0 = enqueued; a negative BSQ_ERR_* = nothing was enqueued (argument
 *     errors) or the launch failed (BSQ_ERR_LAUNCH). Device-side failures (a bounded wait
 *     that gave up) are reported later through bsq_get_device_status.
 *   - Requires a compute capability 10.3 device (GB300); otherwise BSQ_ERR_ARCH.
 */
#ifndef BSQ_H
#define BSQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* bsq_stream_t; /* identical to cudaStream_t */

/* Formats (README section 2, number-format table):
 *   BSQ_MXFP8  E4M3 elements, one UE8M0 (power-of-two) scale per 1x32 block, 8.25 bits/value.
 *   BSQ_NVFP4  e2m1 elements (2 per byte), one E4M3 scale per 1x16 block and one fp32
 *              per-tensor scale g, 4.5 bits/value.
 *   BSQ_MXFP4  e2m1 elements, one UE8M0 scale per 1x32 block, 4.25 bits/value. */
typedef enum { BSQ_MXFP8 = 1, BSQ_NVFP4 = 2, BSQ_MXFP4 = 3 } bsq_format;

/* Flags OR-ed into bsq_quantize's first argument. */
#define BSQ_FMT_MASK 0xFF
#define BSQ_FLAG_SRC_F32 0x100      /* src holds fp32 values; default: bf16 */
#define BSQ_FLAG_GLOBAL_GIVEN 0x200 /* NVFP4: read g from *global_scale instead of computing it
                                       (a static or delayed per-tensor scale, README sections
                                       4.3 and 5.5) */
#define BSQ_FLAG_STOCHASTIC 0x400   /* bsq_quantize_dual: stochastic rounding of the elements */

/* Status codes. */
#define BSQ_OK 0
#define BSQ_ERR_ARG -1     /* null pointer, non-positive size, unknown format or flag */
#define BSQ_ERR_SHAPE -2   /* a size the format or the GEMM cannot tile (see each call) */
#define BSQ_ERR_ALIGN -3   /* a pointer is not 16-byte aligned */
#define BSQ_ERR_ARCH -4    /* no CUDA device, or not compute capability 10.3 */
#define BSQ_ERR_LAUNCH -5  /* the CUDA runtime reported an error at launch */
#define BSQ_ERR_TIMEOUT -6 /* a kernel's bounded wait gave up (device status only) */
#define BSQ_ERR_DEVICE_CHECK -7 /* checked build (libbsq_checked.so) only: a kernel's index check
                                   failed and the access was skipped (device status only) */

/*
 * bsq_codes_bytes: size of the element-code buffer of a rows x cols matrix.
 *   MXFP8: rows * cols bytes (one E4M3 code per byte).
 *   NVFP4, MXFP4: rows * cols / 2 bytes; element 2j in the low nibble of byte j, 2j+1 in
 *   the high nibble. Returns 0 for invalid arguments.
 * Source: the element widths of the README's section 2 number-format table (8-bit E4M3,
 * 4-bit e2m1). The nibble order is a convention: the pages are silent on it.
 */
size_t bsq_codes_bytes(int fmt, int64_t rows, int64_t cols);

/*
 * bsq_scales_bytes: size of the scale buffer of a rows x cols matrix.
 * Source: the block sizes and scale types of the README's section 2 number-format table
 * (one 8-bit scale per 1x32 block for MX, per 1x16 block for NVFP4). The tiled layout below
 * is a convention; the pages are silent on how scales are laid out in memory.
 * Block scales are stored in tiles of 128 rows x 4 scale columns (512 bytes): the scale of
 * row r and block column c lives in tile (r / 128) * ceil(nsc / 4) + c / 4 at byte
 * (r % 32) * 16 + ((r / 32) % 4) * 4 + c % 4, nsc = cols / block size. Rows are padded to
 * 128 and scale columns to 4; padding bytes are written as 0. This is the layout the
 * tensor cores' scale-factor copy consumes, so the GEMM reads it without reshuffling.
 * NVFP4 appends a 16-byte tail {g, amax, 0, 0} (fp32): the per-tensor scale used and the
 * amax of the quantized tensor (the source of a delayed scale for the next call).
 * Returns 0 for invalid arguments.
 */
size_t bsq_scales_bytes(int fmt, int64_t rows, int64_t cols);

/*
 * bsq_quantize: quantize a rows x cols matrix along cols (K) in 1x32 (MX) or 1x16 (NVFP4)
 * blocks.
 *   fmt_flags    bsq_format | BSQ_FLAG_* bits.
 *   src          rows x cols bf16 (default) or fp32 (BSQ_FLAG_SRC_F32) values, finite.
 *   codes        bsq_codes_bytes(fmt, rows, cols) bytes, written.
 *   scales       bsq_scales_bytes(fmt, rows, cols) bytes, written (including padding).
 *   global_scale NVFP4 only, one fp32 in device memory. Without BSQ_FLAG_GLOBAL_GIVEN it
 *                receives g = amax(|src|) / 2688 (may be NULL: g is also in the scale tail);
 *                with the flag it is read as g (must not be NULL). Ignored for MX formats.
 * Rules (README section 2; rounding to nearest even with saturation at the largest finite
 * value, 448 for E4M3 and 6 for e2m1):
 *   MX     per block e = floor(log2(amax)) - emax (emax 8 for E4M3, 2 for e2m1), clamped to
 *          [-127, 127], amax = 0 -> -127; scale byte e + 127; code = RNE_sat(x * 2^-e).
 *   NVFP4  s = E4M3 RNE_sat(bamax / (6 g)); code = e2m1 RNE_sat(x / (s g)), each step one
 *          IEEE fp32 operation; s = 0 gives zero codes carrying the sign of x.
 * Shapes: cols % 32 == 0 (MX) or cols % 16 == 0 (NVFP4), rows and cols below 2^31, else
 * BSQ_ERR_SHAPE; any rows >= 1.
 * Codes and scales are bit-exact functions of the input (no dependence on launch shape).
 */
int bsq_quantize(int fmt_flags, const void* src, int64_t rows, int64_t cols, void* codes, void* scales,
                 float* global_scale, bsq_stream_t stream);

/*
 * bsq_layernorm_quantize: the LayerNorm + quantization kernel of the README's MXFP8 stack
 * ("lightly-train - DINOv3 + EoMT on RTX 5090" README, section 4.3: LN and quantization merged
 * into one kernel). Per row r of a rows x cols matrix:
 *   y[r, c] = (x[r, c] - mean_r) / sqrt(var_r + eps) * gamma[c] + beta[c]
 * with mean_r and the biased variance var_r over the row, in fp32, then y (kept in fp32)
 * quantized along the row as bsq_quantize does: codes and tiled scales of an MX format.
 *   fmt_flags   BSQ_MXFP8 or BSQ_MXFP4, optionally | BSQ_FLAG_SRC_F32
 *   gamma_bf16, beta_bf16   cols bf16 values each, 16-byte aligned
 *   eps         >= 0
 * Codes and scales are the MX quantization of the kernel's fp32 y; a code differs from that of
 * the exact value only where the exact value lies within the fp32 rounding of the statistics
 * and the affine step of a rounding boundary.
 * Work mapping: bf16 rows of at most 1024 elements run one row per warp with the row in
 * registers; other rows are staged through shared memory. Both give the same bytes for the same
 * values.
 * Shapes: as bsq_quantize for MX, and a row of at most 16384 bytes (cols <= 8192 bf16 or 4096
 * fp32), else BSQ_ERR_SHAPE. Errors: BSQ_ERR_ARG for another format or flag, NULL gamma /
 * beta or a negative or non-finite eps; otherwise as bsq_quantize.
 */
int bsq_layernorm_quantize(int fmt_flags, const void* src, const void* gamma_bf16, const void* beta_bf16, float eps,
                           int64_t rows, int64_t cols, void* codes, void* scales, bsq_stream_t stream);

#define BSQ_MAX_BATCH 8
typedef struct {
  const void* src;     /* rows x cols bf16 or fp32 (per fmt_flags) */
  int64_t rows, cols;
  void* codes;         /* bsq_codes_bytes(fmt, rows, cols) bytes, written */
  void* scales;        /* bsq_scales_bytes(fmt, rows, cols) bytes, written */
  float* global_scale; /* NVFP4 only, as bsq_quantize's global_scale; NULL otherwise */
} bsq_quant_item;

/*
 * bsq_quantize_batch: bsq_quantize applied to `count` matrices (1 <= count <= BSQ_MAX_BATCH)
 * in one kernel launch, e.g. a layer's activations and weights together. Every item is
 * validated as in bsq_quantize (its own rows, cols, buffers; global_scale as bsq_quantize's
 * argument) and the whole batch shares fmt_flags (one format, one source type, one
 * NVFP4 scale mode). Results are identical, byte for byte, to `count` bsq_quantize calls.
 * `items` is a host array read during the call only. The batching is an engineering entry
 * point (fewer launches for small matrices); the method itself has no counterpart.
 * Errors: BSQ_ERR_ARG if count is out of range or items is NULL, otherwise the first error
 * any item would give bsq_quantize; nothing is enqueued on an argument error.
 */
int bsq_quantize_batch(int fmt_flags, int count, const bsq_quant_item* items, bsq_stream_t stream);

/*
 * bsq_quantize_dual: dual-layout quantization for the backward GEMMs ("lightly-train - DINOv3 +
 * EoMT on RTX 5090" README, section 4.3, the quantized training stacks: dgrad contracts dY
 * over N and wgrad over M, so dY is needed quantized along both of its dimensions, W along N
 * and X along M; the README's fused FP4 quantizer writes both layouts from one read). From one
 * rows x cols matrix X, in one pass over it:
 *   row_codes, row_scales  the operand bsq_quantize(fmt, X, rows, cols) writes (blocks along
 *                          cols), sized bsq_codes_bytes / bsq_scales_bytes(fmt, rows, cols);
 *   col_codes, col_scales  the operand of X^T (cols x rows, blocks along rows), as
 *                          bsq_quantize(fmt, X^T, cols, rows) would write it, sized
 *                          bsq_codes_bytes / bsq_scales_bytes(fmt, cols, rows).
 * All four are written, scale padding included.
 *   fmt_flags     BSQ_MXFP8, BSQ_MXFP4 or BSQ_NVFP4, | BSQ_FLAG_SRC_F32 (fp32 source, default
 *                 bf16), | BSQ_FLAG_STOCHASTIC, | BSQ_FLAG_GLOBAL_GIVEN (NVFP4 only).
 *   global_scale  NVFP4: one fp32 in device memory, as bsq_quantize's argument (receives the
 *                 computed g, may be NULL; or, with BSQ_FLAG_GLOBAL_GIVEN, supplies g). The one
 *                 g serves both layouts; both scale tails hold {g, amax of X}. Ignored for MX.
 * Block scales follow the rules of bsq_quantize. Without BSQ_FLAG_STOCHASTIC the elements
 * round to nearest even (seed ignored); both layouts are then byte-identical to the two
 * bsq_quantize calls (NVFP4 with the same g). With it (the gradient rounding of quantized
 * training), for v = the element's quotient (MX: x / scale, exact; NVFP4: fp32(x / fp32(s g))):
 * q = |v| / spacing, the spacing of the element format at |v|'s binade (its subnormal step
 * below the smallest normal); |code| = floor(q) + (frac(q) > u), saturating at the largest
 * finite value (448, 6); u = h * 2^-16 with h the 16-bit half i mod 2 (low half first) of word
 * (i mod 8) / 2 of Philox4x32-10 (Salmon et al., "Parallel Random Numbers: As Easy as 1, 2, 3",
 * SC'11) at counter {floor(i/8) low 32 bits, high 32 bits, layout, 0} and key {seed low 32 bits,
 * high 32 bits}; i = r * cols + c in the row layout (layout 0), c * rows + r in the column
 * layout (layout 1). E[code value] = v below saturation wherever frac(q) has at most 16 bits
 * (every bf16 X whose quotient lies in the format's normal range), otherwise within 2^-16 of a
 * spacing; the codes are a function of (X, seed) alone. An NVFP4 block whose
 * scale is 0 gives signed zero codes either way.
 * Shapes: rows % 32 == 0 and cols % 32 == 0, both below 2^31, else BSQ_ERR_SHAPE.
 * Errors: BSQ_ERR_ARG for an unknown format or flag, BSQ_FLAG_GLOBAL_GIVEN without NVFP4 or
 * without global_scale, a NULL buffer or a non-positive size; BSQ_ERR_ALIGN for a buffer not
 * 16-byte aligned or a global_scale not 4-byte aligned.
 */
int bsq_quantize_dual(int fmt_flags, const void* src, int64_t rows, int64_t cols, uint64_t seed, void* row_codes,
                      void* row_scales, void* col_codes, void* col_scales, float* global_scale, bsq_stream_t stream);

/*
 * bsq_delayed_global_scale: the delayed NVFP4 per-tensor scale of quantized training
 * ("lightly-train - DINOv3 + EoMT on RTX 5090" README, section 5.5: the amax found while a
 * tensor is quantized in one step, times a headroom factor, is the next step's scale, so no
 * step spends an extra pass over the tensor on its amax; the README's dY study settles on a
 * headroom of 32). Enqueues one thread computing
 *   *g_out = fp32(fp32(amax * headroom) / 2688)
 * with amax the tail word of prev_scales, an NVFP4 scale buffer of a rows x cols matrix
 * written by bsq_quantize / bsq_quantize_batch / bsq_quantize_dual (either layout's buffer:
 * both tails hold the same amax). Pass g_out to the next quantization of the tensor with
 * BSQ_FLAG_GLOBAL_GIVEN; that call records the new amax in its own tail. Reading the tail and
 * writing g_out are ordered on `stream` only, with no host synchronisation.
 *   prev_scales  bsq_scales_bytes(BSQ_NVFP4, rows, cols) bytes, 16-byte aligned
 *   headroom     finite, > 0
 *   g_out        one fp32 in device memory, 4-byte aligned
 * Errors: BSQ_ERR_ARG (NULL pointer, non-positive size, bad headroom), BSQ_ERR_SHAPE (cols % 16,
 * sizes >= 2^31), BSQ_ERR_ALIGN.
 */
int bsq_delayed_global_scale(const void* prev_scales, int64_t rows, int64_t cols, float headroom, float* g_out,
                             bsq_stream_t stream);

/*
 * bsq_gemm: out[m, n] = bf16_rn(alpha * sum_k Ahat[m,k] * Bhat[n,k] + bias[n]).
 * Source: "lightly-train - DINOv3 + EoMT on RTX 5090" README, section 2 (the block-scaled
 * MXFP8 / NVFP4 / MXFP4 GEMM formats and their tensor-core rates) and section 4.3 (qkv, proj,
 * fc1, fc2 of every block run as these GEMMs, bias fused into the epilogue). Ahat, Bhat are the
 * decoded operands: code value times its block scale (times g for NVFP4, folded into alpha).
 *   A, A_scales  M x K operand as written by bsq_quantize(fmt, ..., M, K, ...).
 *   B, B_scales  N x K operand (the nn.Linear weight layout) from bsq_quantize(fmt, ..., N, K, ...).
 *   bias_bf16    N bf16 values, or NULL for no bias.
 *   out_bf16     M x N bf16, row-major, written.
 *   alpha        1 for MX formats; g_A * g_B for NVFP4, read on the device from the two
 *                scale tails (no host synchronisation).
 * Products are accumulated in fp32 in the tensor cores (tcgen05 block-scaled MMA).
 * Shapes: K % 128 == 0 (MXFP8) or K % 256 == 0 (NVFP4, MXFP4); N % 8 == 0; M >= 1 (rows
 * past M are never written). Otherwise BSQ_ERR_SHAPE.
 */
int bsq_gemm(int fmt, const void* A, const void* A_scales, const void* B, const void* B_scales,
             const void* bias_bf16, void* out_bf16, int64_t M, int64_t N, int64_t K, bsq_stream_t stream);

/*
 * bsq_gemm_splitk: bsq_gemm's result computed with the K dimension cut into `splits` equal
 * ranges of K stages (128 K for MXFP8, 256 for NVFP4 / MXFP4), each (output tile, range) pair
 * one unit of work, for shapes with fewer 256 x 256 output tiles than the GPU has SM pairs and
 * a long K: the weight gradient dW = dY^T X of a linear layer ("lightly-train - DINOv3 + EoMT
 * on RTX 5090" README, section 4.3: the training stacks' wgrad GEMM; M, N the weight's shape, K
 * the token count) has 36 tiles for 76 SM pairs at ViT-B/16 fc1. The method has no split-K of
 * its own: this is an engineering entry point. Each unit stores its raw fp32 sum into slice r
 * of `workspace`; a second kernel adds the slices in order (deterministic) and applies alpha,
 * the bias and the bf16 rounding as bsq_gemm does. The fp32 sum therefore rounds in a different
 * order than bsq_gemm's (within the same tolerance).
 *   splits           1..8 and at most the number of K stages; 1 is bsq_gemm itself
 *   workspace        splits * M * N fp32 in device memory, 16-byte aligned, owned by the caller;
 *                    overwritten, no initial contents needed; unused when splits == 1
 *   workspace_bytes  its size, at least splits * M * N * 4 (else BSQ_ERR_ARG)
 * Other arguments, shapes and errors as bsq_gemm; two launches on `stream`.
 */
int bsq_gemm_splitk(int fmt, const void* A, const void* A_scales, const void* B, const void* B_scales,
                    const void* bias_bf16, void* out_bf16, int64_t M, int64_t N, int64_t K, int splits,
                    void* workspace, size_t workspace_bytes, bsq_stream_t stream);

/*
 * bsq_gemm_splitk_splits: the number of K ranges bsq_gemm_splitk should use on the current
 * device for an M x N x K product: floor(SM pairs / output tiles of 256 x 256), at most 8 and at
 * most K stages / 8 (each range keeps at least 8 stages of the operand pipeline), at least 1 --
 * 2 for ViT-B/16 fc1's weight gradient (36 tiles, 76 SM pairs), 1 for every forward GEMM of the
 * ViT shapes. Returns the count, or a negative error (BSQ_ERR_ARG for an unknown format or a
 * non-positive size, BSQ_ERR_ARCH without a usable device).
 */
int bsq_gemm_splitk_splits(int fmt, int64_t M, int64_t N, int64_t K);

/*
 * bsq_gemm_splitk_scratch: bsq_gemm_splitk with the workspace taken from a fixed 64 MiB device
 * array inside the library instead of a caller buffer, so that a call allocates nothing. The
 * pages describe no counterpart: an engineering entry point.
 *   - The array is placed with the library's device module, once per device; its address is
 *     looked up once per device. No call allocates or frees memory.
 *   - Limit: splits * M * N * 4 bytes <= 64 MiB; a larger request fails with BSQ_ERR_ARG, as
 *     bsq_gemm_splitk does with too small a workspace (splits == 1 needs none).
 *   - Nothing needs to start at zero: each call overwrites the part of the array it uses before
 *     reading it.
 *   - The array is shared by every caller in the process on that device: calls that can overlap
 *     in time (on different streams, or from different host threads) race on it; the caller
 *     orders them.
 * Other arguments, results and errors as bsq_gemm_splitk.
 */
int bsq_gemm_splitk_scratch(int fmt, const void* A, const void* A_scales, const void* B, const void* B_scales,
                            const void* bias_bf16, void* out_bf16, int64_t M, int64_t N, int64_t K, int splits,
                            bsq_stream_t stream);

/*
 * bsq_gemm_gelu: as bsq_gemm with out = bf16_rn(GELU(v)), v = alpha * sum_k Ahat Bhat + bias
 * in fp32, GELU the erf form 0.5 v (1 + erf(v / sqrt 2)) (the "fc1 + GELU" epilogue of every
 * stack in the "lightly-train - DINOv3 + EoMT on RTX 5090" README, section 4.3), evaluated in
 * fp32 with erfc from Abramowitz & Stegun formula 7.1.26: |error| <= 4e-7 |v| + 2^-20 |GELU|.
 * Arguments, shapes and errors as bsq_gemm.
 */
int bsq_gemm_gelu(int fmt, const void* A, const void* A_scales, const void* B, const void* B_scales,
                  const void* bias_bf16, void* out_bf16, int64_t M, int64_t N, int64_t K, bsq_stream_t stream);

/*
 * bsq_gemm_gelu_quantize: the producer-fused fc1 of the README's MXFP8 stack (section 4.3: the
 * fc1 epilogue quantizes the GELU output straight into fc2's operand). y = GELU(v) as in
 * bsq_gemm_gelu, kept in fp32, then quantized along each output row with the MX rule of
 * bsq_quantize into out_fmt (BSQ_MXFP8 or BSQ_MXFP4):
 *   out_codes   bsq_codes_bytes(out_fmt, M, N) bytes, written;
 *   out_scales  bsq_scales_bytes(out_fmt, M, N) bytes (tiled layout, padding zero), written.
 * The pair is exactly an M x N operand as bsq_quantize(out_fmt, y, M, N) lays it out, ready
 * as fc2's A. Codes and scales are the MX quantization of the kernel's fp32 y, which differs
 * from the exact value by the fp32 accumulation and GELU rounding; a code differs from the
 * exact value's code only where that value lies within this error of a rounding boundary.
 * Shapes: as bsq_gemm, and N % 32 == 0. Errors: as bsq_gemm; BSQ_ERR_ARG for another out_fmt
 * or a NULL out_scales; BSQ_ERR_ALIGN for an unaligned out_scales.
 */
int bsq_gemm_gelu_quantize(int fmt, const void* A, const void* A_scales, const void* B, const void* B_scales,
                           const void* bias_bf16, int out_fmt, void* out_codes, void* out_scales, int64_t M,
                           int64_t N, int64_t K, bsq_stream_t stream);

/*
 * bsq_convt2x2: the head's transposed convolution with kernel 2 and stride 2 as a block-scaled
 * GEMM ("lightly-train - DINOv3 + EoMT on RTX 5090" README, section 4.3: the head's two
 * ScaleBlocks (ConvT k2 s2 -> GELU -> depthwise 3x3 -> LN2D) upscale the patch grid, and ConvT1 /
 * ConvT2 are two of the six quantized GEMM classes). Kernel = stride = 2: every output pixel has
 * exactly one input pixel, so
 *   out[b, 2h + dy, 2w + dx, co] = bf16(alpha * sum_ci Ahat[(b, h, w), ci] * Bhat[(2 dy + dx) C_out + co, ci]
 *                                       + bias[co])        (GELU of it when gelu != 0)
 * is one GEMM with N = 4 C_out whose epilogue stores each output column at its output pixel.
 *   A, A_scales  the NHWC input, batch * H * W rows (tokens in (b, h, w) order) x C_in, as written
 *                by bsq_quantize(fmt, ..., batch * H * W, C_in, ...)
 *   B, B_scales  the weight as a 4 C_out x C_in operand: row (2 dy + dx) C_out + co holds tap
 *                (dy, dx) of output channel co, i.e. W_torch[ci, co, dy, dx] of a PyTorch
 *                ConvTranspose2d weight [C_in, C_out, 2, 2]
 *   bias_bf16    C_out bf16 values or NULL
 *   out_bf16     batch x 2H x 2W x C_out bf16 (NHWC), written
 *   alpha        as bsq_gemm (NVFP4: g_A * g_B from the scale tails)
 * GELU is the erf form evaluated as in bsq_gemm_gelu.
 * Shapes: C_in as bsq_gemm's K (multiple of 128 MXFP8, 256 FP4); C_out % 32 == 0; W divides 32
 * or 32 divides W (so that 32 consecutive tokens are whole image rows or part of one); batch *
 * H * W below 2^31. Otherwise BSQ_ERR_SHAPE. Errors: as bsq_gemm.
 */
int bsq_convt2x2(int fmt, const void* A, const void* A_scales, const void* B, const void* B_scales,
                 const void* bias_bf16, void* out_bf16, int64_t batch, int64_t H, int64_t W, int64_t C_in,
                 int64_t C_out, int gelu, bsq_stream_t stream);

/*
 * The three groups of calls below are what stands between a block's linear layers in a training or
 * serving step; the method's pages name LayerNorm, LayerScale and the training stacks' gradients
 * but print no formulas for them, so the formulas are stated here in full. Matrices are bf16, or
 * fp32 with BSQ_FLAG_SRC_F32. Unlike the quantizers' and GEMMs' operands these calls take buffers
 * at any element alignment and of any number of columns; 16-byte aligned rows are the fast path. A block
 * norm on rows of whole 16-byte vectors needs its weights, biases and gate aligned too for that (2 times slower
 * forward, 3 to 5 times backward with one at an odd address); rows of other lengths do not, but all matrices must then
 * start at one offset inside 16 bytes.
 * Inputs may have a row stride (in elements; 0 repeats one row); outputs are contiguous.
 */

/* Norm kinds: z = (v - mean) / sqrt(mean((v - mean)^2) + eps), with mean = 0 for the RMS norm. */
#define BSQ_NORM_RMS 1
#define BSQ_NORM_LAYER 2
#define BSQ_FLAG_PARAMS_F32 0x800 /* weights, biases and gate hold fp32 values; default: bf16 */
#define BSQ_FLAG_POST_NORM 0x1000 /* a norm after the block */
#define BSQ_FLAG_IDS_I64 0x2000   /* expert ids are int64; default: int32 */

/*
 * bsq_block_norm: the norms before and after a block, with the block's gate and the residual scale.
 * Per row, with o = weight_offset (1 for weights stored about zero):
 *   n = z(h) * (post_weight + o) + post_bias       with BSQ_FLAG_POST_NORM, else n = h
 *   x_out = residual_scale * x + gate * n           the residual stream
 *   y = z(x_out) * (pre_weight + o) + pre_bias      the next block's input
 * all in fp32, each output rounded once (y from the unrounded x_out).
 *   kind, flags    BSQ_NORM_*; BSQ_FLAG_SRC_F32 | BSQ_FLAG_PARAMS_F32 | BSQ_FLAG_POST_NORM
 *   rows, cols     rows >= 0; cols >= 1, a row at most 131072 bytes, else BSQ_ERR_SHAPE
 *   gate_groups    rows of `gate`: rows / gate_groups consecutive rows share one (rows must divide
 *                  evenly, else BSQ_ERR_SHAPE). 1: one gate for all rows (LayerScale).
 *   h              the block's output; NULL: none (x_out = residual_scale * x), then without post norm and gate
 *   x              the residual stream
 *   weights, biases, gate    cols values each (gate: gate_groups x cols); NULL weight or gate: 1
 *                  (the offset is not added to a missing weight), NULL bias: 0
 *   x_out          may be NULL, may be x or h itself where that is contiguous
 *   y              may be NULL (no norm before the next block); may be h itself
 *   stats          NULL or rows x 4 fp32, 16-byte aligned: mean and 1/sqrt(..) of the post norm,
 *                  then of the pre norm (zeros for a norm that is not taken); for the backward pass
 */
typedef struct {
  int32_t kind, flags;
  int64_t rows, cols, gate_groups;
  float eps, residual_scale, weight_offset;
  const void *h, *x;
  int64_t h_stride, x_stride;
  const void *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
  void *x_out, *y;
  float* stats;
} bsq_block_norm_args;
int bsq_block_norm(const bsq_block_norm_args* args, bsq_stream_t stream);

/*
 * bsq_block_norm_backward: gradients of bsq_block_norm from those of x_out and y. Rows over 4096 columns (over 4089
 * bf16 or 4093 fp32 columns where rows are no whole number of 16-byte vectors) run on clusters whose CTAs wait for
 * each other's sums; a wait that gives up (2 s) records BSQ_ERR_TIMEOUT in the device status, and the call's
 * outputs are incomplete.
 *   dx_out, dy     NULL: zero. x_out is needed (and pre_weight read) with dy alone; h is needed for
 *                  dh of a post norm and for every gradient of post_weight, post_bias and gate.
 *   stats          as bsq_block_norm wrote it for these rows
 *   dx, dh         rows x cols, NULL: not wanted; dx may be dx_out or dy itself where contiguous
 *   dpost_weight, dpost_bias, dgate (gate_groups x cols), dpre_weight, dpre_bias
 *                  fp32 whatever the parameters are, NULL: not wanted. Column sums are taken in
 *                  fp32 in a fixed order: the same inputs give the same bits.
 *   workspace      bsq_block_norm_backward_workspace bytes, 16-byte aligned; may be NULL where no
 *                  parameter's gradient is wanted
 */
typedef struct {
  int32_t kind, flags;
  int64_t rows, cols, gate_groups;
  float residual_scale, weight_offset;
  const void *dx_out, *dy, *x_out, *h;
  int64_t dx_out_stride, dy_stride, x_out_stride, h_stride;
  const float* stats;
  const void *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
  void *dx, *dh;
  float *dpost_weight, *dpost_bias, *dgate, *dpre_weight, *dpre_bias;
  void* workspace;
  size_t workspace_bytes;
} bsq_block_norm_grad_args;
int bsq_block_norm_backward(const bsq_block_norm_grad_args* args, bsq_stream_t stream);
/* Bytes of bsq_block_norm_backward's workspace (flags: BSQ_FLAG_SRC_F32 matters); 0 for invalid arguments or
 * without a usable device. */
size_t bsq_block_norm_backward_workspace(int flags, int64_t rows, int64_t cols, int64_t gate_groups);

/*
 * bsq_expert_sort: where each token's choices of experts go when rows are sorted by expert.
 * Slot i = token * topk + j names expert ids[i]; an id outside [0, experts) is a dropped choice.
 *   counts[e]      slots of expert e                                              (experts int32)
 *   offsets[e]     first row of expert e; offsets[e + 1] = offsets[e] + counts[e] rounded up to a
 *                  multiple of `align`                                        (experts + 1 int32)
 *   position[i]    row of slot i, -1 for a dropped one. Slots of one expert keep their order.
 *   slot[r]        slot of row r, -1 for a row of none, for all r < capacity
 * With align = 128 each expert's rows cover whole scale tiles, so that its part of a quantized
 * rows matrix is an operand by itself. capacity must be at least bsq_expert_capacity(slots, experts, align) =
 * slots + min(experts, slots) * (align - 1) rounded up to `align`: enough whatever the ids are.
 *   flags          BSQ_FLAG_IDS_I64
 *   tokens, topk, experts, align      tokens >= 0; the others >= 1; experts at most
 *                  BSQ_MAX_EXPERTS, slots and capacity below 2^31, else BSQ_ERR_SHAPE
 *   workspace      bsq_expert_sort_workspace(slots, experts) bytes (0: NULL will do), 16-byte aligned
 */
#define BSQ_MAX_EXPERTS 2048
int bsq_expert_sort(int flags, const void* ids, int64_t tokens, int64_t topk, int64_t experts, int64_t align,
                    int64_t capacity, int32_t* counts, int32_t* offsets, int32_t* position, int32_t* slot,
                    void* workspace, size_t workspace_bytes, bsq_stream_t stream);
int64_t bsq_expert_capacity(int64_t slots, int64_t experts, int64_t align);
size_t bsq_expert_sort_workspace(int64_t slots, int64_t experts);

/*
 * bsq_expert_gather: rows[r] = x[slot[r] / topk] for r < capacity, zeros where slot[r] names none.
 * position and slot are one bsq_expert_sort's, here and below; a value out of range, or a row and a slot
 * that do not name each other, count as none.
 *   flags          BSQ_FLAG_SRC_F32
 *   x              tokens x cols; rows: capacity x cols. cols at most 2^30, else BSQ_ERR_SHAPE (here and below)
 */
int bsq_expert_gather(int flags, const void* x, int64_t x_stride, const int32_t* position, const int32_t* slot,
                      int64_t tokens, int64_t topk, int64_t cols, int64_t capacity, void* rows, bsq_stream_t stream);

/*
 * bsq_expert_combine: out[t] = sum over j of weights[t, j] * y[position[t, j]], added in fp32 in the
 * order of j and rounded once; dropped choices add nothing (what stands in their weights is not
 * read). weights (tokens x topk fp32) NULL: 1, which is the gradient of bsq_expert_gather.
 */
int bsq_expert_combine(int flags, const void* y, int64_t y_stride, const int32_t* position, const float* weights,
                       int64_t tokens, int64_t topk, int64_t cols, int64_t capacity, void* out, bsq_stream_t stream);

/*
 * bsq_expert_combine_backward: dy[r] = weights[slot[r]] * dout[slot[r] / topk], zeros where slot[r]
 * names none; dweights[t, j] = <dout[t], y[position[t, j]]> in fp32, 0 for a dropped choice.
 * dy: capacity x cols.
 */
int bsq_expert_combine_backward(int flags, const void* dout, int64_t dout_stride, const void* y, int64_t y_stride,
                                const int32_t* position, const int32_t* slot, const float* weights, int64_t tokens,
                                int64_t topk, int64_t cols, int64_t capacity, void* dy, float* dweights,
                                bsq_stream_t stream);

/*
 * The linear layers of dense and of expert blocks beyond the plain product. The pages fuse bias, GELU and residual
 * into their GEMMs' epilogues and print no formulas; these are stated here in full. Products are block-scaled as
 * bsq_gemm's, sums fp32, each output rounded once. Operands and outputs are 16-byte aligned.
 */

/* Activations: act(v) and its derivative. GELU: v Phi(v) with the normal distribution's Phi (erf form); GELU_TANH: its
 * form by tanh, v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2; SILU: v / (1 + exp(-v)); RELU: max(v, 0), derivative
 * 0 at 0. Evaluated in fp32, within 1e-6 |v| (GELU 2.8e-7 |v| at most where measured). Of GELU's small values at negative v
 * that is more than fp32's own step: 5e-5 of the value at -3, 2e-3 at -5; it shows in fp32 outputs alone. */
#define BSQ_ACT_NONE 0
#define BSQ_ACT_GELU 1
#define BSQ_ACT_GELU_TANH 2
#define BSQ_ACT_SILU 3
#define BSQ_ACT_RELU 4
#define BSQ_FLAG_OUT_F32 0x4000    /* out, and the residual, hold fp32; default: bf16 */
#define BSQ_FLAG_STACK_COLS 0x8000 /* the experts' weights stand side by side along the depth (see B) */

/*
 * One product of rows x depth with cols x depth operands; experts = 0: one weight for all rows, else row r of
 * expert e's segment takes the e-th weight. Segments are bsq_expert_sort's: expert e's rows are offsets[e] to
 * offsets[e] + counts[e], behind them up to offsets[e + 1], behind the last segment and ahead of the first stand rows of
 * none. Any alignment will do. Values out of range are taken as the nearest in range; segments must not overlap.
 *   A, A_scales    rows x depth operand (bsq_quantize). Rows of none may hold anything.
 *   B, B_scales    experts = 0: cols x depth operand. Else the experts' weights quantized as one matrix:
 *                  (experts cols) x depth, one below the other; with BSQ_FLAG_STACK_COLS cols x (experts depth), side
 *                  by side, as bsq_quantize_dual's column-wise operand of (experts depth) x cols lays them out. NVFP4:
 *                  one per-tensor scale for all experts.
 *   rows >= 0, depth % 128 == 0, cols % 8 == 0 (% 128 with experts), experts <= BSQ_MAX_EXPERTS, experts * cols and
 *   experts * depth below 2^31; else BSQ_ERR_SHAPE
 * bsq_gemm_act: v = alpha * A B^T + bias; out = residual + act(v); pre = v. Where bsq_gemm or bsq_gemm_gelu give the same
 *   (one weight, no residual, no `pre`, bf16), they are faster from 33 rows on, this call up to 32.
 *   bias           bf16, cols values (experts x cols), or NULL
 *   residual       rows x cols of out's type, row stride residual_stride (elements, >= cols, below 2^31, whole 16-byte
 *                  vectors), or NULL; may be `out` itself where contiguous. Not with experts.
 *   out            rows x cols; pre: rows x cols bf16, or NULL. With experts, rows of none are zeros in both.
 * bsq_gemm_act_backward: v = alpha * A B^T; out = v * act'(grad_pre); dbias = column sums of out before its rounding.
 *   The gradient towards a layer's input (A: its dY, B: its weights column-wise), on through the activation in front
 *   of it, and that layer's bias gradient.
 *   grad_pre       rows x cols bf16, what bsq_gemm_act kept as `pre`, row stride as the residual's; given exactly with an
 *                  activation. Values in rows of none are not used.
 *   dbias          fp32, cols (experts x cols), or NULL. Added in a fixed order: the same inputs give the same bits.
 *   workspace      bsq_gemm_act_backward_workspace bytes with dbias, else NULL will do
 * The fields of the other call are zero or NULL.
 */
typedef struct {
  int32_t fmt, flags, activation;
  int64_t rows, cols, depth, experts;
  const void *A, *A_scales, *B, *B_scales;
  const int32_t *counts, *offsets;
  const void* bias;
  const void* residual;
  int64_t residual_stride;
  const void* grad_pre;
  int64_t grad_pre_stride;
  void *out, *pre;
  float* dbias;
  void* workspace;
  size_t workspace_bytes;
} bsq_linear_args;
int bsq_gemm_act(const bsq_linear_args* args, bsq_stream_t stream);
int bsq_gemm_act_backward(const bsq_linear_args* args, bsq_stream_t stream);
/* 0 for invalid arguments. */
size_t bsq_gemm_act_backward_workspace(int64_t rows, int64_t cols, int64_t experts);

/*
 * bsq_expert_gemm_wgrad: the experts' weight gradients, out[e] = alpha * dY[rows of e]^T X[rows of e] (N x K each,
 * zeros for an expert without rows), from the column-wise operands that bsq_quantize_dual makes of the sorted rows:
 *   dY, X          N x rows and K x rows operands, blocks along the rows
 *   counts, offsets  as above, with offsets of multiples of 128 (bsq_expert_sort's align), the last one too: the scales'
 *                  tiles begin there, and a sum takes in whole steps of 32 rows (MXFP8) or 64. An expert whose segment
 *                  begins elsewhere, or ends inside its last step and ahead of the operands' last row, gets zeros, and the
 *                  device status BSQ_ERR_SHAPE. Rows of none inside a segment must be zeros, as bsq_expert_gather,
 *                  bsq_gemm_act with experts and bsq_expert_combine_backward leave them.
 *   fmt_flags      bsq_format | BSQ_FLAG_OUT_F32
 *   out            experts x N x K
 *   rows % 32 == 0, K % 8 == 0, experts * N below 2^31, else BSQ_ERR_SHAPE
 */
int bsq_expert_gemm_wgrad(int fmt_flags, const void* dY, const void* dY_scales, const void* X, const void* X_scales,
                          const int32_t* counts, const int32_t* offsets, int64_t rows, int64_t N, int64_t K,
                          int64_t experts, void* out, bsq_stream_t stream);

/* One gradient tensor: elems contiguous values, fp32 (f32 != 0) or bf16. dst may be src. elems may
 * be 0. Nothing else may overlap. */
typedef struct {
  const void* src;
  void* dst;
  int64_t elems;
  int32_t f32;
} bsq_grad_item;

/*
 * bsq_grad_norm: the norm of `count` tensors taken as one vector (dst is not used):
 *   norm_kind BSQ_GRAD_NORM_L2   sqrt(sum g^2), squares kept whole over all of fp32's range
 *   norm_kind BSQ_GRAD_NORM_MAX  max |g|
 * written to *norm (one fp32, device). NaN if any element is, else inf if any is or where the norm leaves
 * fp32's range.
 * bsq_clip_grad_norm: the same, and dst = src * max_norm / (norm + eps) for every tensor, or dst = src
 * where norm + eps <= max_norm. A NaN norm makes every dst NaN. No host synchronisation.
 *   count          >= 0; items is a host array, read before the call returns
 *   max_norm, eps  >= 0, finite max_norm or infinity (nothing is clipped); eps finite
 *   workspace      bsq_clip_grad_norm_workspace(count) bytes, 16-byte aligned
 */
#define BSQ_GRAD_NORM_L2 1
#define BSQ_GRAD_NORM_MAX 2
int bsq_grad_norm(int count, const bsq_grad_item* items, int norm_kind, float* norm, void* workspace,
                  size_t workspace_bytes, bsq_stream_t stream);
int bsq_clip_grad_norm(int count, const bsq_grad_item* items, int norm_kind, float max_norm, float eps, float* norm,
                       void* workspace, size_t workspace_bytes, bsq_stream_t stream);
/* 0 for a negative count or without a usable device. */
size_t bsq_clip_grad_norm_workspace(int count);

/*
 * bsq_get_device_status: synchronise `stream`, then read and clear the current device's
 * status word. Returns BSQ_OK, BSQ_ERR_TIMEOUT (a kernel's bounded wait on an mbarrier
 * gave up; that kernel returned early and its outputs are incomplete), BSQ_ERR_DEVICE_CHECK (the
 * checked build only: a kernel computed an index outside one of its buffers and skipped that
 * access) or BSQ_ERR_LAUNCH (a CUDA error while synchronising).
 * The checked build, libbsq_checked.so, is the same library compiled with BSQ_DEVICE_CHECKS=1:
 * every global load or store whose address a kernel computes itself (not the tensor copies, which
 * the tensor maps bound) is tested against its buffer's size first. It is the stand-in for a
 * memory checker. The block norms, expert rows and gradient norms have no such extra tests: the
 * indexes that they read from memory (slots, rows, ids) are tested in every build.
 */
int bsq_get_device_status(bsq_stream_t stream);

/*
 * bsq_selftest_timeout: enqueue a one-thread kernel that waits on an mbarrier nothing
 * arrives on, bounded by limit_ns nanoseconds of %globaltimer; it then records
 * BSQ_ERR_TIMEOUT in the device status word and returns. Exercises the failure path of
 * every bounded wait without faulting or hanging the GPU. limit_ns in [1e3, 1e10].
 */
int bsq_selftest_timeout(int64_t limit_ns, bsq_stream_t stream);

/*
 * bsq_selftest_device_check: enqueue a one-thread kernel whose single index check fails. The
 * checked build (libbsq_checked.so) records BSQ_ERR_DEVICE_CHECK in the device status word; the
 * normal build, whose checks compile to nothing, records nothing. Shows which build is loaded and
 * that its checks report through the status word without a trap.
 */
int bsq_selftest_device_check(bsq_stream_t stream);

/*
 * bsq_test_inject_stall: a test of the failure path of the kernels that wait on barriers, with no
 * GPU fault: arms a one-shot stall for the calling thread's next launch of one kernel class.
 *   kernel         BSQ_KERNEL_GEMM (every bsq_gemm* and bsq_convt2x2 launch), BSQ_KERNEL_DUAL
 *                  (bsq_quantize_dual) or BSQ_KERNEL_LAYERNORM (bsq_layernorm_quantize on fp32
 *                  sources or rows longer than 1024 elements: its shared-memory kernel; bf16 rows
 *                  of at most 1024 elements run a kernel that waits on no barrier, and the stall
 *                  stays armed past such a launch)
 *                  or BSQ_KERNEL_NORM (bsq_block_norm_backward on rows that a cluster holds, see there:
 *                  one CTA of each cluster sends no more sums after `after_stages` rows of a gate
 *                  row's; the stall stays armed past a launch on shorter rows)
 *                  or BSQ_KERNEL_LINEAR (bsq_gemm_act, its backward pass and bsq_expert_gemm_wgrad)
 *   after_stages   >= 0: the producers of that launch stop issuing loads -- and never announce the
 *                  missing bytes -- after this many pipeline stages per CTA, so a consumer waits for
 *                  a stage that never arrives; -1: disarm any stall armed on the calling thread
 *   wait_limit_ns  the limit of every bounded wait in that launch, in [1e3, 1e10] (the default
 *                  limit is 2 s)
 * The starved wait gives up after wait_limit_ns; the kernel then records BSQ_ERR_TIMEOUT in the
 * device status word, every role leaves its loop, the loads already issued are waited for (so
 * nothing is left in flight), tensor-core work drains, TMEM is released and the kernel returns.
 * The launch's outputs are incomplete; the next launch of the kernel runs normally. The method has
 * no counterpart: this exists for the tests. Errors: BSQ_ERR_ARG for an unknown kernel, after_stages
 * below -1 or a limit out of range.
 */
#define BSQ_KERNEL_GEMM 1
#define BSQ_KERNEL_DUAL 2
#define BSQ_KERNEL_LAYERNORM 3
#define BSQ_KERNEL_NORM 5
#define BSQ_KERNEL_LINEAR 6
int bsq_test_inject_stall(int kernel, int64_t after_stages, int64_t wait_limit_ns);

/*
 * bsq_test_norm_cut: how bsq_block_norm_backward cuts its rows on a GPU of num_sms SMs, for tests of sizes
 * that no test allocates; no device is used. `widest`: the longest row stride; `vectors`: whether alignment
 * lets 16-byte vectors be read. cut: whether they are, CTAs of a row, warps of a row in a CTA, rows at once in a CTA,
 * alignment classes, rows of a block (its classes' CTAs or clusters share them), blocks, and the bytes
 * that bsq_block_norm_backward_workspace asks for. BSQ_ERR_* as that call, BSQ_ERR_ARG without rows.
 */
int bsq_test_norm_cut(int flags, int64_t rows, int64_t cols, int64_t gate_groups, int64_t widest, int vectors,
                      int num_sms, int64_t cut[8]);

/* bsq_last_error: the calling thread's last non-zero return code (0 if none). */
int bsq_last_error(void);

/* bsq_strerror: a static string describing a status code. */
const char* bsq_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* BSQ_H */
