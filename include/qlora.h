/*
 * qlora.h -- C ABI of the MI355X (gfx950) QLoRA linear-layer library.
 *
 * The layer: a frozen weight W (d_out x d_in) stored as blockwise NF4 with
 * double-quantized scales, plus a trainable rank-r adapter (A, B):
 *     forward   Y  = X W_hat^T + s (X A^T) B^T,          s = fl32(alpha / r)
 *     backward  dX = dY W_hat + s (dY B) A,  dA = s (dY B)^T X,  dB = s dY^T (X A^T)
 * where W_hat is the restored (dequantized, bf16) weight and no gradient is
 * ever formed for W.
 *
 * Sources (page titles and sections):
 *   "QLoRA技术从入门到精通" §2(3) NF4 grid; §3(1) offline quantization
 *       (blocks, absmax scale, normalize, nearest level, 4-bit index, 8-bit
 *       quantization of the scales); §3(2) forward (restore to 16 bit, two
 *       branches, alpha / r); §3(3) backward (frozen base, only A and B).
 *   "LoRA 与 QLoRA：把大模型微调拆成可负担的工程" §2 (h = W x + (alpha/r) B A x,
 *       shapes of A and B), §8 (bf16 compute, bias none).
 *   "【X 长文】LoRA 与 QLoRA：用一块 GPU 微调大模型", quantization section
 *       (64-value blocks, NF4 levels with an exact 0, about 4.13 bits per
 *       weight with 8-bit scales) and QLoRA section (gradient passes through
 *       the restored weight to A and B).
 *   "7、QLoRA 量化微调" §7.1 (16 ascending level indices; group storage).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All matrices are dense and row-major.  bf16 tensors cross the ABI as
 *   uint16_t bit patterns.  Shapes (T = tokens, K = d_in, N = d_out):
 *     W [N][K] fp32, X [T][K], Y [T][N], A [r][K], B [N][r], dY [T][N],
 *     dX [T][K] (bf16); U [T][r], dA [r][K], dB [N][r] (fp32).
 * - Stored weight format (written by qlora_quantize_nf4):
 *     packed [N][K/2] uint8: 4-bit level indices, element 2j of the flattened
 *            weight in the HIGH nibble of byte j, element 2j+1 in the low one;
 *     codes  [N*K/bs] uint8: 8-bit code of each block's absmax scale, a block
 *            being bs consecutive weights of the flattened weight (bs =
 *            desc.blocksize: 64, 128 or 256; blocks may span rows);
 *     consts [ceil(N*K/bs/256)] fp32: per group of 256 consecutive block
 *            scales, the group's largest scale c_g.
 *   Block b is restored with s'_b = fl32(fl32(code_b) * fl32(c_g / 255)) and
 *   each weight as bf16_rne(fl32(T[q] * s'_b)).  With dq_blocksize == 0 there
 *   are no codes: consts [N*K/bs] holds each block's fp32 absmax s_b, and
 *   s'_b = s_b.
 * - Device pointers: every tensor argument is device memory owned by the
 *   caller (the library never allocates, frees or retains device memory and
 *   keeps no state between calls).  Descriptors and output-size pointers are
 *   host memory.
 * - stream: a hipStream_t passed as void* (NULL = the null stream).  Every
 *   compute call only enqueues work on that stream and returns without
 *   synchronizing; outputs are valid once the stream has reached that point.
 * - Errors: functions return QLORA_OK (0) or a negative QLORA_ERR_* code.
 *   Arguments are validated on the host before anything is enqueued -- for
 *   the calls on several layers, every layer before the first launch -- so a
 *   call that fails validation has no side effect.  QLORA_ERR_HIP reports a
 *   failed launch (hipGetLastError after enqueueing); work enqueued before
 *   it by the same call may then have run.
 * - Size limit: the kernels address each dense operand with 32-bit byte
 *   offsets, so the packed weight (N*K/2 bytes), X (T*K*2), Y and dY (T*N*2),
 *   dX (T*K*2) and the [T][2r] rank-r pairs of the workspace must each be
 *   below 2^31 - 16 bytes; larger calls return QLORA_ERR_SHAPE (the workspace
 *   queries too).  Dimensions are below 2^31.
 * - W, packed, X, dY, A, B, Y, dX, U_out, U_in, dA and dB must be 16-byte
 *   aligned (QLORA_ERR_UNSUPPORTED otherwise); codes and consts need only
 *   their element alignment.  A forward
 *   call with at most 16 tokens takes the weight-streaming kernel when K is
 *   a multiple of the block size and either codes is 16-byte aligned and
 *   K/bs is at most about 2000 (8-bit codes), or consts is 16-byte aligned
 *   and K/bs is at most about 1000 (fp32 block scales, dq_blocksize 0); else
 *   the tiled kernel (same results within the accuracy stated below).
 * - Inputs must be finite; results for NaN/Inf inputs are unspecified.
 * - Hot-path preconditions: blocksize 64 (also 128 or 256), dq_blocksize 256 (also 0),
 *   d_in % 64 == 0, d_out % 64 == 0, 0 <= r <= 128, T >= 0 (T == 0 is a
 *   no-op).  r == 0 means the base branch only.
 */
#ifndef QLORA_NF4_H
#define QLORA_NF4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  QLORA_OK = 0,
  QLORA_ERR_NULL = -1,        /* a required pointer is NULL */
  QLORA_ERR_SHAPE = -2,       /* a size is out of range or not a multiple it must be */
  QLORA_ERR_UNSUPPORTED = -3, /* a format parameter the library does not implement */
  QLORA_ERR_WORKSPACE = -4,   /* workspace is NULL or smaller than the size query returned */
  QLORA_ERR_HIP = -5,         /* the HIP runtime reported an error while enqueueing */
  QLORA_ERR_SCRATCH_LIMIT = -6 /* the call needs more scratch than QLORA_STATIC_SCRATCH_BYTES */
};

/* Descriptor of the stored base weight. */
typedef struct qlora_nf4_desc {
  int64_t d_out;        /* N: rows of W */
  int64_t d_in;         /* K: columns of W */
  int32_t blocksize;    /* weights per absmax block: 64, 128 or 256 ("QLoRA技术从入门到精通"
                           §3(1): blocks of e.g. 64 or 256 values) */
  int32_t dq_blocksize; /* block scales per second-level group: 256, or 0 for no second level
                           (the fp32 block scales are kept: consts holds one per block, codes is
                           empty and may be NULL; "7、QLoRA 量化微调" §7.1, 4.5 bits per weight) */
  int32_t table;        /* level table: QLORA_TABLE_NF4 (0) or QLORA_TABLE_UNIFORM (1) */
} qlora_nf4_desc;

/*
 * Level tables.  QLORA_TABLE_NF4: the NF4 table (qlora_nf4_levels).
 * QLORA_TABLE_UNIFORM: 16 equally spaced levels -1 + 2i/15 on [-1, 1]
 * ("7、QLoRA 量化微调" §7.1, with its worked example: 0.27 in a group of
 * absmax 1.52 -> index 9 -> 0.304); it has no zero level.  Everything else
 * (blocks, scale codes, packing, kernels) is the same.  The table is not
 * stored with the quantized weight: every call on a weight must pass the desc
 * it was quantized with.  Any other value: QLORA_ERR_UNSUPPORTED.
 */
#define QLORA_TABLE_NF4 0
#define QLORA_TABLE_UNIFORM 1

/* Human-readable name of a status code.  Never NULL; static storage. */
const char* qlora_status_string(int status);

/*
 * The library's NF4 level table and decision thresholds (host copy).
 * levels[16]: ascending, levels[0] = -1, levels[7] = 0, levels[15] = +1; the
 *   medians of 7 equal-probability slices of the lower half of N(0,1) and of
 *   8 slices of the upper half, each half scaled by its largest magnitude
 *   ("QLoRA技术从入门到精通" §2(3); "【X 长文】..." NF4 paragraph).
 * thresholds[15]: thresholds[k] is the largest float32 that is not closer to
 *   levels[k+1] than to levels[k]; the index of a normalized value x is the
 *   number of thresholds it exceeds (nearest level, ties to the lower index).
 * Either pointer may be NULL.  Host only; never touches the GPU.
 */
int qlora_nf4_levels(float* levels, float* thresholds);

/*
 * The same for either level table (QLORA_TABLE_NF4 or QLORA_TABLE_UNIFORM);
 * the thresholds follow the same rule.  Errors: UNSUPPORTED for another table.
 */
int qlora_table_levels(int32_t table, float* levels, float* thresholds);

/*
 * Sizes in bytes of the three stored-weight buffers for descriptor d.
 * Host only.  Errors: NULL (d or any out pointer), SHAPE, UNSUPPORTED.
 */
int qlora_nf4_sizes(const qlora_nf4_desc* d, size_t* packed_bytes, size_t* codes_bytes,
                    size_t* consts_bytes);

/*
 * Offline quantization of W (fp32 [N][K], device) into packed / codes /
 * consts (device, sizes from qlora_nf4_sizes) -- "QLoRA技术从入门到精通" §3(1):
 * per block (desc.blocksize weights) absmax scale s_b, x = fl32(w / s_b) (IEEE division),
 * nearest NF4 level (ties to the lower index; an all-zero block gives index 7),
 * two indices per byte; then per group of 256 block scales c_g = max s_b and
 * code_b = rint_half_even(fl32(fl32(s_b / c_g) * 255)) (0 when c_g == 0).
 * Indices use the exact s_b.  Results are bit-exact and deterministic.
 * Errors: NULL, SHAPE, UNSUPPORTED, HIP.
 */
int qlora_quantize_nf4(const qlora_nf4_desc* d, const float* W, uint8_t* packed, uint8_t* codes,
                       float* consts, void* stream);

/*
 * The same quantization of a base weight held in a 16-bit format
 * ("QLoRA技术从入门到精通" §3(1): the FP16 base model is converted offline to
 * the 4-bit form).  w_format: QLORA_W_F32 (W is float*, the call above),
 * QLORA_W_BF16 or QLORA_W_F16 (W is [N][K] uint16 bit patterns).  Each value
 * is widened exactly to fp32 and then quantized as above, so the outputs are
 * bit-identical to qlora_quantize_nf4 on the widened weight.  W and packed
 * 16-byte aligned.  Errors: NULL, SHAPE, UNSUPPORTED (unknown w_format,
 * alignment), HIP.
 */
#define QLORA_W_F32 0
#define QLORA_W_BF16 1
#define QLORA_W_F16 2
int qlora_quantize_nf4_typed(const qlora_nf4_desc* d, const void* W, int32_t w_format, uint8_t* packed,
                             uint8_t* codes, float* consts, void* stream);

/*
 * Workspace (device bytes) qlora_linear_fwd needs for T tokens and rank r.
 * Host only.  Errors: NULL, SHAPE, UNSUPPORTED.
 */
int qlora_fwd_workspace_bytes(const qlora_nf4_desc* d, int64_t T, int32_t r, size_t* bytes);

/*
 * Forward of the layer -- "QLoRA技术从入门到精通" §3(2); "LoRA 与 QLoRA：..." §2:
 *   U = X A^T (fp32 [T][r]),  Y = bf16( X W_hat^T + s U B^T ),  s = fl32(alpha/r).
 * W_hat is restored tile by tile on chip and never written to memory.
 * X [T][K], A [r][K], B [N][r], Y [T][N] are bf16 bits (device).  U_out
 * (fp32 [T][r], device) receives U for the backward pass; may be NULL.
 * A and B may be NULL only when r == 0; X and Y only when T == 0.
 * workspace: device scratch of at
 * least qlora_fwd_workspace_bytes (may be NULL if that size is 0); its
 * contents on entry are ignored.  Y must not alias any input.
 * Accuracy: fp32 accumulation of bf16 products; deterministic (no atomics).
 * Errors: NULL, SHAPE, UNSUPPORTED, WORKSPACE, HIP.
 */
int qlora_linear_fwd(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                     const float* consts, int64_t T, const uint16_t* X, int32_t r, float alpha,
                     const uint16_t* A, const uint16_t* B, uint16_t* Y, float* U_out,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * The forward above for callers that cannot allocate device memory -- code
 * recorded into a HIP graph, serving loops, harnesses that forbid hipMalloc:
 * the same kernels and the same results, bit for bit, as qlora_linear_fwd,
 * with no workspace argument.  The scratch comes from a device array of
 * QLORA_STATIC_SCRATCH_BYTES inside the library, one per GPU, kept until the
 * process ends; the call itself allocates and frees nothing.  A call whose
 * scratch (qlora_fwd_workspace_bytes) exceeds it returns
 * QLORA_ERR_SCRATCH_LIMIT before anything is enqueued (at r = 64: above
 * 32768 tokens).  All calls on one GPU share that GPU's array: two calls
 * that may run at the same time on one GPU (other streams, other host
 * threads) race on it and must be ordered by the caller.  The array's
 * contents on entry are ignored.  The stream must belong to the current
 * device (the array's address is looked up for it).  Other arguments,
 * accuracy and errors as qlora_linear_fwd; also HIP when the array cannot be
 * located.
 */
#define QLORA_STATIC_SCRATCH_BYTES (16u << 20)
int qlora_linear_fwd_noalloc(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                             const float* consts, int64_t T, const uint16_t* X, int32_t r, float alpha,
                             const uint16_t* A, const uint16_t* B, uint16_t* Y, float* U_out, void* stream);

/*
 * Workspace (device bytes) qlora_linear_bwd needs for T tokens and rank r.
 * Host only.  Errors: NULL, SHAPE, UNSUPPORTED.
 */
int qlora_bwd_workspace_bytes(const qlora_nf4_desc* d, int64_t T, int32_t r, size_t* bytes);

/*
 * Backward of the layer -- "QLoRA技术从入门到精通" §3(3); "【X 长文】..." QLoRA
 * section (the gradient reaches A and B through the restored weight; the base
 * weight is frozen, so no dW exists):
 *   G  = dY B
 *   dX = bf16( dY W_hat + s G A )        (skipped when dX == NULL)
 *   dA = s G^T X        fp32 [r][K], overwritten (not accumulated)
 *   dB = s dY^T U       fp32 [N][r], overwritten (not accumulated)
 * U_in: fp32 [T][r] saved by the forward; NULL recomputes U = X A^T.
 * dA and dB are required when r > 0 and ignored when r == 0; X and dY may
 * be NULL only when T == 0 (then dA and dB are set to zero).
 * workspace: at least qlora_bwd_workspace_bytes.  Outputs must not alias inputs.
 * Deterministic (no atomics).  Errors: NULL, SHAPE, UNSUPPORTED, WORKSPACE, HIP.
 */
int qlora_linear_bwd(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                     const float* consts, int64_t T, const uint16_t* X, int32_t r, float alpha,
                     const uint16_t* A, const uint16_t* B, const float* U_in, const uint16_t* dY,
                     uint16_t* dX, float* dA, float* dB, void* workspace, size_t workspace_bytes,
                     void* stream);

/*
 * The backward above for gradient accumulation over micro-batches ("LoRA 与
 * QLoRA：..." §10: gradient accumulation simulates a larger effective batch):
 * identical, except that the adapter gradients are added to what dA and dB
 * hold on entry,
 *   dA += s G^T X,   dB += s dY^T U,
 * each element read, added once in fp32 and written (deterministic; the sum
 * over the micro-batch is formed first, then added).  T == 0 leaves dA and dB
 * unchanged.  dX is written as by qlora_linear_bwd.  Same errors.
 */
int qlora_linear_bwd_accumulate(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                                const float* consts, int64_t T, const uint16_t* X, int32_t r, float alpha,
                                const uint16_t* A, const uint16_t* B, const float* U_in, const uint16_t* dY,
                                uint16_t* dX, float* dA, float* dB, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Export of the restored weight -- "QLoRA技术从入门到精通" §3(2) (the 4-bit
 * weight restored to a 16-bit float, table value times the block's scale):
 *   W_hat[N][K] = bf16_rne(fl32(T[q] * s'))   (bf16 bits, device)
 * Bit-identical to the weight the fused products restore on chip.  packed,
 * codes, consts as produced by qlora_quantize_nf4; W_hat must be 16-byte
 * aligned and must not alias the inputs.
 * Errors: NULL, SHAPE, UNSUPPORTED, HIP.
 */
int qlora_dequantize_nf4(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                         const float* consts, uint16_t* W_hat, void* stream);

/*
 * The adapter merged into the restored weight -- "LoRA 与 QLoRA：把大模型微调拆成
 * 可负担的工程" §3 (W + (alpha/r) B A after training); "【X 长文】LoRA 与 QLoRA：
 * 用一块 GPU 微调大模型", QLoRA section (with a 4-bit base, the merge goes into
 * the restored 16-bit weight, not into the 4-bit one):
 *   W_merged[N][K] = bf16_rne( fl32( W_hat + fl32(s * (B A)) ) ),  s = fl32(alpha / r)
 * A [r][K] and B [N][r] are bf16 bits (device, 16-byte aligned); B A is
 * accumulated in fp32 (MFMA order).  r = 0 gives W_hat exactly.  1 <= r <= 128
 * otherwise.  The 4-bit arrays are not modified.
 * Errors: NULL, SHAPE, UNSUPPORTED, HIP.
 */
int qlora_merge_lora(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                     const float* consts, int32_t r, float alpha, const uint16_t* A, const uint16_t* B,
                     uint16_t* W_merged, void* stream);

/*
 * Forward of n (1..4) layers that share their input X -- the projections of
 * one layer input, e.g. the query, key and value projections or the gate and
 * up projections; "LoRA 与 QLoRA：..." §8 targets every linear module, so
 * these arrive together.  Each layer i is the forward of qlora_linear_fwd
 * with d[i], packed[i], codes[i], consts[i], A[i], B[i], Y[i] and U_out[i];
 * all share X, T, r and alpha.  The layers must have the same d_in,
 * blocksize and dq_blocksize (tables may differ).  With at most 16 tokens the
 * rows of every weight are streamed in ONE launch (one workgroup per group of
 * row tiles, whichever weight they belong to), so small projections do not
 * leave the GPU idle and X is read from HBM once.  With more tokens, when
 * n > 1, every d_out is a multiple of 256, all layers use one table and the
 * weights' 256 x 256 output tiles number 512 or more, each layer's U runs
 * first and then ONE product covers all the weights (their output columns
 * side by side, each tile writing into its own layer's Y); otherwise the
 * layers run one after another.  Either way each Y element is the same
 * fp32 sum, rounded once.  The pointer arrays are host memory holding device
 * pointers; U_out may be NULL, or hold NULL entries.  Workspace:
 * qlora_multi_fwd_workspace_bytes.  Errors: as qlora_linear_fwd, and SHAPE
 * (n outside 1..4, different d_in), UNSUPPORTED (different block format).
 */
int qlora_multi_fwd_workspace_bytes(int32_t n, const qlora_nf4_desc* d, int64_t T, int32_t r, size_t* bytes);
int qlora_linear_fwd_multi(int32_t n, const qlora_nf4_desc* d, const uint8_t* const* packed,
                           const uint8_t* const* codes, const float* const* consts, int64_t T, const uint16_t* X,
                           int32_t r, float alpha, const uint16_t* const* A, const uint16_t* const* B,
                           uint16_t* const* Y, float* const* U_out, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * Backward of n (1..4) layers that share their input X (as for
 * qlora_linear_fwd_multi): X's gradient is the sum of the layers' shares,
 *   dX = bf16( sum_i (dY_i W_hat_i + s G_i A_i) ).
 * When n > 1, T > 0, dX is given and all layers use one table, dX is ONE
 * product: its contraction runs over the rows of every weight in turn (each
 * against its layer's dY), then over every layer's rank-r term, all in one
 * fp32 sum per element, rounded once.  Otherwise it is formed layer after
 * layer: the first layer's product writes dX, and each later one rounds its
 * own share to bf16, adds it to what dX holds and rounds again.  dA[i] and
 * dB[i] are each layer's own, overwritten.  U_in may be NULL or hold NULL
 * entries (U recomputed).  dX may be NULL.  Each layer has its own slice of
 * the workspace (qlora_multi_bwd_workspace_bytes is the sum of the slices).
 * Errors: as qlora_linear_bwd, and SHAPE (n outside 1..4, different d_in),
 * UNSUPPORTED (different block format).
 */
int qlora_multi_bwd_workspace_bytes(int32_t n, const qlora_nf4_desc* d, int64_t T, int32_t r, size_t* bytes);
int qlora_linear_bwd_multi(int32_t n, const qlora_nf4_desc* d, const uint8_t* const* packed,
                           const uint8_t* const* codes, const float* const* consts, int64_t T, const uint16_t* X,
                           int32_t r, float alpha, const uint16_t* const* A, const uint16_t* const* B,
                           const float* const* U_in, const uint16_t* const* dY, uint16_t* dX, float* const* dA,
                           float* const* dB, void* workspace, size_t workspace_bytes, void* stream);

/*
 * LoRA dropout on the adapter's input ("LoRA 与 QLoRA：..." §4.3; its §8
 * configuration uses lora_dropout 0.05).  The base branch takes X unchanged;
 * the adapter takes X_d = bf16_rne(fl32(x * c)) where kept and 0 where
 * dropped, c = fl32(1 / fl32(1 - p)):
 *   forward   U = X_d A^T,  Y = bf16(X W_hat^T + s U B^T)
 *   backward  dX = bf16(bf16(dY W_hat) + keep * c * (s G A)),  dA = s G^T X_d,
 *             dB = s dY^T U          (G = dY B; U as saved by the forward)
 * keep: the mask, an input (the random draw is the caller's): device,
 * [T][K/8] bytes, bit j of byte i (least significant first) keeps element
 * 8i + j of the row.  p in [0, 1).  The adapter's share of dX is added to the
 * rounded base share, so dX is rounded twice (once more than without
 * dropout).  Workspace: qlora_dropout_workspace_bytes (backward = 0 or 1);
 * its first T*K*2 bytes (rounded up to 256) hold X_d.  accumulate != 0 adds
 * to dA and dB as qlora_linear_bwd_accumulate does.  Other arguments as in
 * qlora_linear_fwd / qlora_linear_bwd.  r == 0 or T == 0: the plain call.
 * Errors: as those calls, and NULL (keep when T > 0 and r > 0),
 * UNSUPPORTED (p outside [0, 1)).
 */
int qlora_dropout_workspace_bytes(const qlora_nf4_desc* d, int64_t T, int32_t r, int32_t backward, size_t* bytes);
int qlora_linear_fwd_dropout(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                             const float* consts, int64_t T, const uint16_t* X, int32_t r, float alpha,
                             const uint16_t* A, const uint16_t* B, const uint8_t* keep, float p, uint16_t* Y,
                             float* U_out, void* workspace, size_t workspace_bytes, void* stream);
int qlora_linear_bwd_dropout(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                             const float* consts, int64_t T, const uint16_t* X, int32_t r, float alpha,
                             const uint16_t* A, const uint16_t* B, const float* U_in, const uint16_t* dY,
                             const uint8_t* keep, float p, uint16_t* dX, float* dA, float* dB, int32_t accumulate,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * 8-bit forms
 * -----------
 * The 8-bit form of a matrix M [rows][cols] (cols a multiple of 64): one
 * e4m3 code per element (OCP: largest finite value 448, 0x7F and 0xFF NaN)
 * and one power-of-two scale 2^(e - 127), kept as the byte e, per block of
 * block_rows x 128 elements, block_rows being 1 (layer inputs, gradients) or
 * 128 (weights).  The last block of a row, and the last row of blocks, may be
 * short.
 *   codes  [rows][cols] uint8
 *   scales [ceil(rows / block_rows)][4 ceil(cols / 512)] uint8: the row's
 *          ceil(cols / 128) bytes e, then bytes 127 up to whole dwords
 * e is the smallest byte in 1 .. 254 with
 *   (largest finite |x| of the block) <= 448 * 2^(e - 127)
 * and code = e4m3(x * 2^(127 - e)), rounded to nearest even (exact scaling,
 * one rounding); an element that is not finite becomes a NaN code and takes
 * no part in the largest.  Rows keep their own scales, so a range of rows of
 * a form by rows is the form of those rows.
 *
 * One form serves twice.  It is the checkpoint of a layer's input for the
 * backward pass, at half the memory of bf16 ("LoRA 与 QLoRA：..." §7, §10:
 * activations are what grows with the context; checkpointing trades them for
 * compute): qlora_linear_bwd_checkpoint and qlora_fp8_linear_bwd take it
 * where qlora_linear_bwd takes X.  And it is the operand of the products of a
 * layer whose frozen weight is kept at 8 bits (block_rows 128).
 *
 * codes and M are 16-byte aligned, scales 4-byte aligned;
 * rows * ceil(cols / 512) < 2^27 and rows * cols <= 2^36 - 2^12 (SHAPE
 * otherwise).
 * Scales other than 1 .. 254 are not produced; results for them are
 * unspecified.
 */
int qlora_fp8_sizes(int64_t rows, int64_t cols, int32_t block_rows, size_t* codes_bytes, size_t* scales_bytes);

/*
 * M [rows][cols] (device; m_format QLORA_W_F32, QLORA_W_BF16 or QLORA_W_F16)
 * -> codes, scales (device, sizes from qlora_fp8_sizes).  rows == 0 does
 * nothing.  Bit-exact and deterministic.
 * Errors: NULL, SHAPE, UNSUPPORTED (block_rows, m_format, alignment), HIP.
 */
int qlora_quantize_fp8(int64_t rows, int64_t cols, int32_t block_rows, const void* M, int32_t m_format,
                       uint8_t* codes, uint8_t* scales, void* stream);

/*
 * codes, scales -> M_hat [rows][cols] bf16 = bf16_rne(code * 2^(e - 127)).
 * Exact for e >= 3 and |code| * 2^(e - 127) < 2^128.  With e = 1 or 2 values
 * below bf16's least step, 2^-133, are rounded to it; and finite elements of
 * 1.9375 * 2^127 and above have the code 256 * 2^120 = 2^128, which is restored
 * as an infinity (here and where U, dA and dB read the form).  For a layer
 * input that is recomputed from, and for export of an 8-bit weight.
 * Errors: NULL, SHAPE, UNSUPPORTED (block_rows, alignment), HIP.
 */
int qlora_dequantize_fp8(int64_t rows, int64_t cols, int32_t block_rows, const uint8_t* codes, const uint8_t* scales,
                         uint16_t* M_hat, void* stream);

/*
 * Forward of a layer whose frozen weight W [d_out][d_in] is kept in the 8-bit
 * form (block_rows 128) and whose input is in the 8-bit form by rows:
 *   U = X_hat A^T (fp32 [T][r]),  Y = bf16( X_hat W_hat^T + s U B^T )
 * X_hat, W_hat being the values the forms stand for.  A [r][d_in], B
 * [d_out][r], Y [T][d_out] bf16; U_out (fp32 [T][r]) may be NULL; r == 0 (A, B
 * NULL) is the base product alone.  Sums are fp32, except that the matrix
 * units add the products of eight consecutive codes aligned to the largest of
 * the eight, which drops what is below 2^-13 of it.  s U enters its product in
 * fp32 with at most 128 tokens, with more as two bf16 terms (16 bits).  What is
 * not finite in the input becomes NaN in its own token's Y and U.
 * Deterministic.  Size limits, alignment and errors as qlora_linear_fwd (the
 * weight's codes in place of the packed weight; the rank-r pairs are [T][2r],
 * [N][2r] and [K][2r], 2r rounded up to a multiple of 64; scales 4-byte
 * aligned); the workspace is 16-byte aligned.
 */
int qlora_fp8_fwd_workspace_bytes(int64_t d_out, int64_t d_in, int64_t T, int32_t r, size_t* bytes);
int qlora_fp8_linear_fwd(int64_t d_out, int64_t d_in, const uint8_t* W_codes, const uint8_t* W_scales, int64_t T,
                         const uint8_t* X_codes, const uint8_t* X_scales, int32_t r, float alpha, const uint16_t* A,
                         const uint16_t* B, uint16_t* Y, float* U_out, void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * Its backward (dY [T][d_out] bf16):
 *   G  = dY B
 *   dX = bf16( dY_hat W_hat + s G A )     dY_hat: the 8-bit form of dY by rows
 *   dA = s G^T X_hat   fp32 [r][d_in],  dB = s dY^T U   fp32 [d_out][r]
 * accumulate == 0 overwrites dA and dB, otherwise they are added to (one fp32
 * addition per element).  dX may be NULL (the first layer: adapter gradients
 * only).  U_in NULL recomputes U from X_hat.  X_codes and X_scales may be
 * NULL when r == 0.  dA and dB carry fp32 accuracy (G and U enter their
 * products with 24 bits); s G enters dX as s U does Y.  T == 0: dA and dB become
 * zero, or stay as they are when accumulating.  Other arguments, limits and
 * errors as above and as qlora_linear_bwd.
 */
int qlora_fp8_bwd_workspace_bytes(int64_t d_out, int64_t d_in, int64_t T, int32_t r, size_t* bytes);
int qlora_fp8_linear_bwd(int64_t d_out, int64_t d_in, const uint8_t* W_codes, const uint8_t* W_scales, int64_t T,
                         const uint8_t* X_codes, const uint8_t* X_scales, int32_t r, float alpha, const uint16_t* A,
                         const uint16_t* B, const float* U_in, const uint16_t* dY, uint16_t* dX, float* dA, float* dB,
                         int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The backward of an NF4 layer (qlora_linear_bwd) whose input was kept as its
 * 8-bit form by rows:
 *   dX = bf16( dY W_hat + s G A ),  dA = s G^T X_hat,  dB = s dY^T U
 * U_in: as saved by the forward; NULL recomputes X_hat A^T.  dX is formed as
 * by qlora_linear_bwd (it does not depend on X).  accumulate, T == 0, r == 0
 * and dX == NULL as for qlora_fp8_linear_bwd.  There is no form of this call
 * with LoRA dropout or over several layers.
 * Errors: as qlora_linear_bwd, and SHAPE (from the workspace query too) where
 * A (r*K*2 bytes) or B (r*N*2) is not below 2^31 - 16 bytes; the workspace is
 * 16-byte aligned.
 */
int qlora_checkpoint_workspace_bytes(const qlora_nf4_desc* d, int64_t T, int32_t r, size_t* bytes);
int qlora_linear_bwd_checkpoint(const qlora_nf4_desc* d, const uint8_t* packed, const uint8_t* codes,
                                const float* consts, int64_t T, const uint8_t* X_codes, const uint8_t* X_scales,
                                int32_t r, float alpha, const uint16_t* A, const uint16_t* B, const float* U_in,
                                const uint16_t* dY, uint16_t* dX, float* dA, float* dB, int32_t accumulate,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * The two ends of the layers
 * --------------------------
 * What forms a layer's input X and takes its dX back (qlora_norm_*), and what
 * turns the last layer's Y, the logits, into a training loss and its dY or
 * into an answer's scores (qlora_token_logprob*, qlora_distill_*): the calls
 * between the layers of a training step ("QLoRA技术从入门到精通" §3: forward,
 * loss, backward, update of A and B).
 *
 * Residual norm, per token over D channels (D a multiple of 64, at most
 * 16384; T < 2^22):
 *   m  = block * r_b,  r_b = 1 / sqrt(mean(block^2) + eps)
 *   h' = h + scale * gate * post_weight * m
 *   x  = (h' * r) * weight,  r = 1 / sqrt(mean(h'^2) + eps)
 * block: a layer's output, bf16 [T][D]; NULL leaves h as it is (h_out is then
 * not written and may be NULL).  post_weight [D] or NULL: without it there is
 * no norm behind the block, m = block.  gate [D] or NULL (1).  stream_format:
 * QLORA_W_F32 or QLORA_W_BF16, of h, h_out, dh_out and dh.  weight_format: the
 * same two, of weight, post_weight and gate.  Sums and statistics are fp32; x
 * is formed from h' before h' is rounded to the stream's type.  The squares
 * have to stay in fp32's range (block and h' between 1e-16 and 1e16 in size
 * always do, and zeros with an eps).
 * X: bf16 [T][D] or NULL.  codes, scales: x in the 8-bit form by rows (sizes
 * from qlora_fp8_sizes, from x in fp32), for qlora_fp8_linear_fwd; both NULL
 * or both given; X or they are required.  stats: fp32 [T][2], (r, r_b), for
 * the backward; r_b is 1 without a norm behind the block.
 * h_out may be h.  Otherwise outputs must not alias inputs.  Matrices and
 * vectors are 16-byte aligned, scales and stats 4-byte.
 * With eps 0 a row of zeros has r = inf and x NaN.
 * Deterministic.  Errors: NULL (post_weight or gate without a block, too),
 * SHAPE, UNSUPPORTED (formats, alignment, eps negative or not finite, scale
 * not finite), HIP.
 */
int qlora_norm_fwd(int64_t T, int64_t D, const void* h, int32_t stream_format, const uint16_t* block,
                   const void* weight, const void* post_weight, const void* gate, int32_t weight_format, float scale,
                   float eps, void* h_out, uint16_t* X, uint8_t* codes, uint8_t* scales, float* stats, void* stream);

/*
 * Its backward.  dX bf16 [T][D]: the gradient of x (a layer's dX); dh_out: that
 * of h' from everything behind it, in the stream's type, or NULL (none);
 * h_out: h' as written by the forward, or h where there was no block.  With
 * n = h' r and m = block r_b:
 *   dh     = dh_out + r (weight dX - n mean(weight dX n))  (the gradient of h)
 *   dp     = scale gate dh                                 (dh before rounding)
 *   dblock = dp, or r_b (post_weight dp - m mean(post_weight dp m))   bf16
 *   dweight = sum_t dX n, dgate = scale post_weight sum_t dh m,
 *   dpost_weight = scale gate sum_t dh m                   fp32 [D]
 * dweight NULL: no gradients of weights (frozen norms); otherwise
 * dpost_weight and dgate are given exactly where post_weight and gate are.
 * accumulate != 0 adds to them, each element once; T == 0 then leaves them,
 * else sets them to 0.  dh may be dh_out.  workspace (with dweight only): at
 * least qlora_norm_bwd_workspace_bytes, 16-byte aligned.  Deterministic (no
 * atomics).  Errors: as the forward, and WORKSPACE.
 */
int qlora_norm_bwd_workspace_bytes(int64_t T, int64_t D, size_t* bytes);
int qlora_norm_bwd(int64_t T, int64_t D, const uint16_t* dX, const void* h_out, int32_t stream_format,
                   const uint16_t* block, const void* weight, const void* post_weight, const void* gate,
                   int32_t weight_format, float scale, const float* stats, const void* dh_out, void* dh,
                   uint16_t* dblock, float* dweight, float* dpost_weight, float* dgate, int32_t accumulate,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Log probabilities under q = softmax(scale * z), z being the first `vocab`
 * elements of each row of logits: format QLORA_W_F32, QLORA_W_BF16 or
 * QLORA_W_F16, rows ld >= vocab elements apart (a head whose rows were filled
 * up to a multiple of 64), any alignment of whole elements.  scale in
 * (0, 2^100]: the reciprocal of a temperature.  T < 2^22 rows.
 *   stats   fp32 [T][2]: M = max z and log S, S = sum exp(scale (z - M)); the
 *           row's log-sum-exp is scale M + log S
 *   logprob fp32 [T][n]: log q of tokens [T][n], n <= 128; a token outside
 *           0 .. vocab - 1 (a label of -100) is none and has log probability 0
 *   entropy fp32 [T], or NULL: -sum q log q
 *   top_ids [T][top], top_logprob fp32 [T][top]: the `top` (<= 128, <= vocab)
 *           largest logits of the row, largest first, ties to the lower token
 * A logit of -inf has probability 0 (no term in the entropy).  A row of nothing
 * else, a mask that leaves nothing, has M = log S = -inf, log probabilities
 * -inf and entropy 0.  NaN or +inf makes its own row's log probabilities and
 * entropy NaN; among the alternatives NaN comes last.
 * Sums are fp32 and join in 64 bits.  Deterministic.
 * Errors: NULL, SHAPE, UNSUPPORTED (format, alignment, scale), HIP.
 */
int qlora_token_logprob(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale,
                        int32_t n, const int64_t* tokens, float* logprob, float* stats, float* entropy, int32_t top,
                        int64_t* top_ids, float* top_logprob, void* stream);

/*
 * The gradient of the logits from d_logprob fp32 [T][n] and, or NULL,
 * d_entropy fp32 [T] (which needs the forward's entropy); stats as written by
 * the forward:
 *   dz_j = scale ( sum over tokens that name j of d - q_j sum of all d
 *                  - d_entropy q_j (log q_j + entropy) )
 * Tokens that are none take no part.  dlogits has the logits' format, rows of
 * out_cols >= vocab elements out_ld apart; columns from vocab on become 0 (so
 * that it is the dY of a head with more rows than tokens).  dlogits may be the
 * logits themselves, with the same row stride; otherwise the two must not
 * overlap.  Rows that start as far from a 16-byte boundary as the logits' do
 * take half the time of others.  A row whose weights are all 0, and one of -inf alone, has gradient
 * 0 whatever its logits hold.  The top alternatives carry no gradient.
 * T * (out_cols / 4096 + 2) < 2^24 is always enough (SHAPE beyond the launch).
 */
int qlora_token_logprob_bwd(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale,
                            int32_t n, const int64_t* tokens, const float* stats, const float* entropy,
                            const float* d_logprob, const float* d_entropy, void* dlogits, int64_t out_cols,
                            int64_t out_ld, void* stream);

/*
 * Distillation from a teacher's k (1 .. 128) top tokens of each row: ids
 * [T][k], values fp32 [T][k] (a teacher's top_ids and top_logprob, from
 * qlora_token_logprob at this loss's temperature).  q is the student's, as
 * above.
 *   rest == 0: p = softmax(values) over the k tokens (values may be logits)
 *     loss = sum_i p_i (log p_i - log q_i)
 *   rest == 1: p = exp(values), and what is left, left = max(0, 1 - sum p), is
 *     a bucket against the student's probability q_r outside the k tokens:
 *     loss = sum_i p_i (log p_i - log q_i) + left (log left - log q_r)
 * loss fp32 [T].  An id outside 0 .. vocab - 1 is no entry (a shorter list); a
 * row without entries has loss 0 and no gradient.  A token named twice has both
 * entries' p.  Values are finite or -inf (p = 0, no term).  p > 0 where q = 0
 * gives +inf; where q_r = 0 the bucket is left out.
 * stats fp32 [T][4]: M, log S, the whole of p that the gradient sees, and
 * left / q_r (at most 1e30; 0 without a bucket).  The loss is formed in 64 bits
 * from sums in fp32.  Deterministic.
 * Gradient (d_loss fp32 [T]; multiply it by the square of the temperature
 * where that is wanted):
 *   dz_j = scale d_loss ( whole q_j - sum of the p that name j )  listed tokens
 *        = scale d_loss ( whole - left / q_r ) q_j                the others
 * dlogits and its columns, strides and limits as qlora_token_logprob_bwd.
 * Rows, formats, alignment and errors as above (values, loss, stats and d_loss
 * 4-byte, ids 8-byte aligned).
 */
int qlora_distill_fwd(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale, int32_t k,
                      const int64_t* ids, const float* values, int32_t rest, float* loss, float* stats, void* stream);
int qlora_distill_bwd(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale, int32_t k,
                      const int64_t* ids, const float* values, int32_t rest, const float* stats, const float* d_loss,
                      void* dlogits, int64_t out_cols, int64_t out_ld, void* stream);

/*
 * AdamW update of the adapter parameters ("QLoRA技术从入门到精通" §3(3):
 * after the backward pass the optimizer updates only A and B, never the
 * quantized base weight).  The arithmetic is the published AdamW method
 * (Loshchilov and Hutter, decoupled weight decay), per element in fp32 with
 * the fp32 hyperparameters as given; the factors below that depend on them
 * (1 - beta, 1 - lr * weight_decay, the bias corrections) are formed in double
 * on the host and rounded to fp32 once:
 *   g = grad * grad_scale;  p *= 1 - lr * weight_decay
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p -= (lr / (1 - beta1^step)) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *   param_bf16 = bf16_rne(p)        (skipped when param_bf16 == NULL)
 * param, grad, exp_avg (m), exp_avg_sq (v): fp32 [n], device, 16-byte
 * aligned, updated in place (grad is read only); param_bf16: uint16 [n]
 * bf16 bits, 8-byte aligned.  Lay out every adapter of a model in one arena
 * to update them all in one call; with gradient accumulation, grad_scale =
 * 1 / (number of micro-batches) averages them.  The paged placement of the
 * optimizer state is not part of this call.  No buffer may alias another.
 * n == 0 does nothing (the buffers may then be NULL).
 * Errors: NULL (h; param, grad, exp_avg or exp_avg_sq when n > 0), SHAPE (n < 0),
 * UNSUPPORTED (step < 1, beta outside [0, 1), eps < 0, non-finite
 * hyperparameters, alignment), HIP.
 */
typedef struct qlora_adamw_hparams {
  float lr;
  float beta1;
  float beta2;
  float eps;
  float weight_decay;
  float grad_scale;
  int64_t step;  /* 1 for the first update */
} qlora_adamw_hparams;

int qlora_adamw_step(const qlora_adamw_hparams* h, int64_t n, float* param, const float* grad, float* exp_avg,
                     float* exp_avg_sq, uint16_t* param_bf16, void* stream);

/*
 * Per-kernel timing (measurement support; not an operation of the layer).
 * qlora_trace_enable(1) makes every subsequent kernel launch of the library
 * record a hipEvent before and after it on the launch stream (event objects
 * are created on first use and reused; no device memory is allocated);
 * qlora_trace_enable(0) (the default) records nothing.
 * qlora_trace_read waits for the recorded events, adds their elapsed times to
 * per-kernel totals and writes up to max_stats entries {name, launches,
 * total_ms} (name: static string) for the kernels launched so far; *count
 * receives the number of kernels with launches.  reset != 0 clears the
 * totals afterwards.  Errors: NULL (count, or stats with max_stats > 0), HIP.
 * Not thread-safe with respect to concurrent compute calls on other threads.
 */
/*
 * qlora_trace_select: like qlora_trace_enable, but only the kernels whose bit
 * is set in kernel_mask are bracketed (bit k = the kernel named by
 * qlora_trace_kernel_name(k)), so a caller can time the big kernels without
 * adding events between all the small ones.  qlora_trace_kernel_name returns
 * a static name, or NULL for k outside the library's kernel list.
 */
int qlora_trace_select(uint32_t kernel_mask);
const char* qlora_trace_kernel_name(int kernel);

typedef struct qlora_kernel_stat {
  const char* name;
  int64_t launches;
  double total_ms;
} qlora_kernel_stat;

int qlora_trace_enable(int enable);
int qlora_trace_read(qlora_kernel_stat* stats, int max_stats, int* count, int reset);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_NF4_H */
