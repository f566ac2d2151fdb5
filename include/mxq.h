/*
 * mxq.h -- C ABI of the B200 (sm_100a) microscaling W4A4 linear-layer library (libmxq.so).
 *
 * The library implements the hot path of a block-scaled quantized linear layer,
 * Out = A * W^T with A [M, K] activations and W [N, K] weights (nn.Linear layout):
 *   - MXFP4: E2M1 elements in blocks of 32 along K with one E8M0 (power-of-two) scale per block,
 *     the EVEN rule for weights and the CEIL rule for per-token dynamic activation quantization
 *     ("Qwen3.5-27B-MXFP4-QAD-W4A4-LR1e-5-s1000", "How this checkpoint was produced", Training row;
 *      "Qwen3.5-9B-MXFP4-QAD-W4A4-LR1e-5-s3000", "Training mode" paragraph);
 *   - NVFP4: E2M1 elements, blocks of 16 with an E4M3 scale, and one fp32 per-tensor global scale
 *     ("Qwen3.5-27B-NVFP4-RTN-weight-only", first paragraph; "Qwen3.5-27B-NVFP4-GPTQ", Recipe row);
 *   - MXFP8: E4M3 elements, blocks of 32 with an E8M0 scale
 *     ("intel-ai/Qwen3.8-27B-MXFP4-AutoRound", section 1 and section 7, OCP MX).
 *
 * Scale rules (block amax over |x|, e clamped to [-127, 127], amax = 0 gives e = -127):
 *   EVEN  e = floor(log2 amax) - emax_elem           (emax_elem 2 for E2M1, 8 for E4M3)
 *   CEIL  e = least integer with amax <= elem_max * 2^e   (elem_max 6 for E2M1, 448 for E4M3)
 * MX elements are RNE(x / 2^e) on the element grid, saturating at +-elem_max.
 * NVFP4 (fp32 IEEE, g = global scale in the decode direction, x ~ q * s * g):
 *   s = RNE_E4M3_satfinite(fl(fl(amax/6) / g)) (0 for an all-zero block), d = fl(dec(s) * g),
 *   q_i = RNE_E2M1_sat(fl(x_i * fl(1/d))); when d == 0 every code is a zero that keeps x_i's sign.
 *   Where fl(1/d) overflows to +inf (d < 2^-128, only with an fp32-subnormal g), a nonzero x_i
 *   saturates to +-6 and a zero x_i stays a zero with its sign (0 * inf has no E2M1 code).
 *
 * Conventions for every call:
 *   - Pointers marked (device) are device memory of the current CUDA device; the caller owns and
 *     allocates every buffer.  The compute calls allocate nothing.
 *   - Calls are asynchronous and stream-ordered on `stream` (a cudaStream_t; NULL = legacy default).
 *   - Return MXQ_OK (0) or a negative MXQ_ERR_* code.  Argument errors are detected on the host
 *     before anything is launched; MXQ_ERR_CUDA reports a failed launch.
 *   - Device pointers must be 16-byte aligned.
 *   - Quantized FP4 data: [rows, K/2] bytes, element 2i in bits 0-3 and element 2i+1 in bits 4-7
 *     of byte i of the row.  MXFP8 data: [rows, K] bytes of E4M3 codes.
 *   - Row-major scales: [rows, K/bs] bytes.  Swizzled scales (what the GEMM consumes): tiles of
 *     128 rows x 4 scale columns, 512 bytes each, ordered [ceil(rows/128)][ceil((K/bs)/4)]; inside a
 *     tile, scale (r, c) sits at byte (r%32)*16 + ((r%128)/32)*4 + c%4.  Padding bytes are zero.
 */
#ifndef MXQ_H
#define MXQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mxq_stream_t; /* same type as cudaStream_t */

typedef enum { MXQ_MXFP4 = 0, MXQ_NVFP4 = 1, MXQ_MXFP8 = 2 } mxq_fmt;
typedef enum { MXQ_RULE_EVEN = 0, MXQ_RULE_CEIL = 1 } mxq_rule; /* ignored for NVFP4 */
typedef enum { MXQ_OUT_BF16 = 0, MXQ_OUT_FP32 = 1 } mxq_out;
typedef enum { MXQ_SF_ROWMAJOR = 0, MXQ_SF_SWIZZLED = 1 } mxq_sf_layout;

#define MXQ_OK 0
#define MXQ_ERR_NULL (-1)        /* a required pointer is NULL */
#define MXQ_ERR_SHAPE (-2)       /* M, N or K out of range, or K not a multiple of what fmt needs */
#define MXQ_ERR_ALIGN (-3)       /* a pointer is not 16-byte aligned */
#define MXQ_ERR_UNSUPPORTED (-4) /* unknown fmt / rule / out / layout */
#define MXQ_ERR_WORKSPACE (-5)   /* workspace smaller than mxq_linear_workspace_size() */
#define MXQ_ERR_CUDA (-6)        /* a CUDA launch or query failed */
#define MXQ_ERR_TIMEOUT (-7)     /* a kernel gave up on a bounded wait (see mxq_device_status) */
#define MXQ_ERR_DEVICE (-8)      /* the current device is not sm_100 */

/* Block size along K: 32 for MXFP4/MXFP8, 16 for NVFP4. */
int mxq_block_size(mxq_fmt fmt);

/* Bytes of quantized element data for a [rows, K] matrix (rows*K/2 for FP4, rows*K for MXFP8). */
int mxq_q_bytes(int64_t rows, int64_t K, mxq_fmt fmt, size_t* bytes);

/* Bytes of the scale tensor for a [rows, K] matrix in the given layout (swizzled is padded). */
int mxq_sf_bytes(int64_t rows, int64_t K, mxq_fmt fmt, mxq_sf_layout layout, size_t* bytes);

/*
 * Quantize x [M, K] bf16 (device, row-major, K contiguous) along K.
 *   fmt, rule     element format and MX scale rule (rule ignored for NVFP4).
 *   global_scale  (device) fp32[1], the NVFP4 decode-direction global scale g > 0; NULL otherwise.
 *   q_out         (device) mxq_q_bytes() bytes; sf_out (device) mxq_sf_bytes(layout) bytes.
 * Requires M >= 1 and K >= bs with K % bs == 0.  The activation path ("Qwen3.5-9B-MXFP4-QAD-W4A4-
 * LR1e-5-s3000", "Training mode") is fmt=MXFP4, rule=CEIL; the RTN weight export
 * ("Qwen3.5-27B-NVFP4-RTN-weight-only", Training row: round-to-nearest) is rule=EVEN.
 */
int mxq_quantize(const void* x_bf16, int64_t M, int64_t K, mxq_fmt fmt, mxq_rule rule,
                 const float* global_scale, void* q_out, void* sf_out, mxq_sf_layout layout,
                 mxq_stream_t stream);

/*
 * NVFP4 quantization with a running-max activation global scale, the observer fused into the
 * quantizer ("Qwen3.5-27B-NVFP4-GPTQ", Serving-KL table and caveat: the RTN export's running-max
 * input scales).  The block scales use g = fl(*amax_in / (6 * 448)), the running state from earlier
 * batches (device fp32[1], positive); in the same pass *amax_out receives max(*amax_in, max |x|),
 * the state for the next call.  amax_in and amax_out must be different buffers (swap them between
 * calls).  Other arguments as mxq_quantize with fmt = NVFP4.
 */
int mxq_quantize_running(const void* x_bf16, int64_t M, int64_t K, const float* amax_in, float* amax_out, void* q_out,
                         void* sf_out, mxq_sf_layout layout, mxq_stream_t stream);

/*
 * Fake quantization (quantize, then dequantize back to bf16): y = bf16(dq(Q(x))) with exactly the
 * codes and scales mxq_quantize produces, decoded in the format's precision (MX: elem * 2^e, exact;
 * NVFP4: fl32(elem * d), d = fl32(dec(s) * g)) and rounded once to bf16 (RNE).  This is the
 * fake-quantized forward of quantization-aware training, bit-identical to the serving quantizer
 * ("Qwen3.5-9B-MXFP4-QAD-W4A4-LR1e-5-s3000", "Training mode": W4A4 fake-quant, EVEN weights, CEIL
 * activations).  x, y: [M, K] bf16 (device); y may be x (in place).  Arguments as mxq_quantize.
 */
int mxq_fake_quantize(const void* x_bf16, int64_t M, int64_t K, mxq_fmt fmt, mxq_rule rule, const float* global_scale,
                      void* y_bf16, mxq_stream_t stream);

/*
 * Re-lay row-major scales [rows, kblocks] (device) into the swizzled tensor-core layout
 * (device, mxq_sf_bytes(SWIZZLED) bytes, padding zeroed).  Pure byte permutation.
 * The pages do not describe this layout: they only store the scales as U8 tensors
 * ("intel-ai/Qwen3.8-27B-MXFP4-AutoRound", section 1 "Model summary", Weight dtype row) that the
 * serving FP4 kernel consumes.  The layout is
 * the one the tcgen05 block-scaled MMA reads its scale factors in (128-row x 4-column tiles, see the
 * conventions above); this library's own reading, confirmed end to end by the GEMM parity tests.
 *   sf_rowmajor  (device) rows * kblocks bytes, read only.
 *   sf_swizzled  (device) mxq_sf_bytes(rows, K, fmt, MXQ_SF_SWIZZLED) bytes, written whole.
 * Errors: MXQ_ERR_NULL for a NULL pointer, MXQ_ERR_SHAPE unless 1 <= rows < 2^31 and
 * 1 <= kblocks < 2^24; nothing is launched then.
 */
int mxq_swizzle_scales(const uint8_t* sf_rowmajor, int64_t rows, int64_t kblocks, uint8_t* sf_swizzled,
                       mxq_stream_t stream);

/*
 * NVFP4 per-tensor global scale of x (n bf16 values, device): amax_out = max |x| and
 * g_out = fl(amax / (6 * 448)) in fp32 (decode direction), both device fp32[1].  This is the
 * running-max form of input_global_scale ("Qwen3.5-27B-NVFP4-GPTQ", Serving-KL table, RTN row).
 */
int mxq_global_scale(const void* x_bf16, int64_t n, float* g_out, float* amax_out, mxq_stream_t stream);

/*
 * Tensor amax of x (n bf16 values, device, 16-byte aligned): *amax_out = max |x| (device fp32[1],
 * exact: a bf16 value is an fp32 value).  This is the tensor-max helper a caller uses to derive a
 * dynamic NVFP4 global scale or to feed a running-max observer ("Qwen3.5-27B-NVFP4-GPTQ",
 * Serving-KL table: running-max versus static input scales); mxq_global_scale is the same
 * reduction followed by g = fl(amax / (6 * 448)).  Errors: MXQ_ERR_NULL, MXQ_ERR_SHAPE (n < 1),
 * MXQ_ERR_ALIGN; nothing is launched then.  Stream-ordered; allocates nothing.
 */
int mxq_amax(const void* x_bf16, int64_t n, float* amax_out, mxq_stream_t stream);

/*
 * Block-scaled GEMM on the tcgen05 tensor cores: out[M, N] = alpha * dq(A) dq(B)^T, fp32
 * accumulation, alpha = g_A[0] * g_B[0] for NVFP4 and 1 otherwise ("Qwen3.5-9B-MXFP4-QAD-W4A4-
 * LR1e-5-s3000", Serving: FP4 GEMM on quantized activations and weights).
 *   A_q [M, K] and B_q [N, K] quantized data (device); A_sf, B_sf SWIZZLED scales (device).
 *   g_A, g_B  (device) fp32[1] NVFP4 global scales; ignored (may be NULL) for MX formats.
 *   out       (device) [M, N] bf16 (RNE) or fp32, row-major.
 * Requires M, N >= 1; K >= 64 with K % 64 == 0 for FP4 and K % 32 == 0 for MXFP8.  There is no
 * lower bound on N beyond 1.
 */
int mxq_gemm(const void* A_q, const uint8_t* A_sf, const void* B_q, const uint8_t* B_sf, const float* g_A,
             const float* g_B, int64_t M, int64_t N, int64_t K, mxq_fmt fmt, mxq_out out_type, void* out,
             mxq_stream_t stream);

/*
 * Weight-only (W4A16) GEMM: out[M, N] = alpha * A dq(W)^T with bf16 activations A and MXFP4 or
 * NVFP4 weights, alpha = g_W[0] for NVFP4 and 1 for MXFP4.  This is the weight-only serving mode:
 * "Qwen3.5-27B-NVFP4-RTN-weight-only" (activations run bf16, no input_global_scale) and the
 * Marlin mode of "Qwen3.5-27B-MXFP4-QAD-W4A4-LR1e-5-s1000" ("Evaluation results": one weight
 * artifact serves W4A4 and W4A16).  W is dequantized to bf16 inside the kernel and multiplied on
 * the tcgen05 tensor cores (bf16 x bf16, fp32 accumulation).
 *   A        (device) [M, K] bf16, row-major.
 *   W_q      (device) [N, K/2] packed E2M1 codes; W_sf (device) their SWIZZLED scales, the same
 *            bytes mxq_gemm and mxq_linear read.
 *   g_W      (device) fp32[1] NVFP4 global scale of W; ignored (may be NULL) for MXFP4.
 *   out      (device) [M, N] bf16 (RNE) or fp32, row-major.
 * Requires fmt MXQ_MXFP4 or MXQ_NVFP4 (else MXQ_ERR_UNSUPPORTED), M, N >= 1, K >= 64 with
 * K % 64 == 0, 16-byte aligned pointers.  The dequantized weights are exact in bf16 for every
 * scale the EVEN-rule weight quantizer emits (E8M0 codes up to 252, E4M3 codes up to 0x7E); larger
 * E8M0 codes can overflow and are outside the contract.  Stream-ordered; allocates nothing.
 */
int mxq_gemm_w4a16(const void* A, const void* W_q, const uint8_t* W_sf, const float* g_W, int64_t M, int64_t N,
                   int64_t K, mxq_fmt fmt, mxq_out out_type, void* out, mxq_stream_t stream);

/* Workspace bytes mxq_linear needs for M tokens of width K (quantized A plus swizzled scales). */
size_t mxq_linear_workspace_size(int64_t M, int64_t K, mxq_fmt fmt);

/*
 * Kernels one mxq_linear call launches for this problem on the current device: 1 when the GEMM
 * quantizes its own activations (up to 32 tokens with several K splits; the workspace then stays
 * unused), 2 otherwise (quantizer, then GEMM).  The shape checks of mxq_linear come first (negative
 * MXQ_ERR_* codes), then the device check (MXQ_ERR_DEVICE / MXQ_ERR_CUDA without a usable sm_100
 * device).  Useful to plan CUDA-graph capture and to count launches.
 */
int mxq_linear_kernel_count(int64_t M, int64_t N, int64_t K, mxq_fmt fmt);

/*
 * Quantized linear layer, the W4A4 serving path: the activations are quantized dynamically per
 * token at run time and multiplied with the pre-quantized weights by an FP4 GEMM
 * ("Qwen3.5-9B-MXFP4-QAD-W4A4-LR1e-5-s3000", Serving, W4A4 bullet; the CEIL activation rule from its
 * "Training mode" paragraph).  out = dq(Q(x)) dq(W)^T * alpha with Q the quantizer of mxq_quantize.
 *   x_bf16     (device) [M, K] bf16 activations, row-major.
 *   W_q, W_sf  (device) the pre-quantized weights [N, K] (mxq_quantize output) with SWIZZLED scales.
 *   g_W, g_A   (device) fp32[1] NVFP4 global scales of W and of x (decode direction); ignored (may
 *              be NULL) for MX formats.
 *   act_rule   MX scale rule of the activations (ignored for NVFP4).
 *   workspace  (device) at least mxq_linear_workspace_size(M, K, fmt) bytes, caller-owned, 16-byte
 *              aligned: the quantized activations and their swizzled scales (up to 32 tokens the
 *              call may not touch it).
 *   out        (device) [M, N] bf16 (RNE) or fp32, row-major.
 * Requirements as mxq_gemm, plus M * K / 8 < 2^31.  The quantizer and the GEMM run back to back on
 * `stream` with programmatic dependent launch (one launch up to 32 tokens, see
 * mxq_linear_kernel_count); A is quantized once, not once per output tile.  Errors are checked in
 * this order before anything is launched: MXQ_ERR_UNSUPPORTED (fmt, act_rule, out_type),
 * MXQ_ERR_NULL, MXQ_ERR_SHAPE, MXQ_ERR_ALIGN, MXQ_ERR_WORKSPACE (ws_bytes too small),
 * MXQ_ERR_DEVICE; MXQ_ERR_CUDA reports a failed launch.
 */
int mxq_linear(const void* x_bf16, const void* W_q, const uint8_t* W_sf, const float* g_W, const float* g_A,
               int64_t M, int64_t N, int64_t K, mxq_fmt fmt, mxq_rule act_rule, mxq_out out_type,
               void* workspace, size_t ws_bytes, void* out, mxq_stream_t stream);

/*
 * mxq_linear without a caller-supplied workspace.  The pages have no counterpart: this call exists
 * for callers that are not allowed to allocate device memory -- e.g. plugins inside a host
 * framework that owns all device memory and passes only input and output buffers, or processes
 * under a fixed device-memory cap that must not grow (or synchronise the device through an
 * allocation) while serving.
 *
 * The activation workspace comes from a static array inside the library, MXQ_NOALLOC_SCRATCH_BYTES
 * bytes per GPU, held by every GPU that loads the library until the process exits.  Problems
 * whose mxq_linear_workspace_size(M, K, fmt) exceeds that size are rejected with
 * MXQ_ERR_WORKSPACE before anything is launched (8 MiB covers, e.g., up to 2048 tokens at K = 5120
 * for FP4).  Other arguments, requirements, error codes (in mxq_linear's order, the scratch limit
 * taking the place of the workspace size) and results are exactly those of mxq_linear: the same
 * kernels on the same bytes, so the output is bit-identical.  The caller still provides x, the
 * quantized weights and `out`.  The call allocates nothing.
 *
 * The first call on a device looks up the array's device address (once per device, with that
 * device current); make that first call before any stream capture.  All calls share the one array
 * and it keeps the last call's contents (each call rewrites everything it reads), so calls whose
 * executions overlap on the GPU -- e.g. on two streams without ordering between them -- race.
 */
#define MXQ_NOALLOC_SCRATCH_BYTES (8u << 20)
int mxq_linear_noalloc(const void* x_bf16, const void* W_q, const uint8_t* W_sf, const float* g_W,
                       const float* g_A, int64_t M, int64_t N, int64_t K, mxq_fmt fmt, mxq_rule act_rule,
                       mxq_out out_type, void* out, mxq_stream_t stream);

/*
 * ------------------------------------------------------------------------------------------------
 * A paged key/value cache held in 4 bits (MXFP4 or NVFP4), and attention over it.  The pages name no
 * such cache; its blocks, scales and rounding are those of mxq_quantize along the head dimension.
 *
 * One layer of the cache is num_pages pages of page_size tokens (a multiple of 16, at most 1024) for
 * kv_heads heads of head_dim D (64, 128 or 256) elements:
 *   uint8 [num_pages][kv_heads][page_size / 16][unit],  unit = mxq_kv_unit_bytes(D, fmt) bytes.
 * A unit holds 16 tokens of one head as  K codes (8 D bytes) | V codes (8 D) | K scales | V scales, with
 * nb = D / 32 (MXFP4) or D / 16 (NVFP4) scale bytes a token and side.  "Row bytes" are a token's D / 2
 * bytes of codes, byte i = elements 2i (low nibble) and 2i + 1.
 *   K codes   dealt to four quarters t of D / 8 bytes: NVFP4 quarter t is row bytes [t D/8, (t+1) D/8);
 *             MXFP4 quarter t is the row's 32-bit words t, t + 4, t + 8, ...  Quarters are cut in pieces
 *             of min(16, D / 8) bytes, stored [piece][token][t].
 *   V codes   row byte 8 j + g of a token is byte (token % 2) D/16 + j of the D/8-byte record of lane
 *             4 g + (token % 8) / 2 of the token's group of eight; records are cut in pieces of
 *             min(16, D / 8) bytes, stored [token / 8][piece][lane].
 *   K scales  [token][nb].     V scales  [token / 2][nb][token % 2].
 * A slot is page * page_size + offset, the place of one token; num_pages * page_size < 2^31.
 * Sequence b's token p lies in page block_table[b][p / page_size].
 * The kernels check what they read on the device before they use it as an index.  What they find out of
 * range is skipped and recorded in the device status word (mxq_device_status), first finding first:
 * 0x200 a slot, 0x201 a page of the block table, 0x202 q_start (outside q, falling, or more than max_q rows: the sequence
 * gets none), 0x203 a length the table cannot hold (the sequence has what the table holds).  A negative length is 0.
 */

/* Bytes of one unit (16 tokens of one head). */
int mxq_kv_unit_bytes(int head_dim, mxq_fmt fmt, size_t* bytes);

/*
 * Quantize tokens into the cache: k, v [tokens, kv_heads, D] bf16 (device; element strides k_token_stride
 * and so on, multiples of 8, the innermost dimension contiguous) go to slots[i] (device int32; negative:
 * the token is skipped).  Blocks along D, rule and global scales as in mxq_quantize; g_k, g_v (device)
 * fp32[1] for NVFP4.  Bytes of other tokens are left as they are.  Slots of one call are distinct; where
 * two are not, their place receives a mixture of both tokens.  tokens = 0 does nothing.
 */
int mxq_kv_append(const void* k, const void* v, int64_t tokens, int kv_heads, int head_dim, int64_t k_token_stride,
                  int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                  mxq_fmt fmt, mxq_rule rule, const float* g_k, const float* g_v, void* cache, int64_t num_pages,
                  int page_size, mxq_stream_t stream);

/*
 * Read tokens back as bf16: k_out, v_out [tokens, kv_heads, D] (device, contiguous) receive the values
 * that mxq_fake_quantize gives for what was appended at slots[i] (negative or out of range: zeros).
 */
int mxq_kv_read(const void* cache, int64_t num_pages, int page_size, int kv_heads, int head_dim, mxq_fmt fmt,
                const int32_t* slots, int64_t tokens, const float* g_k, const float* g_v, void* k_out, void* v_out,
                mxq_stream_t stream);

/* Workspace bytes of mxq_kv_attention on the current device (0 for arguments it refuses). */
size_t mxq_kv_attention_workspace_size(int64_t batch, int64_t max_q, int heads, int kv_heads, int head_dim);

/*
 * Attention over the cache: out[i] = sum_p w_ip V_p with w_i = softmax over the visible tokens p of
 * scale * q_i . K_p, for heads = kv_heads * group query heads (head h reads kv head h / group).
 *   q            (device) [rows, heads, D] bf16; element strides q_token_stride, q_head_stride, multiples
 *                of 8; the innermost dimension contiguous.
 *   block_table  (device) int32 [batch][table_stride], the first max_pages columns used; entries of pages
 *                without a token that some row of the sequence sees (behind its last, in front of all windows)
 *                are not read.  kv_lens (device) int32 [batch]: tokens in the cache, the query tokens' own
 *                included.
 *   q_start      (device) int32 [batch + 1]: sequence b's query rows are q_start[b] .. q_start[b + 1] - 1,
 *                at most max_q; NULL: max_q rows each, rows = batch * max_q.
 *   causal       query j of a sequence's n sees the tokens up to its own, kv_lens[b] - n + j; 0: all.
 *   window       > 0: only the last `window` of the tokens up to its own; 0: no limit.
 *   g_k, g_v     (device) fp32[1] NVFP4 global scales; ignored (may be NULL) for MXFP4.
 *   out          (device) [rows, heads, D] bf16 (RNE) or fp32.  lse (device) fp32 [rows, heads], the natural
 *                logarithm of the softmax's denominator, or NULL.  A row that sees no token gets zeros and
 *                -inf.  Rows of no sequence are left as they were.  Neither overlaps an input.
 *   workspace    (device) at least mxq_kv_attention_workspace_size(...) bytes; needs no preparation.
 * max_pages * page_size <= 2^30 - 1024.  Scores, softmax and sums are fp32.  Rounded to fewer bits are q, to 2^-32
 * of its row's largest element (MXFP4 with many rows: not at all), and probabilities, for the product with V, to
 * f16: 2^-11 of one, or 2^-28 of the row's largest where that is more; with few rows their product with V's scale
 * once more so; MXFP4 with many rows keeps 16 bits.  ("Many": more than 16 rows a sequence and kv head for NVFP4
 * with heads of 128, 48 else; never with heads of 256.)  MXFP4 keys and values below 2^-90 and blocks of scale byte
 * 0 may count as zero.  Scale bytes that are not numbers, which the quantizer never writes, have an effect on
 * rows that see the token alone.  Results do not depend on timing.  Two launches.  Calls that may run at the same
 * time need a workspace each.
 */
int mxq_kv_attention(const void* q, int64_t rows, int64_t q_token_stride, int64_t q_head_stride, const void* cache,
                     int64_t num_pages, int page_size, int heads, int kv_heads, int head_dim, mxq_fmt fmt,
                     const int32_t* block_table, int64_t table_stride, int64_t max_pages, const int32_t* kv_lens,
                     int64_t batch, const int32_t* q_start, int64_t max_q, float scale, int causal, int64_t window,
                     const float* g_k, const float* g_v, mxq_out out_type, void* out, float* lse, void* workspace,
                     size_t ws_bytes, mxq_stream_t stream);

/*
 * Page bookkeeping.  The state lies on the device: block_table int32 [table_rows][table_stride] (max_pages
 * columns used, -1 where a sequence has no page), kv_lens int32 [table_rows], refs int32 [num_pages] (how
 * many sequences hold a page; 0: free).  A call names n (at most MXQ_KV_MAX_SEQS) different rows
 * (at most MXQ_KV_MAX_TABLE) and does all of its work or none:
 *   info (device) int32[2]  info[0] = 0, or -1: a row outside the table, named twice or in an unfit state,
 *                           -2: a count or length that is negative or too long, -3: not enough free pages;
 *                           info[1] = the pages concerned (0 if refused).
 * Calls are stream-ordered and may be captured into a graph; n = 0 is such a call too: info becomes {0, 0}.
 */
#define MXQ_KV_MAX_SEQS 4096
#define MXQ_KV_MAX_TABLE 65536

/*
 * Room for add[i] more tokens in row seqs[i]: takes free pages, lowest index first in the order of the
 * call's rows, and adds to kv_lens.  A last page that is not full and held by several rows (refs > 1 in front
 * of the call) is copied first, in all layers, so that the others keep their tokens.  That holds for each of the
 * call's rows: where it names all holders of a page, all of them copy it and the page becomes free, so that until
 * then one page more is taken (and -3 answered where it is missing) than the rows need.  The cache is `layers`
 * layers of page_bytes = kv_heads * page_size / 16 * unit bytes a page, layer_stride bytes apart.
 *   slots  (device) int32 [slots_cap] or NULL: the slots of the new tokens, row after row, then -1 (all -1 if refused).
 *   workspace (device) mxq_kv_reserve_workspace_size(n) bytes (n = 0: may be NULL).   info[1] = pages taken.
 */
size_t mxq_kv_reserve_workspace_size(int64_t n);
int mxq_kv_reserve(const int32_t* seqs, const int32_t* add, int64_t n, int32_t* block_table, int64_t table_rows,
                   int64_t table_stride, int64_t max_pages, int32_t* kv_lens, int32_t* refs, int64_t num_pages,
                   int page_size, void* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes, int32_t* slots,
                   int64_t slots_cap, int32_t* info, void* workspace, size_t ws_bytes, mxq_stream_t stream);

/*
 * Row children[i], which must be empty, becomes a copy of row parents[i] that shares all of its pages.  A
 * row may be the parent of many, but not a parent and a child.  info[1] = page references added.
 */
int mxq_kv_fork(const int32_t* parents, const int32_t* children, int64_t n, int32_t* block_table, int64_t table_rows,
                int64_t table_stride, int64_t max_pages, int32_t* kv_lens, int32_t* refs, int64_t num_pages,
                int page_size, int32_t* info, mxq_stream_t stream);

/*
 * Cut row seqs[i] to new_lens[i] tokens (0: free it); pages that it no longer needs lose a reference and
 * their table entries become -1.  info[1] = page references dropped.
 */
int mxq_kv_truncate(const int32_t* seqs, const int32_t* new_lens, int64_t n, int32_t* block_table, int64_t table_rows,
                    int64_t table_stride, int64_t max_pages, int32_t* kv_lens, int32_t* refs, int64_t num_pages,
                    int page_size, int32_t* info, mxq_stream_t stream);

/*
 * Pack the pages in use into [0, live): the i-th page in use at or behind `live` moves, in all layers, into
 * the i-th free page in front of it; refs and the first ceil(kv_lens / page_size) entries of every table row
 * follow.  workspace (device) mxq_kv_compact_workspace_size(num_pages) bytes.   info[1] = live.
 */
size_t mxq_kv_compact_workspace_size(int64_t num_pages);
int mxq_kv_compact(int32_t* block_table, int64_t table_rows, int64_t table_stride, int64_t max_pages,
                   const int32_t* kv_lens, int32_t* refs, int64_t num_pages, int page_size, void* cache, int64_t layers,
                   int64_t layer_stride, int64_t page_bytes, int32_t* info, void* workspace, size_t ws_bytes,
                   mxq_stream_t stream);

/* Read the device status word that kernels set when a bounded wait gives up (0 = clean).
 * Synchronizes `stream`.  If reset != 0 the word is cleared afterwards. */
int mxq_device_status(int* status_out, int reset, mxq_stream_t stream);

/* Self-test of the bounded-wait path: launches one CTA that waits on a barrier nothing completes,
 * with a limit of timeout_ns; the kernel records MXQ_ERR_TIMEOUT in the status word and returns.
 * Returns MXQ_OK if the launch succeeded (read the outcome with mxq_device_status). */
int mxq_selftest_timeout(uint64_t timeout_ns, mxq_stream_t stream);

/* Human-readable name of an MXQ_* code. */
const char* mxq_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* MXQ_H */
