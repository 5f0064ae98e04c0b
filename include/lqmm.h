/*
 * lqmm.h -- C interface of liblqmm, block-quantized weight matrix multiply for
 * AMD Instinct MI355X (gfx950).
 *
 * The operations are the hot path of local LLM inference described in
 * "Resumo Tecnico: Llamas na Web" (summary of the LlamaWeb paper), section
 * "Design de Shader Consciente de Quantizacao": for the decode mat-vec the
 * llama.cpp weight blocks are dequantized directly in registers; for the
 * prefill matmul the blocks are loaded, dequantized into shared memory (LDS
 * here) and reused. The plain tiled fp32 matmul is the one printed in
 * "Compute Shaders con WebGPU para Inferencia ML", section "El Nucleo:
 * Multiplicacion de Matrices en WGSL".
 *
 * Conventions shared by every call
 * --------------------------------
 * - Tensor pointers are DEVICE pointers (hipMalloc'd or torch CUDA tensors),
 *   owned by the caller. The library never allocates, frees or synchronizes.
 * - Every matrix is dense, row-major and contiguous; fp16 values are raw
 *   IEEE binary16 bits (uint16_t).
 * - Every pointer must be 16-byte aligned (LQMM_ERR_ALIGN otherwise).
 * - `stream` is a hipStream_t passed as void* (NULL = the null stream). A call
 *   only validates its arguments and enqueues kernels on that stream; it
 *   returns before the GPU work finishes. Device-side faults surface at the
 *   caller's next synchronization.
 * - All argument checks run on the host before any HIP call, so invalid
 *   arguments are reported without touching the GPU and with nothing
 *   enqueued. Sizes are int64_t; sizes <= 0 are LQMM_ERR_SHAPE (an empty
 *   problem is not a call to make). Outputs must not overlap inputs.
 * - Calls are thread-safe and re-entrant: the only library state is set up
 *   once per device under std::call_once (the device's properties, and each
 *   kernel's LDS limit on its first launch there).
 * - NaN and Inf inputs propagate; no value is checked.
 *
 * Weight block layouts (llama.cpp / GGUF style). The pages name the formats
 * (legacy Q4_0/Q8_0 and the K-quants) and describe them as flat buffers of
 * packed integers with the dequantization chosen at compile time; the byte
 * layout below is the llama.cpp one:
 *   Q4_0: 32 weights in 18 bytes: [d: fp16][qs: 16 bytes]. Weight j (j < 16)
 *         is the low nibble of qs[j], weight j+16 its high nibble;
 *         w = d * (q - 8) with q in 0..15.
 *   Q8_0: 32 weights in 34 bytes: [d: fp16][q: 32 x int8]; w = d * q.
 *   Q4_K: 256 weights in 144 bytes: [d: fp16][dmin: fp16][scales: 12 bytes]
 *         [qs: 128 bytes]. Sub-block s (weights 32s..32s+31) has a 6-bit
 *         scale sc_s and a 6-bit min m_s packed in `scales`:
 *           s < 4 : sc_s = scales[s] & 63,  m_s = scales[s+4] & 63
 *           s >= 4: sc_s = (scales[s+4] & 15) | ((scales[s-4] >> 6) << 4)
 *                   m_s  = (scales[s+4] >> 4) | ((scales[s]   >> 6) << 4)
 *         Weight l of sub-block s has q = the low (even s) or high (odd s)
 *         nibble of qs[32*(s/2) + l]; w = d * sc_s * q - dmin * m_s.
 * A quantized weight matrix W has N rows (output features) of K weights
 * (input features); row n is stored as K/32 (Q4_0, Q8_0) or K/256 (Q4_K)
 * consecutive blocks, and rows follow each other with no padding. fp16
 * scales are used as stored, subnormals included.
 *
 * Precision
 * ---------
 * Accumulation is fp32 everywhere. The quantized GEMVs round each activation
 * x to fp16 (round to nearest even, no scaling) before the dot products:
 * |x| must stay below 65504 (larger values become infinite), and in the
 * fp16 normal range, 2^-14 <= |x| < 65504, x contributes a relative rounding
 * error of at most 2^-11 per element; smaller |x| are rounded to fp16
 * subnormals, an absolute error of at most 2^-25 per element. For one or two
 * activation rows per pass the dequantized weights are exact (the block
 * scales are applied in fp32). From three rows up the GEMVs run on the fp16
 * matrix cores and round each dequantized weight to fp16: Q4_0 once
 * (d*(q-8)); Q4_K rounds d*sc and dmin*m to fp16 once per sub-block and then
 * each weight once (one fused multiply-add).
 * The Q8_0 GEMM rounds each dequantized weight d*q to fp16 (one rounding)
 * and the output to fp16. The fp32 GEMM uses fp32 matrix-core products with
 * fp32 accumulation.
 */
#ifndef LQMM_H
#define LQMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LQMM_OK = 0,
  LQMM_ERR_NULL = 1,      /* a required pointer is NULL */
  LQMM_ERR_SHAPE = 2,     /* a size is <= 0, not a block multiple, or too large */
  LQMM_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned */
  LQMM_ERR_WORKSPACE = 4, /* the call needs a workspace (split-K partial sums) and got none or too small a one */
  LQMM_ERR_DEVICE = 5,    /* no usable HIP device, or it is not a gfx950 GPU */
  LQMM_ERR_LAUNCH = 6,    /* a kernel launch failed (hipGetLastError) */
  LQMM_ERR_TYPE = 7       /* an element type that the call does not take */
} lqmm_status;

/* Largest size accepted for any dimension (elements). */
#define LQMM_MAX_DIM ((int64_t)1 << 31)
/* lqmm_gemm_q8_0_f16 needs K < LQMM_GEMM_MAX_K (LQMM_ERR_SHAPE otherwise). */
#define LQMM_GEMM_MAX_K ((int64_t)1 << 22)

/*
 * Dense fp32 GEMM: C[M x N] = A[M x K] * B[K x N], all fp32 row-major.
 * The tiled matmul of "Compute Shaders con WebGPU para Inferencia ML",
 * "El Nucleo: Multiplicacion de Matrices en WGSL": any M, N, K >= 1, ragged
 * edges handled by zero padding, C overwritten (no alpha/beta).
 */
lqmm_status lqmm_sgemm(const float *A, const float *B, float *C,
                       int64_t M, int64_t N, int64_t K, void *stream);

/*
 * Q4_0 GEMV (decode): y[b][n] = sum_k W[n][k] * x[b][k] for b < batch.
 * W: N x (K/32) Q4_0 blocks (N*K/32*18 bytes); x: batch x K fp32;
 * y: batch x N fp32 (overwritten). K % 32 == 0; any batch >= 1 (the batch
 * rows share each weight load: up to 2 rows per pass on the vector ALUs, up
 * to 16 per pass on the matrix cores, which take over from 3 rows).
 * Dequantization happens in registers ("Llamas na Web", "Design de Shader
 * Consciente de Quantizacao", mat-vec case).
 * workspace/workspace_bytes: device memory for split-K plans, which split a
 * row's K range over several workgroups (on different CUs) and add their
 * partial sums in a fixed order (results do not depend on timing). At least
 * lqmm_gemv_workspace_bytes(N, K, batch) bytes, 16-byte aligned, owned by
 * the caller, zero-filled once before its first use: every completed call
 * leaves the bytes it used (arrival counters and partial sums) zero again. Calls that may run at the same
 * time (other streams, other threads) must not share a workspace. NULL (or
 * too few bytes) is valid: the planner then uses no split-K plan, except
 * when a tuning override forces one (LQMM_ERR_WORKSPACE).
 */
lqmm_status lqmm_gemv_q4_0(const void *W, const float *x, float *y,
                           int64_t N, int64_t K, int64_t batch,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * lqmm_gemv_q4_0 for callers that cannot allocate device memory or pass a
 * workspace: code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation. Same arguments (without the workspace) and same
 * results as lqmm_gemv_q4_0 given a workspace. Its split-K plans use a
 * static device array of LQMM_NOALLOC_SCRATCH_BYTES instead, one per GPU,
 * held until the process ends; the call itself allocates and frees nothing.
 * Before each split-K launch it zeroes the plan's arrival counters with a
 * kernel on `stream`. Every call on a GPU shares that GPU's array, so calls
 * that may overlap on one GPU (other streams, other threads) race: order
 * them. A split-K plan needing more scratch than the array holds (possible
 * only when a tuning override forces one) returns LQMM_ERR_WORKSPACE.
 */
#define LQMM_NOALLOC_SCRATCH_BYTES ((size_t)1 << 20)
lqmm_status lqmm_gemv_q4_0_noalloc(const void *W, const float *x, float *y,
                                   int64_t N, int64_t K, int64_t batch, void *stream);

/*
 * Q8_0 x fp16 GEMM (prefill): Y[m][n] = sum_k X[m][k] * W[n][k], i.e.
 * Y = X * W^T. W: N x (K/32) Q8_0 blocks; X: M x K fp16; Y: M x N fp16
 * (fp32 accumulation, rounded to nearest even at the end). K % 32 == 0 and
 * K < LQMM_GEMM_MAX_K.
 * The raw weight blocks of each output tile are loaded into LDS and each
 * weight is dequantized once per workgroup, in registers, into the fp16
 * matrix-core operand that every row of the M tile reuses ("Llamas na Web",
 * "Design de Shader Consciente de Quantizacao", matmul case: blocks loaded
 * into shared memory, dequantized and reused). When K % 64 == 32 a second
 * kernel writes dequantized fp16 tiles to LDS instead.
 */
lqmm_status lqmm_gemm_q8_0_f16(const void *W, const uint16_t *X, uint16_t *Y,
                               int64_t M, int64_t N, int64_t K, void *stream);

/*
 * Q4_K GEMV (decode): y[b][n] = sum_k W[n][k] * x[b][k].
 * W: N x (K/256) Q4_K super-blocks (N*K/256*144 bytes); x: batch x K fp32;
 * y: batch x N fp32. K % 256 == 0; any batch >= 1. Arguments as for
 * lqmm_gemv_q4_0.
 */
lqmm_status lqmm_gemv_q4_k(const void *W, const float *x, float *y,
                           int64_t N, int64_t K, int64_t batch,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * The other format x phase pairs and more block formats. "Llamas na Web",
 * "Design de Shader Consciente de Quantizacao" applies both kernel styles to
 * every quantization format (mat-vec: dequantize in registers; matmul:
 * dequantize into shared memory and reuse) and adds a format by adding its
 * dequantization routine.
 *
 * Decode GEMVs y[b][n] = sum_k W[n][k] * x[b][k]; arguments, layouts,
 * workspace and precision as for lqmm_gemv_q4_0 (x rounded to fp16, block
 * scales applied in fp32, fp32 accumulation; every activation row on the
 * vector ALUs, in passes of up to four rows). Split-K plans, for rows longer
 * than one wave's slice (2048 weights of Q8_0 or the int4 layout, 4096 when
 * N is at least four times the CU count; 8192 of Q6_K or Q2_K; 2048 of
 * q1_0, 4096 when N is at least four times the CU count), need the
 * workspace (LQMM_ERR_WORKSPACE without it).
 *   lqmm_gemv_q8_0: W is N x (K/32) Q8_0 blocks (34 bytes), K % 32 == 0.
 *   lqmm_gemv_q6_k: W is N x (K/256) Q6_K super-blocks (210 bytes), K % 256 ==
 *     0. Super-block: [ql 128][qh 64][scales 16 x int8][d fp16];
 *     w = d * scales[k/16] * (q - 32), q = 6 bits: weight k = 128h + 32j + l
 *     (h < 2, j < 4, l < 32) has low 4 bits from the low (j < 2) or high
 *     (j >= 2) nibble of ql[64h + 32(j%2) + l], high 2 bits from bits
 *     2j..2j+1 of qh[32h + l].
 *   lqmm_gemv_q2_k: W is N x (K/256) Q2_K super-blocks (84 bytes), K % 256 ==
 *     0. Super-block: [scales 16][qs 64][d fp16][dmin fp16]; scales[g] =
 *     sc | m << 4 for weights 16g..16g+15; w = d * sc * q - dmin * m, q =
 *     bits 2j..2j+1 of qs[32h + l] for weight k = 128h + 32j + l.
 *   lqmm_gemv_q1_0: the 1-bit format "Llamas na Web" names under
 *     "Extensibilidade" (q1_0; the page gives no bytes), read as the _0
 *     family at one bit per weight: W is N x (K/32) blocks of 6 bytes,
 *     [d fp16][4 bytes of code bits]; the bit c of weight j is bit j % 8 of
 *     code byte j / 8; w = d * (2c - 1). K % 32 == 0.
 *   lqmm_gemv_i4g32: the int4 layout of "Compute Shaders con WebGPU para
 *     Inferencia ML", "Yendo a Cuantizado: Matmul INT4" (GPTQ/AWQ style):
 *     Wq holds N*K/8 32-bit words, weight (n, k) being nibble (n*K + k) % 8
 *     (bits 4i..4i+3) of word (n*K + k) / 8, a two's-complement code s in
 *     -8..7; scales and zeros are fp32 arrays of N x K/32 (per row and group
 *     of 32 along K); w = (s - zero) * scale. K % 32 == 0. (The page writes
 *     result[row * N + col] with row = weight row; y here is batch x N like
 *     every GEMV of this library.)
 */
lqmm_status lqmm_gemv_q8_0(const void *W, const float *x, float *y,
                           int64_t N, int64_t K, int64_t batch,
                           void *workspace, size_t workspace_bytes, void *stream);
lqmm_status lqmm_gemv_q6_k(const void *W, const float *x, float *y,
                           int64_t N, int64_t K, int64_t batch,
                           void *workspace, size_t workspace_bytes, void *stream);
lqmm_status lqmm_gemv_q2_k(const void *W, const float *x, float *y,
                           int64_t N, int64_t K, int64_t batch,
                           void *workspace, size_t workspace_bytes, void *stream);
lqmm_status lqmm_gemv_q1_0(const void *W, const float *x, float *y,
                           int64_t N, int64_t K, int64_t batch,
                           void *workspace, size_t workspace_bytes, void *stream);
lqmm_status lqmm_gemv_i4g32(const uint32_t *Wq, const float *scales,
                            const float *zeros, const float *x, float *y,
                            int64_t N, int64_t K, int64_t batch,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * Prefill GEMMs Y = X * W^T over Q4_0 (K % 32 == 0) and Q4_K (K % 256 == 0)
 * weights: X is M x K fp16, Y is M x N fp16, fp32 accumulation, K <
 * LQMM_GEMM_MAX_K. Each step's blocks are dequantized to fp16 into LDS
 * tiles reused by the whole M tile: each weight rounded once to fp16 (Q4_0
 * d*(q-8); Q4_K d*sc*q - dmin*m formed in fp32). Output rounded to nearest
 * even.
 */
lqmm_status lqmm_gemm_q4_0_f16(const void *W, const uint16_t *X, uint16_t *Y,
                               int64_t M, int64_t N, int64_t K, void *stream);
lqmm_status lqmm_gemm_q4_k_f16(const void *W, const uint16_t *X, uint16_t *Y,
                               int64_t M, int64_t N, int64_t K, void *stream);

/*
 * ---- serving operators ------------------------------------------------------
 * What a decoder layer runs between its weight products: keys and values into
 * a paged cache, attention over that cache, and products with 8-bit float
 * weights. Element types are passed as lqmm_type values (LQMM_ERR_TYPE for any
 * other); row strides (ld*) are in elements and a multiple of 16 bytes
 * (LQMM_ERR_ALIGN), the elements of one row (all heads of one token) are
 * contiguous. Index arrays (positions, slots, page numbers, lengths, rope
 * tables) and lse need only their element's alignment, all other pointers 16
 * bytes.
 */
typedef enum { LQMM_F32 = 0, LQMM_F16 = 1, LQMM_BF16 = 2 } lqmm_type;

/*
 * The paged cache. Memory of num_pages pages of page_size tokens (a power of
 * two, 8 .. 1024), fp16 or bf16, for n_kv_heads heads of head_dim (64, 96, 128
 * or 256) elements:
 *   k_cache [num_pages][n_kv_heads][page_size][head_dim]
 *   v_cache [num_pages][n_kv_heads][page_size / 8][head_dim][8]
 * In v_cache the eight tokens of an aligned group of eight are adjacent for
 * each dimension (token o of a page is element o % 8 of group o / 8), which is
 * the order that the matrix cores take. A token's slot is
 * page * page_size + (its place in the page).
 */

/*
 * Angles of the position rotation: turns[i] = inv_freq[i] / (2 pi) as a 64-bit
 * fraction of a turn, for n frequencies. HOST pointers, host arithmetic; copy
 * the table to the device once. position * turns[i] mod 2^64 is then the angle
 * with its whole turns dropped, at any position. LQMM_ERR_SHAPE when a
 * frequency is not finite.
 */
lqmm_status lqmm_rope_turns(const double *inv_freq, int64_t n, uint64_t *turns);

/*
 * Rotate q and k by their positions, append k and v to the cache.
 * q: tokens x (n_q_heads * head_dim), row stride ldq; k, v: tokens x
 * (n_kv_heads * head_dim), row strides ldk, ldv; all of in_type (fp32, fp16 or
 * bf16; slices of one projection's output are such rows). q_out: tokens x
 * n_q_heads x head_dim of cache_type (fp16 or bf16). q may be NULL, with
 * n_q_heads 0: only k and v are appended. positions: one int32 per token.
 * slots: one int64 per token; a token whose slot is negative or past the cache
 * is not appended (its q is still rotated). Two tokens with the same slot
 * leave a mixture of them there. rope_turns: rotary_dim / 2 entries; rotary_dim is a
 * multiple of 16, at most head_dim, and 0 (with NULL positions and
 * rope_turns) rotates nothing. Pair i of a head is elements (i, i +
 * rotary_dim / 2), or (2i, 2i + 1) when `interleaved` is not 0; elements from
 * rotary_dim on are copied. Computed in fp32, each result rounded once.
 */
lqmm_status lqmm_kv_append(const void *q, const void *k, const void *v, int in_type,
                           int64_t ldq, int64_t ldk, int64_t ldv,
                           const int32_t *positions, const int64_t *slots,
                           const uint64_t *rope_turns, int64_t rotary_dim, int interleaved,
                           void *q_out, void *k_cache, void *v_cache, int cache_type,
                           int64_t tokens, int64_t n_q_heads, int64_t n_kv_heads,
                           int64_t head_dim, int64_t page_size, int64_t num_pages,
                           void *stream);

/*
 * Attention of a batch of sequences over the cache. Every sequence's keys are
 * the prefix_len tokens of the shared pages prefix_pages (read once for all
 * sequences; prefix_len 0, with NULL pages, is none), then its own: sequence
 * b's seq_lens[b] tokens in pages[b][0 .. max_pages). (A prefix whose last
 * page is not full is followed by a new page.) seq_lens counts the tokens of
 * the sequence's own pages, the new ones, whose keys are appended before this
 * call, among them. q: tokens x (n_q_heads * head_dim) of `type` (the cache's:
 * fp16 or bf16), row stride ldq; n_q_heads is a multiple of n_kv_heads and
 * query head h reads key head h / (n_q_heads / n_kv_heads). The tokens of
 * sequence b are rows q_start[b] .. q_start[b + 1] - 1 of q (int32, batch + 1
 * entries, on the device); NULL is one token per sequence (tokens == batch).
 * max_q is at least the largest count of them (1 with NULL q_start; a
 * sequence's rows past it are left out). New token i of n sees the prefix and
 * its sequence's keys 0 .. seq_lens[b] - n + i. out: tokens x n_q_heads x head_dim of `type`; lse
 * (NULL: not wanted): tokens x n_q_heads fp32, the logarithm of the sum of
 * exp(scale * q.k). A row that sees no key gets zeros and -infinity, and so does
 * a row that is left out or lies outside q_start[0] .. q_start[batch] - 1.
 *
 * Logits, maxima, sums and outputs are fp32; the weights are rounded to `type`
 * for the second product and the output is rounded once. Lengths and page
 * numbers are read on the device and bounded there: a length is cut to what
 * max_pages pages hold, a page number outside the cache reads page 0. Memory
 * past a sequence's length is never used, whatever it holds. A NaN or infinity
 * in a key or value reaches the rows that see its key, and no others; a row with
 * a logit that is NaN is NaN, in out and lse.
 * The keys are split by what max_pages pages hold, since lengths are not known
 * on the host: a table wider than the batch's longest sequence needs (as a
 * captured graph has to pass) is correct, and slower, because parts without
 * keys are planned, written and joined too.
 * workspace: lqmm_attn_prefix_workspace_bytes() bytes (partial results; need
 * not be zeroed; LQMM_ERR_WORKSPACE when smaller); calls that may overlap
 * must not share it. The result does not depend on timing.
 */
lqmm_status lqmm_attn_prefix(const void *q, int64_t ldq, const void *k_cache, const void *v_cache,
                             int type, const int32_t *prefix_pages, int64_t prefix_len,
                             const int32_t *pages, int64_t max_pages, const int32_t *seq_lens,
                             const int32_t *q_start, int64_t max_q, void *out, float *lse,
                             float scale, int64_t tokens, int64_t batch, int64_t n_q_heads,
                             int64_t n_kv_heads, int64_t head_dim, int64_t page_size,
                             int64_t num_pages, void *workspace, size_t workspace_bytes,
                             void *stream);
/* Bytes that call needs for these sizes on the current device (0: none, also
 * for sizes that the call refuses and when there is no device). */
size_t lqmm_attn_prefix_workspace_bytes(int64_t prefix_len, int64_t max_pages, int64_t max_q,
                                        int64_t tokens, int64_t batch, int64_t n_q_heads,
                                        int64_t n_kv_heads, int64_t head_dim, int64_t page_size);

/*
 * 8-bit float products with a scale for each block of 128. Codes are e4m3
 * (finite-only, largest value 448). Weights: W is N x K codes, wscale
 * ceil(N/128) x ceil(K/128) fp32 (one for each 128 x 128 block, the last ones
 * cut short by N and K). Activations: Xq is M x K codes, xscale ceil(K/128) x
 * M fp32: xscale[b * M + m] belongs to columns 128b .. 128b + 127 of row m.
 *   Y[m][n] = sum_k Xq[m][k] xscale[k/128][m] W[n][k] wscale[n/128][k/128]
 * with fp32 accumulation, rounded once to y_type (fp32, fp16 or bf16). Y is
 * M x N. K is a multiple of 16 and < LQMM_GEMM_MAX_K; any M and N.
 */
lqmm_status lqmm_gemm_f8b128(const uint8_t *W, const float *wscale, const uint8_t *Xq,
                             const float *xscale, void *Y, int y_type, int64_t M, int64_t N,
                             int64_t K, void *stream);

/*
 * Activations to that form: for each row and group of 128 columns
 *   scale = max(max |x| / 448, 2^-126),  code = x / scale to nearest even.
 * X: M x K of x_type (fp32, fp16, bf16), row stride ldx; Xq: M x K codes;
 * xscale: ceil(K/128) x M. K is a multiple of 16. A NaN gives a NaN code; an
 * infinity makes its whole group's products NaN.
 */
lqmm_status lqmm_quant_f8b128(const void *X, int x_type, int64_t ldx, uint8_t *Xq, float *xscale,
                              int64_t M, int64_t K, void *stream);

/*
 * ---- serving operators in fewer bits -----------------------------------------
 *
 * The 8-bit paged cache. Each token's vector of one head is head_dim e4m3 codes
 * (finite-only, largest value 448; 0x7F and 0xFF are NaN) and a power of two,
 * held as one byte, its exponent + 127:
 *   k_cache  [num_pages][n_kv_heads][page_size][head_dim]           codes
 *   v_cache  [num_pages][n_kv_heads][page_size / 8][head_dim][8]    codes
 *   k_scales, v_scales  [num_pages][n_kv_heads][page_size]          bytes
 * A vector x is held with the least exponent e for which max |x| <= 448 * 2^e,
 * at least -60 (smaller values lose digits) and at most 60, or 7 in a call whose
 * type is fp16 (larger values are held as the largest code); its codes are x *
 * 2^-e to nearest even. An infinity or NaN is held as NaN and does not count for
 * e. Reading, bytes 1 to 253 are scales; what 0, 254 and 255 stand for is left
 * open, for the rows that see such a key. Which type a cache was written for is
 * not kept with it: attention whose type is fp16 takes scales above 2^7 as 2^7.
 */

/*
 * lqmm_kv_append with a norm of each head of q and k before the rotation,
 *   y = x / sqrt(mean(x^2) + eps) * weight,
 * into a 16-bit cache (NULL scales; of `type`) or an 8-bit one (both scales).
 * q_norm, k_norm: head_dim fp32 weights each, the same for every head; NULL: no
 * norm. eps >= 0. q_out is of `type` (fp16 or bf16) with either cache.
 * Everything else is as for lqmm_kv_append. No other token's codes or scales
 * are touched.
 */
lqmm_status lqmm_kv_append_norm(const void *q, const void *k, const void *v, int in_type,
                                int64_t ldq, int64_t ldk, int64_t ldv, const int32_t *positions,
                                const int64_t *slots, const uint64_t *rope_turns,
                                int64_t rotary_dim, int interleaved, const float *q_norm,
                                const float *k_norm, float eps, void *q_out, void *k_cache,
                                void *v_cache, uint8_t *k_scales, uint8_t *v_scales, int type,
                                int64_t tokens, int64_t n_q_heads, int64_t n_kv_heads,
                                int64_t head_dim, int64_t page_size, int64_t num_pages,
                                void *stream);

/*
 * The 8-bit cache back to dense rows, for handing a conversation on: row
 * starts[b] + j of k_out and v_out (tokens x n_kv_heads x head_dim of `type`:
 * fp32, fp16 or bf16) is token j of sequence b's pages[b][0 .. max_pages), each
 * value rounded once (exact in fp32 and bf16; fp16 has steps of 2^-24 and values
 * past 65504 are infinite). starts: batch + 1 int32, not decreasing, on the
 * device. Rows before starts[0] and from starts[batch] on are zeros, and so are
 * tokens past the page table; a page number outside the cache reads page 0.
 */
lqmm_status lqmm_kv_read_f8(const uint8_t *k_cache, const uint8_t *v_cache, const uint8_t *k_scales,
                            const uint8_t *v_scales, const int32_t *pages, int64_t max_pages,
                            const int32_t *starts, void *k_out, void *v_out, int type,
                            int64_t tokens, int64_t batch, int64_t n_kv_heads, int64_t head_dim,
                            int64_t page_size, int64_t num_pages, void *stream);

/*
 * lqmm_attn_prefix over the 8-bit cache; `type` (fp16 or bf16) is that of q and
 * out. Keys and values enter the products exactly, but for fp16 values below
 * 2^-14, which may enter in steps of 2^-24, and those of scales above 2^7, which
 * enter as with 2^7 (below 65504). In bf16 a value times its weight is held down
 * to 2^-126, and the sums hold values below 2^114. The rest is as for
 * lqmm_attn_prefix, a NaN code being a NaN value.
 */
lqmm_status lqmm_attn_prefix_f8(const void *q, int64_t ldq, const uint8_t *k_cache,
                                const uint8_t *v_cache, const uint8_t *k_scales,
                                const uint8_t *v_scales, int type, const int32_t *prefix_pages,
                                int64_t prefix_len, const int32_t *pages, int64_t max_pages,
                                const int32_t *seq_lens, const int32_t *q_start, int64_t max_q,
                                void *out, float *lse, float scale, int64_t tokens, int64_t batch,
                                int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                                int64_t page_size, int64_t num_pages, void *workspace,
                                size_t workspace_bytes, void *stream);
/* Bytes that call needs for these sizes (as lqmm_attn_prefix_workspace_bytes). */
size_t lqmm_attn_prefix_f8_workspace_bytes(int64_t prefix_len, int64_t max_pages, int64_t max_q,
                                           int64_t tokens, int64_t batch, int64_t n_q_heads,
                                           int64_t n_kv_heads, int64_t head_dim, int64_t page_size);

/*
 * Microscaled 4-bit floats (OCP Microscaling Formats v1.0, MXFP4). A row of K
 * values (K % 32 == 0) is K / 2 bytes of e2m1 codes, two a byte, the first in
 * the low half, and K / 32 scale bytes, one for each block of 32. A code is a
 * sign (bit 3) and 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale byte s is 2^(s - 127), 255
 * NaN. Scale bytes need no alignment.
 *
 * lqmm_quant_mxfp4: X (M x K of x_type: fp32, fp16, bf16; row stride ldx) to
 * codes and scales: the scale is 2^(floor(log2 max |x|) - 2), at least 2^-127,
 * and the codes are x / scale to nearest even, saturated at 6. A block with an
 * infinity or NaN gets the scale NaN and codes 0.
 */
lqmm_status lqmm_quant_mxfp4(const void *X, int x_type, int64_t ldx, uint8_t *Xq, uint8_t *xscale,
                             int64_t M, int64_t K, void *stream);
/*
 * Y = X * W^T of two such matrices, W: N x K and X: M x K, with fp32 sums,
 * rounded once to y_type (fp32, fp16 or bf16). Y is M x N; any M and N, K a
 * multiple of 32 and < LQMM_GEMM_MAX_K. A block whose scale is NaN makes its
 * row's (or column's) outputs NaN.
 */
lqmm_status lqmm_gemm_mxfp4(const uint8_t *W, const uint8_t *wscale, const uint8_t *Xq,
                            const uint8_t *xscale, void *Y, int y_type, int64_t M, int64_t N,
                            int64_t K, void *stream);

/* Workspace the GEMV calls of these sizes can use, in bytes (0 = none):
 * enough for every GEMV entry point on any device. */
size_t lqmm_gemv_workspace_bytes(int64_t N, int64_t K, int64_t batch);

/* Static, human-readable name of a status code. Takes any int (a status
 * code read back from elsewhere may hold any value); values that are not an
 * lqmm_status give a static "unknown status" string. */
const char *lqmm_status_string(int s);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int lqmm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LQMM_H */
