/*
 * qk.h - C ABI of libqk: ggml block-quantized dequantize, GEMV and GEMM on
 * AMD gfx950 (MI355X), and what a decode step has between them: RMS norm,
 * paged key-value cache and its attention, routing to experts.
 *
 * Block formats (32 weights per block, little-endian binary16 fields, blocks
 * packed back to back, a matrix stored row after row with k/32 blocks per row
 * and no padding):
 *   QK_Q4_0  d[2] qs[16]       18 bytes  w = d*q + (-8*d),  q = nibble 0..15
 *   QK_Q4_1  d[2] m[2] qs[16]  20 bytes  w = d*q + m
 *   QK_Q8_0  d[2] qs[32]       34 bytes  w = d*q,           q = int8
 *   QK_Q5_0  d[2] qh[4] qs[16] 22 bytes  w = (q - 16) * d,  q = 0..31
 *   QK_Q5_1  d[2] m[2] qh[4] qs[16]  24 bytes  w = d*q + m, q = 0..31
 * For Q4_x, quant byte j holds element j in its low nibble and element j+16 in
 * its high nibble.  Source: "llama_cpp 0.12.1 -> 0.12.2" diff of ggml-cuda.cu
 * (diffend, page 4), hunks adding dequantize_block_q4_0, dequantize_block_q4_1
 * and dequantize_block_q8_0_f16; the row launchers dequantize_row_q4_*_cuda
 * give the 32-weight block (nb32 = k/32).
 * Q5_x: the same diff names these formats only in ggml_get_to_fp16_cuda /
 * ggml_get_to_fp32_cuda (dequantize_block_cuda with dequantize_q5_0 / _q5_1);
 * their layout is not printed there and follows ggml's block format: the low
 * four bits of each code as in Q4_x, bit 4 of code t in bit t of qh (a
 * little-endian 32-bit word).  Q5_0's (q - 16) * d makes q = 16 with d < 0
 * a -0.0 (Q4_0's form gives +0.0).
 *
 * Matrix layout follows ggml (ne0 is the contiguous dimension):
 *   W  m rows of k weights (row-major blocks as above);
 *   X  n activation columns of length k, column j starting at element j*ldx;
 *   Y  n output columns of length m, column j starting at element j*ldy.
 *
 * Conventions shared by every call:
 *   - Pointers are device pointers (or host-registered/managed memory the GPU
 *     can read) owned by the caller; they are borrowed until the enqueued work
 *     completes.  The library allocates, frees and synchronizes nothing and
 *     keeps no state, so calls are re-entrant.
 *   - `stream` is a hipStream_t passed as void*; NULL is the null stream.  Work
 *     is enqueued on it and the call returns without waiting.  The current
 *     device is the one that the stream and the pointers belong to.
 *   - The return value is QK_OK or an error code.  When validation fails,
 *     nothing is enqueued.  The library never aborts or prints.
 *   - m == 0, rows == 0 or n == 0 is a no-op returning QK_OK.
 *   - k must be a non-negative multiple of 32 (QK_ERR_INVALID_ARG otherwise).
 *   - Output ranges must not overlap input ranges (QK_ERR_INVALID_ARG).
 */
#ifndef QK_H
#define QK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Block formats (this library's own numbering). */
enum qk_format {
    QK_Q4_0 = 1,
    QK_Q4_1 = 2,
    QK_Q8_0 = 3,
    QK_Q5_0 = 4,
    QK_Q5_1 = 5
};

/* Element types.  QK_X8: blocks of 32 values in 36 bytes, an fp32 scale d and
 * then 32 int8 codes q, value d*q; rows of k/32 blocks back to back.  An output
 * of qk_rms_norm and the input of qk_mul_mat_vec_x8q only. */
enum qk_dtype {
    QK_F32 = 0,
    QK_F16 = 1,
    QK_X8 = 2
};

/* Element types of a key-value cache. */
enum qk_kv_type {
    QK_KV_F16 = 0,
    QK_KV_I8 = 1    /* int8 codes, one fp32 scale per token and head */
};

/* Scores of qk_moe_route. */
enum qk_score {
    QK_SOFTMAX = 0,
    QK_SIGMOID = 1
};

/* Status codes. */
enum qk_status {
    QK_OK = 0,
    QK_ERR_INVALID_ARG = 1,   /* null pointer, bad size, k % 32 != 0, n out of
                                 range, ld too small, overlapping in/out */
    QK_ERR_UNSUPPORTED = 2,   /* unknown format or output dtype */
    QK_ERR_ALIGNMENT = 3,     /* w not 2-byte aligned, or x / y / out not
                                 aligned to their element size */
    QK_ERR_LAUNCH = 4         /* the HIP runtime refused the kernel launch */
};

/* Bytes per 32-weight block: 18, 20, 34, 22 or 24; 0 for an unknown format. */
size_t qk_block_bytes(int fmt);

/* Bytes of one row of k weights (k a multiple of 32); 0 on a bad argument. */
size_t qk_row_bytes(int fmt, int64_t k);

/* Static, human-readable name of a status code (never NULL). */
const char *qk_status_string(int status);

/* Library version as an integer (major*10000 + minor*100 + patch). */
int qk_version(void);

/*
 * qk_dequantize - convert a rows x k quantized matrix to fp32 or fp16.
 *
 *   out[r*k + c] = W[r, c]   for r < rows, c < k.
 *
 * fp32: the value is computed in fp32 in the order shown in the format table
 * (multiply, then add; no fused multiply-add), which is exact for Q4_0, Q8_0
 * and Q5_0 and one round-to-nearest-even for Q4_1 and Q5_1.  Q4_0 with q = 8
 * gives +0.0; Q5_0 with q = 16 gives a zero with the sign of d.
 * fp16: one round-to-nearest-even of that fp32 value (overflow to +-inf,
 * subnormals kept).
 * Source: dequantize_block_q4_0 / _q4_1 / _q8_0_f16 hunks and the
 * ggml_get_to_fp16_cuda / ggml_get_to_fp32_cuda dispatch in the same diff.
 *
 *   fmt        QK_Q4_0, QK_Q4_1, QK_Q8_0, QK_Q5_0 or QK_Q5_1
 *   w          rows*k/32 blocks; 2-byte aligned
 *   rows, k    rows >= 0, k >= 0, k % 32 == 0
 *   out_dtype  QK_F32 or QK_F16
 *   out        rows*k elements of out_dtype, aligned to the element size
 *   stream     hipStream_t or NULL
 */
int qk_dequantize(int fmt, const void *w, int64_t rows, int64_t k,
                  int out_dtype, void *out, void *stream);

/*
 * qk_mul_mat_vec - fused quantized GEMV for decode: dequantize in registers
 * and multiply by 1..8 fp32 activation vectors, accumulating in fp32.
 *
 *   y[j*ldy + i] = sum_c W[i, c] * x[j*ldx + c]   for i < m, j < n   (overwrite)
 *
 * Each product uses the exact fp32 weight value, so the result is within a
 * few fp32 roundings per term of the exact sum: |y - exact| is a small
 * multiple of 2^-24 * sum_c |W[i,c] x[j*ldx+c]|.  With 4..8 columns, weights
 * 4-byte aligned with an even block count and k <= 4096, the multiply-adds
 * run on the matrix cores (fp32 MFMA, each a fused multiply-add with one
 * rounding, like the vector ALU's), in a different order than the vector-ALU
 * kernel the other cases use.
 * Source: dequantize_mul_mat_vec (the "dmmv" tuning block) and the
 * ggml_cuda_op_mul_mat row-range x column-count driver in the same diff,
 * which use it when the right operand is a vector.
 *
 *   w          m rows of k/32 blocks; 2-byte aligned
 *   m, k       m >= 0, k >= 0, k % 32 == 0
 *   x          fp32, 4-byte aligned; n columns, stride ldx >= k
 *   n          0..8 (0 is a no-op; above 8: QK_ERR_INVALID_ARG)
 *   y          fp32, 4-byte aligned; n columns, stride ldy >= m
 */
int qk_mul_mat_vec(int fmt, const void *w, int64_t m, int64_t k,
                   const float *x, int64_t n, int64_t ldx,
                   float *y, int64_t ldy, void *stream);

/*
 * qk_mul_mat_vec_x8 - quantized GEMV with 8-bit activations and integer dot
 * products: as qk_mul_mat_vec, but every 32-element block of each activation
 * column is first quantized (inside the kernel, no scratch memory) to codes
 * q = round-half-even(x / d) with a power-of-two scale d = 2^e, e the
 * smallest integer >= -126 with 127 * 2^e >= max|x| over the block (d = 0 for
 * an all-zero block; d = NaN for a block holding an infinite or NaN value,
 * so every output that uses such a block is NaN), and the products use
 * x^ = d * q:
 *
 *   y[j*ldy + i] = sum_c W[i, c] * x^[j][c]      for i < m, j < n   (overwrite)
 *
 * Per block the weight and activation codes meet in exact 4-way int8 dot
 * products; the result is scaled by d_w * d in fp32 (and Q4_1 adds
 * m_w * d * sum q), so |y - sum_c W x^| is a few fp32 roundings of those
 * per-block terms.  Against the fp32 activations the quantization adds at
 * most sum_c |W[i, c]| * d / 2.
 * Source: the integer-dot GEMV (mul_mat_vec_q, fed by a q8_1 activation
 * quantization) that the "llama_cpp 0.12.1 -> 0.12.2" ggml-cuda.cu diff names
 * in ggml_cuda_mul_mat's kernel choice; its activation format is not on the
 * page, and the power-of-two block scale is this library's.
 *
 * Arguments, layouts and errors as qk_mul_mat_vec (n = 1..8).
 */
int qk_mul_mat_vec_x8(int fmt, const void *w, int64_t m, int64_t k,
                      const float *x, int64_t n, int64_t ldx,
                      float *y, int64_t ldy, void *stream);

/*
 * qk_mul_mat_vec_x8q - qk_mul_mat_vec_x8 over activations that are in 8 bits
 * already: x is n columns of k/32 QK_X8 blocks (fp32 scale, 32 int8 codes),
 * as qk_rms_norm writes them; several products of one vector then share one
 * quantization.  Any scale and codes -128..127 are taken (the product of a
 * weight's and an activation's scale is rounded to fp32).  With the blocks that
 * qk_mul_mat_vec_x8 makes of the same activations the outputs of one column
 * are the same, bit for bit; more columns may run on the matrix cores (exact
 * integer products, fp32 sums over the blocks in another order), and the two
 * then agree within the error bound.
 * The call pays from three or four columns; for one or two, qk_mul_mat_vec on
 * the fp32 activations is as fast or faster, and more precise (Q4_0 4096 x 4096
 * with 1 / 2 / 3 / 4 / 8 columns 5.8 / 6.1 / 6.0 / 6.0 / 6.2 us against 4.5 / 5.4 /
 * 6.4 / 7.6 / 10.4, weights in no cache).
 *
 *   xq         QK_X8 blocks, 4-byte aligned; column j starts at byte j*ldx
 *   ldx        bytes, a multiple of 4, >= k/32*36 (ignored if n == 1)
 * Other arguments, layouts and errors as qk_mul_mat_vec (n = 0..8).
 */
int qk_mul_mat_vec_x8q(int fmt, const void *w, int64_t m, int64_t k,
                       const void *xq, int64_t n, int64_t ldx,
                       float *y, int64_t ldy, void *stream);

/* One problem of a grouped GEMV: y = W x (layout as in qk_mul_mat_vec). */
typedef struct qk_mat_vec_item {
    const void *w;      /* m rows of k/32 blocks, 2-byte aligned */
    int64_t m;          /* rows, m >= 0 (0: skipped) */
    int64_t k;          /* weights per row, k >= 0, k % 32 == 0 */
    const float *x;     /* n fp32 columns of length k, stride ldx >= k */
    int64_t ldx;
    float *y;           /* n fp32 columns of length m, stride ldy >= m */
    int64_t ldy;
} qk_mat_vec_item;

/* Largest `count` qk_mul_mat_vec_batched accepts. */
#define QK_MAX_BATCH 16

/*
 * qk_mul_mat_vec_batched - several independent GEMVs of one format and one
 * column count n in a single launch (for example the q/k/v/o, gate/up and down
 * projections of one decode step, or a set of expert matrices); one launch
 * amortizes the fixed launch cost over all items' weights.  Each item is
 * computed exactly as qk_mul_mat_vec would compute it, bit for bit, except
 * where a single call of 4..8 columns would take the matrix-core kernel: a
 * grouped launch computes every item on the vector ALU, and the two agree
 * within the error bound.  (A one-item call is a single call.)
 * Source: as qk_mul_mat_vec (dequantize_mul_mat_vec under ggml_cuda_op_mul_mat,
 * "llama_cpp 0.12.1 -> 0.12.2" ggml-cuda.cu diff), applied per item.
 *
 *   items      host array of `count` problems (read during the call only)
 *   count      0..QK_MAX_BATCH (0 is a no-op)
 *   n          1..8 columns for every item (0 is a no-op)
 * Errors as qk_mul_mat_vec for each item; additionally QK_ERR_INVALID_ARG for
 * count out of range, items == NULL with count > 0, or an output overlapping
 * any input or any other item's output.
 */
int qk_mul_mat_vec_batched(int fmt, const qk_mat_vec_item *items, int count, int64_t n,
                           void *stream);

/*
 * qk_mul_mat_vec_id - expert-indexed GEMV for mixture-of-experts decode: for
 * every token t and slot s, the GEMV of the expert matrix that ids selects,
 * with the expert id read on the device (no host synchronisation).
 *
 *   e = ids[t*ld_ids + s]
 *   y[t*y_tok + s*y_slot + i] = sum_c W_e[i, c] * x[t*x_tok + s*x_slot + c]
 *        for i < m, s < n_used, t < n_tokens                          (overwrite)
 *   W_e = m rows of k/32 blocks starting at byte e*expert_stride of w
 *
 * Each (t, s) is computed exactly as qk_mul_mat_vec computes one column.  An
 * id outside [0, n_experts) selects nothing: its m outputs are set to NaN and
 * no weight outside the stack is read.
 * Source: ggml_cuda_mul_mat_id, named by a ggml-cuda.cu hunk of the
 * "ggml: backend-agnostic tensor parallelism" compare (whose commit list
 * mentions a Q4_0 expert model with intermediate dimension 768); its
 * definition is not printed there, and this follows ggml's mul_mat_id: one
 * product per (token, selected expert).
 *
 *   w              stack of n_experts matrices, 2-byte aligned
 *   n_experts      >= 1
 *   expert_stride  bytes between experts, even, >= one matrix (ignored if
 *                  n_experts == 1)
 *   m, k           m >= 0, k >= 0, k % 32 == 0
 *   ids            device int32, 4-byte aligned; token t's ids at t*ld_ids
 *   ld_ids         >= n_used (ignored if n_tokens == 1)
 *   n_used         slots per token, >= 0 (0 is a no-op)
 *   n_tokens       >= 0 (0 is a no-op)
 *   x              fp32, 4-byte aligned; x_slot = 0 gives every slot of a
 *                  token the same vector; strides >= 0, in elements
 *   y              fp32, 4-byte aligned; the n_used*n_tokens outputs must not
 *                  overlap: (y_slot >= m and y_tok >= (n_used-1)*y_slot + m)
 *                  or (y_tok >= m and y_slot >= (n_tokens-1)*y_tok + m)
 * Errors: QK_ERR_INVALID_ARG for the conditions above, n_used * n_tokens *
 * ceil(m/8) above INT32_MAX, a null pointer, or y overlapping w, ids or x;
 * QK_ERR_ALIGNMENT as listed; nothing is enqueued on an error.
 */
int qk_mul_mat_vec_id(int fmt, const void *w, int64_t n_experts, int64_t expert_stride,
                      int64_t m, int64_t k, const int32_t *ids, int64_t ld_ids,
                      int64_t n_used, int64_t n_tokens,
                      const float *x, int64_t x_slot, int64_t x_tok,
                      float *y, int64_t y_slot, int64_t y_tok, void *stream);

/*
 * qk_mul_mat - batched GEMM: weights dequantized to fp16 tiles in LDS and
 * multiplied by fp16 activations on the matrix cores, accumulating in fp32.
 *
 *   y[j*ldy + i] = sum_c f16(W[i, c]) * x[j*ldx + c]   for i < m, j < n
 *
 * f16(W) is the qk_dequantize fp16 value (one RNE of the fp32 weight).
 * Every format.
 * Source: the dequantize-to-fp16 then GEMM path (ggml_get_to_fp16_cuda feeding
 * the BLAS mul_mat) and ggml_cuda_mul_mat's choice of a batched kernel when
 * the right operand has more than one column, in the same diff.
 *
 *   x          binary16, 2-byte aligned; n columns, stride ldx >= k
 *   n          n >= 0
 *   y          fp32, 4-byte aligned; n columns, stride ldy >= m
 */
int qk_mul_mat(int fmt, const void *w, int64_t m, int64_t k,
               const void *x_f16, int64_t n, int64_t ldx,
               float *y, int64_t ldy, void *stream);

/*
 * qk_rms_norm - root-mean-square norm of n rows, with the residual's addition.
 *
 *   s[j][c] = x[j][c] + residual[j][c]                  (fp32)
 *   sum[j][c] = s[j][c]                                 (rounded to x_dtype)
 *   y[j][c] = s[j][c] / sqrt(mean_c(s[j][c]^2) + eps) * weight[c]
 *
 * The norm takes s before it is rounded.  The mean is held in fp64 and the
 * factor rounded to fp32 once; y is two more roundings, and one to its type.
 * QK_X8 outputs quantize each 32-element block of y to codes
 * q = round-half-even(y / d) with the scale rule of qk_mul_mat_vec_x8 (d a
 * power of two; 0 for an all-zero block; NaN, with codes 0, for a block that
 * holds an infinite or NaN value).
 *
 *   x_dtype    QK_F32 or QK_F16: x, residual and sum
 *   x          n rows of k elements, stride ldx >= k elements
 *   residual   as x (stride ldr), or NULL for none
 *   weight     fp32[k], or NULL for ones
 *   eps        >= 0
 *   k          >= 1, at most 2^30; a multiple of 32 for QK_X8 outputs
 *   sum        as x (stride lds), or NULL to leave it out; may be x or
 *              residual itself (the same pointer and stride)
 *   y_dtype    QK_F32, QK_F16 or QK_X8
 *   y          n rows; stride ldy in elements (>= k), for QK_X8 in bytes
 *              (>= k/32*36, a multiple of 4)
 * Strides are ignored if n == 1.  Pointers aligned to their element size.
 */
int qk_rms_norm(int x_dtype, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                const float *weight, double eps, int64_t n, int64_t k,
                void *sum, int64_t lds, int y_dtype, void *y, int64_t ldy, void *stream);

/*
 * A paged key-value cache.  Token `slot` of page `p` has, for key-value head
 * h, head_dim contiguous elements starting at element
 * p*page_stride + h*head_stride + slot*slot_stride of k (keys) and of v
 * (values), so that heads may lie outside or inside tokens.  Which pages hold
 * a sequence is told by a page table (device int32): token t of sequence s is
 * slot t % page_size of page table[s*ld_table + t / page_size].
 * QK_KV_I8: an element is code * scale, the scale of a token and head at
 * element p*scale_page_stride + h*scale_head_stride + slot*scale_slot_stride
 * of k_scale and of v_scale.
 * The struct is read during the call only; the pools are the caller's.
 */
typedef struct qk_kv_cache {
    int type;               /* enum qk_kv_type */
    void *k, *v;            /* 16-byte aligned pools */
    float *k_scale, *v_scale;   /* QK_KV_I8 (else ignored) */
    int64_t n_pages;        /* 1..INT32_MAX */
    int64_t n_heads;        /* key-value heads, 1..65535 */
    int64_t page_size;      /* tokens per page, 1..2^20 */
    int64_t head_dim;       /* a multiple of 32 from 32 to 256 */
    int64_t page_stride, head_stride, slot_stride;   /* elements; multiples of 16 bytes; >= 0 */
    int64_t scale_page_stride, scale_head_stride, scale_slot_stride;   /* elements; >= 0 */
} qk_kv_cache;

/*
 * qk_kv_store - write the keys and values of new tokens into a paged cache.
 *
 *   token i goes to position pos[i] of sequence seq[i]
 *
 * QK_KV_F16: rounded to nearest even (overflow to infinity).  QK_KV_I8: per
 * token and head, scale d = max|x| / 127 and codes round-half-even(x / d),
 * both divisions rounded to fp32 (d = 0 and codes 0 where that is 0; codes held
 * to +-127 where d is subnormal; d = NaN and codes 0 where a value is infinite
 * or NaN).
 * A token is left out, and nothing written for it, if its sequence or
 * position is outside the table or its page id outside the pool.  Two tokens
 * of one call must not have the same place.
 *
 *   k, v       fp32; token i, head h at element i*k_tok + h*k_head
 *              (v_tok, v_head), head_dim contiguous elements; strides 0..2^27
 *   n_tokens   >= 0 (0 is a no-op); 2*n_tokens*n_heads <= INT32_MAX
 *   table      device int32, n_seqs rows of max_pages ids, stride ld_table
 *   seq        device int32[n_tokens], or NULL: token i is of sequence i
 *   pos        device int32[n_tokens]
 * Errors: QK_ERR_INVALID_ARG also where rows of the pools overlap.  Keys and
 * values may share memory that holds both in turn (pages, tokens or heads of
 * keys and then values), scales likewise; codes and scales lie apart.
 */
int qk_kv_store(const qk_kv_cache *cache, const float *k, int64_t k_tok, int64_t k_head,
                const float *v, int64_t v_tok, int64_t v_head, int64_t n_tokens,
                const int32_t *table, int64_t ld_table, int64_t n_seqs, int64_t max_pages,
                const int32_t *seq, const int32_t *pos, void *stream);

/*
 * qk_attn_decode - attention of one new token per sequence over a paged cache.
 *
 *   z_t = scale * q . K_t    for the tokens t < lens[s] that the query sees
 *   y   = sum_t exp(z_t) V_t / sum_t exp(z_t)
 *
 * Query head h of n_q_heads takes key-value head h / (n_q_heads / n_heads).
 * With window > 0 the query (the token at lens[s] - 1) sees the last `window`
 * tokens and the first `sinks`; with window == 0 all of them.  Tokens that
 * are not seen are not used, whatever their pages hold, and table entries of
 * pages without a token that is seen are not followed.
 * lens[s] <= 0: zeros.  NaN: lens[s] above max_len, or a page id outside the
 * pool.  The result does not depend on what other sequences hold or on their
 * lengths, and is the same on every run; n_seqs and max_len decide into how many
 * parts a sequence is split, and with that the order of its sums.
 * The scores take q in two fp16 parts (2^-21 of the row's largest |q|), exact
 * keys and fp32 sums; probabilities keep the 24 bits and the exponent of fp32,
 * also where they meet the values.
 * A key that is infinite (an fp16 overflow) with a score of -infinity has
 * probability 0; a score of +infinity, or of -infinity alone, gives NaN.
 *
 *   q          fp32; sequence s, head h at element s*q_seq + h*q_head,
 *              head_dim contiguous elements; strides 0..2^27
 *   n_seqs     >= 0 (0 is a no-op); n_seqs*n_q_heads <= INT32_MAX
 *   n_q_heads  a multiple of the cache's n_heads, at most 2^20
 *   table      device int32, n_seqs rows of the pages of max_len tokens
 *              (ceil(max_len / page_size); entries that are not followed may
 *              hold anything), stride ld_table (ignored if n_seqs == 1)
 *   lens       device int32[n_seqs]: tokens in the cache, the new one among them
 *   max_len    1..2^30, no length is above it; the parts are sized for it, so
 *              a bound far above the lengths costs time (1000 tokens of 8 x 128
 *              8.8 us with their own bound, 21.6 with 131072)
 *   window, sinks   >= 0
 *   y_dtype    QK_F32 or QK_F16; y laid out as q with y_seq, y_head; the rows
 *              must not overlap
 *   workspace  device memory, 16-byte aligned, of the bytes that
 *              qk_attn_decode_workspace gives for these arguments or larger
 *              ones (NULL if 0); it need not be cleared, and is free for other
 *              use once the enqueued work is done
 */
int qk_attn_decode(const qk_kv_cache *cache, const float *q, int64_t q_seq, int64_t q_head,
                   int64_t n_seqs, int64_t n_q_heads, const int32_t *table, int64_t ld_table,
                   const int32_t *lens, int64_t max_len, float scale, int64_t window, int64_t sinks,
                   int y_dtype, void *y, int64_t y_seq, int64_t y_head,
                   void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace that serve qk_attn_decode with up to n_seqs sequences, any
 * max_len up to the given one and, with a window, any window and sinks up to
 * the given ones, over this cache and with n_q_heads; 0 where none of these
 * needs any, and on a bad argument. */
size_t qk_attn_decode_workspace(const qk_kv_cache *cache, int64_t n_seqs, int64_t n_q_heads,
                                int64_t max_len, int64_t window, int64_t sinks);

/*
 * qk_moe_route - choose experts for tokens: the ids that qk_mul_mat_vec_id
 * takes, and their weights.
 *
 *   score = softmax or sigmoid of the token's logits (over all experts)
 *   value = score + bias          (bias decides the choice only)
 *   with n_groups > 1, experts outside the topk_groups best groups are left
 *   out; a group is n_experts/n_groups neighbours, its value the sum of its
 *   group_top (1 or 2) largest values
 *   ids[t][i] = the expert with the i-th largest value, i < n_used
 *   weights[t][i] = score of that expert, over the sum of the n_used with
 *   renorm != 0, times scale
 *
 * Equal values: the lowest index first (groups too).  Without a bias and with
 * group_top == 1 the logits are compared, which both scores rise with; else
 * the fp32 values, whose softmax sum is held in fp64 and rounded once, so that
 * the choice does not hang on the order of a sum.  A NaN value comes last.
 * The ids of a token are always n_used different experts.  Scores of a row
 * of -infinity alone are 0 under softmax; weights whose sum is 0 are 0 with
 * renorm.
 *
 *   logits     fp32, n_tokens rows of n_experts, stride ldx >= n_experts
 *   n_experts  1..1024
 *   n_used     1..64, at most topk_groups * (n_experts / n_groups)
 *   score      QK_SOFTMAX or QK_SIGMOID
 *   bias       fp32[n_experts], or NULL for none
 *   n_groups   1..64, divides n_experts; topk_groups 1..n_groups
 *   ids        int32, stride ld_ids >= n_used
 *   weights    fp32, stride ldw >= n_used
 * Strides are ignored if n_tokens == 1; n_tokens == 0 is a no-op.
 */
int qk_moe_route(const float *logits, int64_t ldx, int64_t n_tokens, int64_t n_experts,
                 int64_t n_used, int score, const float *bias, int64_t n_groups,
                 int64_t topk_groups, int64_t group_top, int renorm, float scale,
                 int32_t *ids, int64_t ld_ids, float *weights, int64_t ldw, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QK_H */
