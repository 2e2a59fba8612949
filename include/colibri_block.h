/*
 * colibri_block.h -- C ABI of the operators around the layer, part of
 * libcolibri.so: what turns the previous layer's output into the next layer's
 * hidden state.  The residual addition with the root-mean-square norm and its
 * Q8_0 form, a quantised matrix product with bias, activation and residual, and
 * attention over a paged int8 cache with its append and read-back.
 *
 * The conventions at the top of colibri.h hold, and its status codes, banks and
 * streams are used.  Lengths that live in device memory are read by the kernels,
 * so every call here can be captured into a graph and replayed on changed ones.
 */
#ifndef COLIBRI_BLOCK_H
#define COLIBRI_BLOCK_H

#include "colibri.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations. */
enum { COLI_F32 = 32, COLI_BF16 = 16 };

/* Activations of the linear product's epilogue: GELU is the exact one,
 * v * (1 + erf(v / sqrt 2)) / 2; SiLU is v / (1 + exp(-v)). */
enum { COLI_ACT_NONE = 0, COLI_ACT_RELU = 1, COLI_ACT_SILU = 2, COLI_ACT_GELU = 3 };

#define COLI_MAX_LINEAR_ROWS (1 << 20)
#define COLI_MAX_LINEAR_K (1 << 15)
#define COLI_KV_BLOCK 64 /* tokens of a cache page, and of one scale */
#define COLI_MAX_SEQS 65535
#define COLI_MAX_SEQ_PAGES (1 << 24)
#define COLI_MAX_KV_HEADS 1024

/*
 * Residual addition and root-mean-square norm.  For each row
 *   t = x + residual              (fp32; t = x where residual is null)
 *   y = t * (1 / sqrt(mean(t^2) + eps)) * weight
 * computed and held in fp32, from t before any rounding.  Outputs, each of
 * which may be null, but not all: sum = t rounded to residual_type; y rounded
 * to y_type; q and d (both or neither) = Q8_0 of the unrounded y by the rule
 * of colibri_quantize_q8_0.  x and residual have rows x_stride and
 * residual_stride elements apart; weight is fp32 [K]; sum, y, q and d are
 * contiguous.  sum may be residual or x itself (same type, stride K); no other
 * overlap.  residual_type is the type of both residual and sum.
 * K % 32 == 0, K <= COLI_MAX_DIM, eps >= 0 and finite; fp32 pointers 16-byte,
 * bf16 pointers 8-byte, q 4-byte aligned; strides multiples of 4, at least K.
 * rows == 0 is a no-op.
 */
typedef struct coli_norm {
    const void* x;
    const void* residual;
    const float* weight;
    void* sum;
    void* y;
    int8_t* q;
    float* d;
    int64_t x_stride, residual_stride;
    int32_t rows, K;
    int32_t x_type, residual_type, y_type;
    float eps;
} coli_norm;

int colibri_add_rms_norm(const coli_norm* n, coli_stream_t stream);

/*
 * Quantised matrix product with its epilogue, for W a bank of one matrix
 * [rows][K] and activations in Q8_0 form (xq int8 [S][K], xd fp32 [S][K/32]):
 *   out[t][r] = act(sum_k scale(r, k) * code(r, k) * xq[t][k] * xd[t][k/32] + bias[r]) + residual[t][r]
 * bias fp32 [rows] or null; residual [S][rows] of out_type or null, and may be
 * out itself; out [S][rows] of out_type, rounded once.  Sums are held in
 * fp32; their order depends on the shape, not on the data, so equal calls give
 * equal bits, but a token's result may differ in the last bits between batch
 * sizes.  Products inside a 32-element block are exact integers; only for bf16
 * outputs of very many tokens (one scale per row) the activations xq * xd enter the
 * matrix cores rounded to fp16 instead, by up to 2^-11 of their value (an eighth of
 * the output's own 2^-8) or 2^-31 of the token's largest scale, whichever is more.
 * SiLU is within 2^-23 (|v| + 8) of its value, GELU within 2^-22 of 1 + |v|.  NaN
 * comes out as NaN.
 * 1 <= rows <= COLI_MAX_LINEAR_ROWS, K <= COLI_MAX_LINEAR_K, K % 32 == 0;
 * xq and W->data 16-byte, out and residual 4-byte aligned.  ws as sized by
 * colibri_linear_workspace_bytes for this bank and type and for S or more
 * tokens (0: invalid arguments).  S == 0 is a no-op.
 */
size_t colibri_linear_workspace_bytes(const coli_qbank* W, int32_t S, int32_t out_type);
int colibri_linear_q(const coli_qbank* W, const int8_t* xq, const float* xd, int32_t S, const float* bias,
                     int32_t act, const void* residual, void* out, int32_t out_type, void* ws,
                     size_t ws_bytes, coli_stream_t stream);

/*
 * A paged cache of keys and values in int8.  A page holds one block of
 * COLI_KV_BLOCK = 64 tokens of every head, with one fp32 scale per (page, head)
 * for keys and one for values: value = code * scale.  k and v: int8
 * [n_pages][n_heads][64 * head_dim], 16-byte aligned; k_scale and v_scale:
 * fp32 [n_pages][n_heads].  Inside a page and head the codes lie in the order
 * in which the matrix cores take them (D = head_dim):
 *   key   (token t, dim c): (t / 32) * 32 D + (c / 16) * 512 + (t % 32) * 16 + c % 16
 *   value (token t, dim c): (t / 32) * 32 D + c * 32 + ((t / 4) % 2) * 16 + ((t % 32) / 8) * 4 + t % 4
 * head_dim is 64, 128, 192 or 256.  Memory of pages that no token was written
 * to needs no initialisation.
 */
typedef struct coli_kv_cache {
    int8_t* k;
    int8_t* v;
    float* k_scale;
    float* v_scale;
    int32_t n_pages, n_heads, head_dim;
} coli_kv_cache;

/*
 * The sequences of one call.  Sequence s owns the rows cu_q[s] .. cu_q[s+1]-1
 * of the packed per-token tensors and has kv_len[s] tokens in the cache, those
 * rows among them: row i of its q_len rows is its token kv_len - q_len + i.
 * Token j lies in page page_table[s][j / 64], place j % 64.  cu_q int32
 * [n_seq + 1], kv_len int32 [n_seq] and page_table int32 [n_seq][max_pages]
 * are device memory.  An entry of page_table outside [0, n_pages) is a missing
 * page: its tokens are not written, read as zeros, and are seen by no query.
 * cu_q does not decrease.  kv_len is taken as at most max_pages * 64 and at least
 * 0, cu_q entries as at most n_tokens; rows before cu_q[0] and from cu_q[n_seq]
 * on are left as they are.  max_q is the
 * expected longest q_len: it sizes the launch, longer ones are slower and
 * equally right.
 */
typedef struct coli_kv_batch {
    const int32_t* page_table;
    const int32_t* cu_q;
    const int32_t* kv_len;
    int32_t n_seq, max_pages;
    int32_t n_tokens; /* rows of the packed tensors */
    int32_t max_q;
} coli_kv_batch;

/*
 * Writes the rows of k and v ([n_tokens][n_heads][head_dim] of `type`, tokens
 * k_stride / v_stride elements apart) to their places, for keys and values
 * alike: the scale of each touched (page, head) becomes
 *   s' = max(s, amax / 127),   amax = max |new values of that block and head|,
 * s being the old scale, or 0 where the block's first token is new; tokens
 * that the block held before are requantised, c' = rnd(c * (s * (1/s'))), new
 * ones get rnd(v * (1/s')), rnd rounding half away from zero and clamping to
 * [-127, 127]; s' = 0 gives codes 0.  Rows with a negative token number are
 * skipped.  Values are finite.  A page that is written stands once in the batch's
 * table, in one place of one sequence.  16-byte (fp32) or 8-byte (bf16) aligned, strides multiples
 * of 4, at least n_heads * head_dim.
 */
int colibri_kv_append(const coli_kv_cache* cache, const coli_kv_batch* batch, const void* k, const void* v,
                      int32_t type, int64_t k_stride, int64_t v_stride, coli_stream_t stream);

/* The values of the rows' tokens, code * scale rounded to `type`, in k and v
 * [n_tokens][n_heads][head_dim] (contiguous; either may be null, not both;
 * 16-byte (fp32) or 8-byte (bf16) aligned).  With q_len = kv_len this reads
 * whole sequences back. */
int colibri_kv_read(const coli_kv_cache* cache, const coli_kv_batch* batch, void* k, void* v, int32_t type,
                    coli_stream_t stream);

/*
 * Attention of the rows' queries over their sequences' cached tokens:
 *   out = sum_j p_j v_j,  p_j = exp(scale q.k_j - lse),  lse = log sum_j exp(scale q.k_j)
 * over the tokens j that the query sees: every cached one, with causal != 0
 * those up to its own token, with window > 0 (causal only) the last `window`
 * of these.  A query that sees none gets out = 0, lse = -inf.  q, out:
 * [n_tokens][n_heads][head_dim] of `type`, tokens q_stride / out_stride
 * elements apart; n_heads is a multiple of the cache's, query head h reads
 * cache head h / (n_heads / cache heads).  lse: fp32 [n_tokens][n_heads] or
 * null.  max_kv is the expected longest kv_len, used like max_q.  q and out
 * 16-byte aligned, strides multiples of 8, at least n_heads * head_dim; out
 * overlaps nothing.  scale is finite, of either sign; n_tokens * (n_heads /
 * cache heads) is under 2^31.  A query with a NaN or an infinity gets NaN in its
 * own out and lse.  A query row enters the scores as whole multiples of a unit,
 * its largest magnitude / 32512 for bf16 and / 8323072 for fp32: a score is off by
 * at most half of one times |scale| sum_c |k_c|, and what lies 2^16 (fp32: 2^24)
 * below the row's largest value takes no part.  Their products with the codes are
 * exact, scores are rounded to fp32 once, softmax statistics and sums are fp32;
 * for bf16 the weights p enter the value product rounded to bf16 (2^-8), for fp32
 * as three bf16 terms.  ws as sized by colibri_kv_attention_workspace_bytes (0: invalid
 * arguments) for this cache's n_heads and head_dim, this type and number of
 * heads, and either exactly this n_seq, n_tokens, max_q and max_kv or, if
 * n_tokens <= n_seq * max_q here, larger ones.
 */
typedef struct coli_kv_attn {
    const void* q;
    void* out;
    float* lse;
    int64_t q_stride, out_stride;
    int32_t type, n_heads;
    int32_t causal, window;
    int32_t max_kv;
    float scale;
} coli_kv_attn;

size_t colibri_kv_attention_workspace_bytes(const coli_kv_cache* cache, const coli_kv_batch* batch,
                                            const coli_kv_attn* attn);
int colibri_kv_attention(const coli_kv_cache* cache, const coli_kv_batch* batch, const coli_kv_attn* attn,
                         void* ws, size_t ws_bytes, coli_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif
