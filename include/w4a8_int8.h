/*
 * w4a8_int8.h -- the 8-bit integer path around the codebook layer: an int8
 * layer, and the attention block's steps over an int8 paged cache, on NVIDIA
 * B200 (sm_100a).  Part of the library that w4a8.h declares.
 *
 * The conventions of w4a8.h hold for every call here: device pointers owned
 * by the caller, no allocation, asynchronous on `stream`, arguments checked
 * on the host before anything is launched, the current device must be
 * sm_100.  bf16 values are passed as their bit patterns (uint16).  Buffers
 * of values, codes and scales must be 16-byte aligned; the index arrays
 * (positions, block table, q_start, kv_len, page lists) 4-byte aligned.
 * Quantisation is the one of w4a8_rotate_quant_act: symmetric, absmax / 127,
 * round half to even.  Inputs are finite, and so are, in fp32, the norms' sums
 * of squares and the attention's scores times log2(e).
 */
#ifndef W4A8_INT8_H_
#define W4A8_INT8_H_

#include "w4a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * The int8 layer: y = x W^T with int8 weights and int8 activations.
 *
 * For the layers that the codebook format does not hold: layers kept out of
 * 4 bits for their accuracy, and layers whose input width the rotation block
 * does not divide (4304 = 16 x 269; ConvRot card, the divisibility rule).
 *   w ~ s_w[n] w_q[n, k],  x ~ s_x[m] x_q[m, k]   (codes int8, scales fp32)
 *   y[m, n] = bf16( s_x[m] s_w[n] sum_k x_q[m, k] w_q[n, k] )
 * The sum is exact (int32).  With `rotate`, x is rotated per 256-block of K
 * by H_256 / 16 before it is quantised, and the weights must have been
 * (w4a8_int8_quantize with rotate); K must then be a multiple of 256.
 * Shapes: M in [1, 16 776 960], N in [1, 2^24], K a positive multiple of 16,
 * at most W4A8_MAX_K.  Weights and their scales are read before a kernel
 * that precedes the call on the stream has completed, if that kernel allows
 * it (programmatic launch); those of this library that write them do not.
 * ------------------------------------------------------------------------ */

/*
 * Quantise R rows of x [R, K] (fp32 when x_is_f32 != 0, else bf16 bits):
 * codes [R, K] int8, s [R] fp32; a row of zeros gives s = 0 and codes 0.
 * Serves weights (rows = output channels) and activations (rows = tokens);
 * a rotated bf16 row gets the codes of w4a8_rotate_quant_act.
 * Errors: NULL, SHAPE, ALIGN, ARCH, CUDA.
 */
w4a8_status w4a8_int8_quantize(const void* x, int32_t x_is_f32, int64_t R, int64_t K, int32_t rotate,
                               int8_t* codes, float* s, void* stream);

/*
 * y [M, N] (bf16 bits) from codes x_q [M, K], w_q [N, K] and scales s_x [M],
 * s_w [N].  Errors: NULL, SHAPE, ALIGN, ARCH, CUDA; a bounded wait that gives
 * up leaves y undefined and is reported by w4a8_get_device_error.
 */
w4a8_status w4a8_int8_gemm(const int8_t* x_q, const float* s_x, int64_t M, const int8_t* w_q,
                           const float* s_w, int64_t N, int64_t K, uint16_t* y, void* stream);

/*
 * Workspace bytes of w4a8_int8_linear (0 for a bad shape): scratch that the
 * quantised activations pass through, in any state.  Two calls that share a
 * workspace must be ordered on the GPU (captured graphs that are replayed at
 * the same time need one each).
 */
size_t w4a8_int8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N);

/*
 * The layer: x [M, K] (bf16 bits) is quantised into the workspace, then
 * w4a8_int8_gemm.  Errors: as w4a8_int8_gemm, and WORKSPACE.
 */
w4a8_status w4a8_int8_linear(const uint16_t* x, int64_t M, int64_t K, int32_t rotate, const int8_t* w_q,
                             const float* s_w, int64_t N, uint16_t* y, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Heads: norm and position rotation
 * ------------------------------------------------------------------------ */

/*
 * bf16 rows [token][head][D], the D values of a head contiguous; strides in
 * elements, multiples of 8 (so that the q, k and v parts of one projection's
 * output can be passed as they lie).
 */
typedef struct {
  uint16_t* data;
  int64_t token_stride, head_stride;
  int32_t heads;
} w4a8_heads;

/*
 * Rotation of pairs by position * inv_freq[i], i < rot_dim / 2: pairs
 * (i, i + rot_dim / 2), or (2 i, 2 i + 1) when `interleaved`; the remaining
 * D - rot_dim values of a head are not turned.  inv_freq is fp64 (device)
 * and carries any scaling for long contexts; `factor` multiplies cosine and
 * sine (the attention factor of such a scaling, else 1).  Angles are formed
 * in fp64 and brought within half a turn there; their sines and cosines are
 * the hardware's, off by up to about 2^-21.  inv_freq NULL: no rotation.  rot_dim is a multiple of 16, at
 * most D.
 */
typedef struct {
  const double* inv_freq;
  int32_t rot_dim, interleaved;
  float factor;
} w4a8_rope;

/*
 * RMS norm of each head of q and k, then the rotation, in one pass:
 *   n = x * rsqrt(mean(x^2) + eps) * weight,  out = rotate(n)
 * in fp32, rounded once to bf16.  q_weight / k_weight are fp32 [D]; NULL
 * leaves that norm out.  q.data or k.data may be NULL (then only the other
 * is done).  An output may be its input (same address and strides, else
 * SHAPE); otherwise outputs share no memory with each other or with an input,
 * and the rows of an output none among themselves (SHAPE).  positions [T]
 * int32 (may be NULL without a rotation).  D is 64, 128 or 256; T in [1, 2^24].
 * Errors: NULL, SHAPE, ALIGN, ARCH, CUDA.
 */
w4a8_status w4a8_qk_norm_rope(const w4a8_heads* q, const w4a8_heads* k, int64_t T, int32_t D,
                              const float* q_weight, const float* k_weight, float eps,
                              const int32_t* positions, const w4a8_rope* rope, const w4a8_heads* q_out,
                              const w4a8_heads* k_out, void* stream);

/* ------------------------------------------------------------------------
 * The int8 paged cache
 *
 * Codes int8 [pages][kv_heads][page][D] and scales fp32 [pages][kv_heads]
 * for K and for V: a page holds `page` consecutive tokens of one sequence,
 * and every (page, head) has its own scale.  page is 16, 32, 64 or 128, D
 * 64, 128 or 256, and pages * kv_heads * page is below 2^31.  The buffers
 * need no initialisation.
 *
 * A batch is B sequences.  Sequence b has the new tokens (rows) q_start[b]
 * .. q_start[b + 1] - 1, which are the last of the kv_len[b] tokens that the
 * cache holds of it; its token t lies in page table[b][t / page].  Entries
 * past a sequence's pages are not read, nor, by w4a8_kv_attention with a
 * window, those of pages that lie before every new token's window.  Rows from q_start[B] up to `tokens`
 * belong to no sequence: outputs there are left as they were.  Numbers that
 * do not fit together (rows outside [0, tokens], more new tokens than
 * kv_len, kv_len past the table) leave that sequence out, and page ids
 * outside [0, pages) leave those tokens out; w4a8_get_device_error then
 * reports W4A8_ERR_INPUT and that sequence's results are undefined (where
 * q_start goes back, so that sequences share rows, those of all of them).
 * ------------------------------------------------------------------------ */
typedef struct {
  int8_t* k_codes;
  int8_t* v_codes;
  float* k_scales;
  float* v_scales;
  int64_t pages;
  int32_t kv_heads, page, head_dim;
} w4a8_kv_cache;

typedef struct {
  const int32_t* table;   /* [batch][table_stride] page ids */
  int64_t table_stride;   /* at most 2^30 / page */
  const int32_t* q_start; /* [batch + 1] */
  const int32_t* kv_len;  /* [batch] */
  int64_t batch;          /* in [1, 65536] */
  int64_t tokens;         /* rows of q, k, v and the outputs, in [1, 2^24] */
} w4a8_kv_batch;

/*
 * Write the new tokens' K and V into the cache, with the norm and rotation
 * of w4a8_qk_norm_rope on K (quantised from fp32, without a rounding to bf16
 * in between) and, when q is given, on q, in the same launch:
 *   scale' = max(scale, absmax(new values) / 127), where scale counts as 0
 *   if the page's first token is written by this call; codes that were there
 *   become rint(code * (scale / scale')) when it grew.
 * k, v [tokens][kv_heads][D]; q and q_out (data NULL: none) [tokens][heads][D];
 * q_out may be q, as in w4a8_qk_norm_rope.
 * positions NULL: a token's position is its place in the sequence.  A call
 * writes each page for one sequence and one place of its block table (a page
 * id that stands there twice gets undefined contents).
 * Errors: NULL, SHAPE, ALIGN, ARCH, CUDA.
 */
w4a8_status w4a8_kv_update(const w4a8_kv_cache* cache, const w4a8_kv_batch* batch, const w4a8_heads* k,
                           const w4a8_heads* v, const w4a8_heads* q, const float* q_weight,
                           const float* k_weight, float eps, const int32_t* positions,
                           const w4a8_rope* rope, const w4a8_heads* q_out, void* stream);

/*
 * Pages back to values: k_out, v_out bf16 [n][kv_heads][page][D] = code *
 * scale of the pages ids[0 .. n) (an id outside the cache gives zeros and
 * W4A8_ERR_INPUT).  The counterpart of w4a8_unpack_dequant for the cache.
 * Errors: NULL, SHAPE, ALIGN, ARCH, CUDA.
 */
w4a8_status w4a8_kv_dequant(const w4a8_kv_cache* cache, const int32_t* ids, int64_t n, uint16_t* k_out,
                            uint16_t* v_out, void* stream);

/*
 * Workspace bytes of w4a8_kv_attention (0 for a bad shape); zero-filled
 * before its first use; every completed call leaves the words that must be
 * zero so, for any shape.  Two calls that share a workspace must be ordered
 * on the GPU (captured graphs that are replayed at the same time need one
 * each).  After a call that reported W4A8_ERR_TIMEOUT, zero it again.
 */
size_t w4a8_kv_attention_workspace_bytes(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim);

/*
 * Causal attention of the new tokens over the cache, which already holds
 * them (w4a8_kv_update):
 *   out_i = sum_j softmax_j(scale q_i . K_j) V_j,  j <= position of i,
 *   and j > position - window when window > 0,
 * K, V = code * scale (a V scale below 2^-80 may count as 0).  Scores, the
 * softmax's maxima and sums, and out until its one rounding are fp32 (q and the
 * codes are exact in the products' fp16 operands); the weights are rounded to
 * fp16 (11 bits) for the product with V, and what is below 2^-32 of a row's
 * largest weight * V scale may count as 0.  q, out
 * [tokens][q_heads][D], q_heads a multiple of kv_heads and at most 128 of them
 * to a key head (head h reads key head h / (q_heads / kv_heads)); out may be q,
 * as in w4a8_qk_norm_rope.
 * Errors: NULL, SHAPE, ALIGN, WORKSPACE, ARCH, CUDA.
 */
w4a8_status w4a8_kv_attention(const w4a8_heads* q, const w4a8_kv_cache* cache, const w4a8_kv_batch* batch,
                              float scale, int32_t window, const w4a8_heads* out, void* workspace,
                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_INT8_H_ */
