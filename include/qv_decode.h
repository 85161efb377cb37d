/*
 * qv_decode.h -- C ABI of libqv for single tokens and short runs of them: what a block of the model
 * needs to take one new token (or a few rows) at a time, with the weights that qv.h's packing calls
 * prepare.
 *
 *   qv_w4a16_linear, qv_w4a16_gemv   few-row products with 4-bit weights; the activations keep their
 *                                    precision (the W4A4 GEMM of qv.h rounds them to 4 bits and
 *                                    works in tiles of 128 rows)
 *   qv_kv_append                     new keys and values into a paged cache, rotated by position
 *   qv_paged_attention               one new token of every sequence over that cache
 *
 * The conventions are those of qv.h: device pointers owned by the caller, asynchronous kernel launches
 * on hip_stream and nothing else (so calls record into a HIP graph), host-side checks before the
 * first HIP call, finite inputs, results that are the same from run to run, 16-byte aligned base
 * pointers.  Strides are in elements; where a row stride need not be a multiple of 16 bytes, the
 * entry point says so.
 */
#ifndef QV_DECODE_H
#define QV_DECODE_H

#include "qv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * qv_w4a16_gemv -- few rows of activations times 4-bit weights with group scales:
 *   Y[m][n] = sum_g w_scale[n][g] * (sum_{k in g} X[m][k] * Wq[n][k]) (+ bias[n]),  optionally GELU.
 * X is taken as it is (already rotated, or against weights that were never rotated).
 *   X        [M][ldx] fp32 or bf16; every M is accepted, and the kernel is made for M up to 16 or so.
 *   K        multiple of 128 in [128, 65536] (else QV_ERR_UNSUPPORTED).
 *   Wq       [N][K/2] packed int4 codes in the layout of qv.h;  N >= 1, any up to 2^29 - 64.
 *   group    128, 256 or 512 dividing K, or K itself (one scale per output channel).
 *   w_scale  [N][K / group] fp32 (qv_pack_weights_grouped; with group = K: qv_pack_weights).
 *   bias     [N] fp32 or NULL.   epi  QV_EPI_NONE or QV_EPI_GELU (0.5 y erfc(-y / sqrt 2)).
 *   Y        [M][ldy] fp32 or bf16, rounded once, to nearest even; ldy >= N, any (rows need no alignment).
 * Every product of an activation and a code is exact (an fp32 or rotated activation is split into three bf16
 * pieces that sum to it), sums are fp32.
 */
qv_status qv_w4a16_gemv(const void* X, qv_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t* Wq,
                        const float* w_scale, int64_t group, const float* bias, int64_t N, qv_epilogue epi, void* Y,
                        qv_dtype y_dtype, int64_t ldy, void* hip_stream);

/* Bytes of workspace qv_w4a16_linear needs: the rotated rows in fp32, rounded up to 256 bytes (0 for
 * invalid sizes). */
size_t qv_w4a16_linear_workspace_size(int64_t M, int64_t K);

/*
 * qv_w4a16_linear -- the online layer with 4-bit weights and unquantized activations: the rows are
 * rotated and smoothed in fp32 as in qv_hadamard_smooth_quant and multiplied as in qv_w4a16_gemv.
 *   K           1024 or 4096.   inv_smooth  [K] fp32, NULL = ones.
 *   workspace   at least qv_w4a16_linear_workspace_size(M, K) bytes, 256-byte aligned, reused freely.
 */
qv_status qv_w4a16_linear(const void* X, qv_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, const float* inv_smooth,
                          const uint8_t* Wq, const float* w_scale, int64_t group, const float* bias, int64_t N,
                          qv_epilogue epi, void* Y, qv_dtype y_dtype, int64_t ldy, void* workspace,
                          size_t workspace_bytes, void* hip_stream);

typedef enum { QV_KV_BF16 = 0, QV_KV_INT8 = 1 } qv_kv_dtype;

/*
 * A paged cache of keys and values: num_pages pages of page_size tokens for each of `heads` heads.
 * Element (page p, head h, slot t, channel d) of either is at p page_stride + h head_stride +
 * t token_stride + d, so [page][head][slot][d] and [page][slot][head][d] both fit.
 *   head_dim 64 or 128;  page_size a multiple of 16 (up to 65536).
 *   QV_KV_BF16: bf16 values;  k_scale and v_scale are not used.
 *   QV_KV_INT8: int8 codes with one fp32 scale per token and head, k_scale / v_scale
 *               [num_pages][heads][page_size] dense; the value is code * scale, scale = max |x| / 127.
 * Strides are positive multiples of 16 bytes (below 2^24 elements for token_stride, 2^31 for the others).
 */
typedef struct {
  void* k_pages;
  void* v_pages;
  float* k_scale;
  float* v_scale;
  int64_t num_pages;
  int64_t heads;
  int64_t page_size;
  int64_t head_dim;
  int64_t page_stride;
  int64_t head_stride;
  int64_t token_stride;
  int32_t dtype; /* qv_kv_dtype */
} qv_kv_cache;

/* Input rows [T][heads][head_dim] with unit channel stride: token t, head h at t token_stride +
 * h head_stride (a slice of a packed qkv tensor fits).  16-byte aligned, strides multiples of 16 bytes; rows that are
 * written must not overlap (QV_ERR_SHAPE). */
typedef struct {
  const void* data;
  int64_t token_stride;
  int64_t head_stride;
} qv_heads;

/*
 * qv_kv_append -- keys and values of T new tokens into the cache, K (and Q) rotated by position on
 * the way; single tokens and prompts alike.
 *   page_table  [num_seqs][ld_table] int32: page of tokens [p page_size, (p + 1) page_size) of a sequence;
 *               ld_table >= max_pages, any.
 *   token_seq   [T] int32 sequence of each token, or NULL: token t is sequence t (then T <= num_seqs).
 *   token_index [T] int32 place of each token in its sequence (the number of tokens before it).
 *               A token whose sequence, place or page lies outside the table or the cache is not stored.
 *               No two tokens of a call may have the same place.
 *   K, V        [T][heads][head_dim] of x_dtype (fp32 or bf16).
 *   cos, sin    [places][head_dim / (2 axes)] fp32 tables, or both NULL for no rotation.  The head_dim
 *               channels are `axes` (1 or 2) blocks of w = head_dim / axes; axis a turns the pairs
 *               (x[j], x[j + w/2]) of its block by the angle of row position[t][a]:
 *                 x'[j] = x[j] cos - x[j + w/2] sin,   x'[j + w/2] = x[j + w/2] cos + x[j] sin
 *               in fp32, every product and sum rounded by itself.
 *   position    [T][axes] int32, or NULL with axes = 1: token_index.  A token with a position outside
 *               [0, places) is not stored, and its rows of Q_out are NaN.
 *   Q, Q_out    [T][q_heads][head_dim] of x_dtype, rotated in the same way, or both NULL (q_heads = 0).
 *               Q_out may be Q itself with the same strides.
 * bf16 caches round the rotated value once, to nearest even.  int8 caches take the scale of each
 * (token, head) from its rotated fp32 values: scale = max |x| / 127, code = clamp(rne(x / scale), -128,
 * 127), both quotients correctly rounded; a zero or subnormal scale becomes 0 with zero codes, and a row that
 * is not finite gets a scale of NaN with zero codes.
 */
qv_status qv_kv_append(const qv_kv_cache* cache, const int32_t* page_table, int64_t num_seqs, int64_t max_pages,
                       int64_t ld_table, const int32_t* token_seq, const int32_t* token_index, int64_t T,
                       const qv_heads* K, const qv_heads* V, qv_dtype x_dtype, const float* cos, const float* sin,
                       int64_t places, int64_t axes, const int32_t* position, const qv_heads* Q, const qv_heads* Q_out,
                       int64_t q_heads, void* hip_stream);

/* Bytes of workspace qv_paged_attention needs for B sequences whose page table holds up to `capacity`
 * tokens each (max_pages * page_size): the partial results of the split length, rounded up to 256
 * bytes and at least 256 (0 for invalid sizes). */
size_t qv_paged_attention_workspace_size(int64_t B, int64_t q_heads, int64_t heads, int64_t head_dim,
                                         int64_t capacity);

/*
 * qv_paged_attention -- attention of one new token of each of B sequences over the paged cache:
 *   O[b][i] = sum_t softmax_t(scale Q[b][i] . k[t][i / (q_heads / heads)]) v[t][i / (q_heads / heads)]
 * over the tokens max(0, lens[b] - window) <= t < lens[b] (window = 0: all of them).
 *   Q           [B][q_heads][head_dim] fp32 or bf16;  q_heads a multiple of the cache's heads.  B times the blocks
 *               of a sequence (one for up to 16 query heads of a cache head) is below 2^24, B q_heads below 2^25 (else
 *               QV_ERR_UNSUPPORTED).
 *   page_table  as for qv_kv_append, B rows.  Tokens on a page outside [0, num_pages) do not take part
 *               (a page may be given back once a window has left it behind).
 *   lens        [B] int32 tokens of each sequence, the new one included; cut to [0, max_pages * page_size].
 *               A sequence with no token gives zeros.  What the cache holds behind them is not used.  A query of NaN
 *               (qv_kv_append makes them), or a NaN among the tokens, gives NaN.
 *   O           [B][q_heads][head_dim] of Q's type.  Scores, softmax and sums are fp32; probabilities are
 *               not rounded, and an fp32 query is taken as three bf16 pieces that sum to it.
 *   workspace   at least qv_paged_attention_workspace_size(B, q_heads, heads, head_dim, max_pages *
 *               page_size) bytes, 256-byte aligned, reused freely.
 */
qv_status qv_paged_attention(const qv_heads* Q, qv_dtype q_dtype, int64_t B, int64_t q_heads, const qv_kv_cache* cache,
                             const int32_t* page_table, int64_t max_pages, int64_t ld_table, const int32_t* lens,
                             float scale, int64_t window, const qv_heads* O, void* workspace, size_t workspace_bytes,
                             void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* QV_DECODE_H */
