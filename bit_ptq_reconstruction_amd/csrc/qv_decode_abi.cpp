// qv_decode_abi.cpp -- the C ABI of the single-token entry points (declared in include/qv_decode.h):
// host-side argument checks, then the kernel launches on the caller's stream.  Every check runs
// before the first HIP call, so a rejected call launches nothing and touches no device state.
#include "qv_decode.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "qv_decode_checks.h"
#include "qv_decode_internal.h"

namespace {

constexpr int64_t kMaxChannels = kMaxThreads / 512 * 64;  // blocks of 512 threads and 64 channels

qv_status check_w4a16(const void* X, qv_dtype xt, int64_t M, int64_t K, int64_t ldx, const uint8_t* Wq,
                      const float* ws, int64_t group, const float* bias, int64_t N, qv_epilogue epi, const void* Y,
                      qv_dtype yt, int64_t ldy) {
  if (!valid_dtype(xt) || !valid_dtype(yt) || (epi != QV_EPI_NONE && epi != QV_EPI_GELU)) return QV_ERR_DTYPE;
  if (M < 0 || N < 0 || K <= 0) return QV_ERR_SHAPE;
  if ((K % 128) != 0 || K > 65536) return QV_ERR_UNSUPPORTED;
  if (group != K && ((group != 128 && group != 256 && group != 512) || (K % group) != 0)) return QV_ERR_UNSUPPORTED;
  if (ldx < K || ldy < N || ldx > kMaxDim || ldy > kMaxDim) return QV_ERR_SHAPE;
  if (M > kMaxInt || N > kMaxChannels) return QV_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return QV_OK;
  if (!X || !Wq || !ws || !Y) return QV_ERR_NULL;
  if (!aligned(X) || !aligned(Wq) || !aligned(ws) || !aligned(bias) || !aligned(Y) ||
      ((ldx * dtype_bytes(xt)) % 16) != 0)
    return QV_ERR_ALIGN;
  return QV_OK;
}

}  // namespace

extern "C" {

qv_status qv_w4a16_gemv(const void* X, qv_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t* Wq,
                        const float* w_scale, int64_t group, const float* bias, int64_t N, qv_epilogue epi, void* Y,
                        qv_dtype y_dtype, int64_t ldy, void* hip_stream) {
  try {
    qv_status st = check_w4a16(X, x_dtype, M, K, ldx, Wq, w_scale, group, bias, N, epi, Y, y_dtype, ldy);
    if (st != QV_OK || M == 0 || N == 0) return st;
    return hip_status(qv::launch_w4a16(X, x_dtype == QV_BF16, M, K, ldx, false, nullptr, Wq, w_scale, group, bias, N,
                                       epi == QV_EPI_GELU, Y, y_dtype == QV_BF16, ldy, nullptr,
                                       static_cast<hipStream_t>(hip_stream)));
  } catch (...) {
    return QV_ERR_INTERNAL;
  }
}

size_t qv_w4a16_linear_workspace_size(int64_t M, int64_t K) {
  if (M < 0 || K <= 0 || M > kMaxDim || K > kMaxDim / 4) return 0;
  if (M != 0 && K > (int64_t{1} << 60) / M) return 0;
  return round256(static_cast<size_t>(M) * static_cast<size_t>(K) * 4);
}

qv_status qv_w4a16_linear(const void* X, qv_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, const float* inv_smooth,
                          const uint8_t* Wq, const float* w_scale, int64_t group, const float* bias, int64_t N,
                          qv_epilogue epi, void* Y, qv_dtype y_dtype, int64_t ldy, void* workspace,
                          size_t workspace_bytes, void* hip_stream) {
  try {
    qv_status st = check_w4a16(X, x_dtype, M, K, ldx, Wq, w_scale, group, bias, N, epi, Y, y_dtype, ldy);
    if (st != QV_OK) return st;
    if (K != 1024 && K != 4096) return QV_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return QV_OK;
    if (!aligned(inv_smooth)) return QV_ERR_ALIGN;
    if (!workspace || workspace_bytes < qv_w4a16_linear_workspace_size(M, K)) return QV_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return QV_ERR_ALIGN;
    return hip_status(qv::launch_w4a16(X, x_dtype == QV_BF16, M, K, ldx, true, inv_smooth, Wq, w_scale, group, bias, N,
                                       epi == QV_EPI_GELU, Y, y_dtype == QV_BF16, ldy, static_cast<float*>(workspace),
                                       static_cast<hipStream_t>(hip_stream)));
  } catch (...) {
    return QV_ERR_INTERNAL;
  }
}

qv_status qv_kv_append(const qv_kv_cache* cache, const int32_t* page_table, int64_t num_seqs, int64_t max_pages,
                       int64_t ld_table, const int32_t* token_seq, const int32_t* token_index, int64_t T,
                       const qv_heads* K, const qv_heads* V, qv_dtype x_dtype, const float* cos, const float* sin,
                       int64_t places, int64_t axes, const int32_t* position, const qv_heads* Q, const qv_heads* Q_out,
                       int64_t q_heads, void* hip_stream) {
  try {
    qv_status st = check_cache(cache);
    if (st != QV_OK) return st;
    if (!valid_dtype(x_dtype)) return QV_ERR_DTYPE;
    st = check_table(page_table, num_seqs, max_pages, ld_table, cache);
    if (st != QV_OK) return st;
    if (T < 0 || q_heads < 0 || T > kMaxDim || q_heads > 65536) return QV_ERR_SHAPE;
    if (!token_seq && T > num_seqs) return QV_ERR_SHAPE;
    if (axes != 1 && axes != 2) return QV_ERR_UNSUPPORTED;
    if (places < 0 || places > kMaxInt) return QV_ERR_SHAPE;
    if (!cos != !sin) return QV_ERR_NULL;
    if ((Q == nullptr) != (Q_out == nullptr) || (Q == nullptr) != (q_heads == 0)) return QV_ERR_NULL;
    if (T == 0) return QV_OK;
    if (!K || !V || !token_index || (cos && !position && axes != 1)) return QV_ERR_NULL;
    if (!aligned(token_seq, 4) || !aligned(token_index, 4) || !aligned(position, 4) || !aligned(cos) || !aligned(sin))
      return QV_ERR_ALIGN;
    const qv_heads* rows[] = {K, V, Q, Q_out};
    for (const qv_heads* h : rows) {
      if (!h) continue;
      st = check_heads(h, x_dtype, cache->head_dim);
      if (st != QV_OK) return st;
    }
    if (Q_out) st = check_output(Q_out, T, q_heads, cache->head_dim);
    if (st != QV_OK) return st;
    qv::AppendArgs a = {};
    a.cache = *cache;
    a.page_table = page_table;
    a.num_seqs = num_seqs;
    a.max_pages = max_pages;
    a.ld_table = ld_table;
    a.token_seq = token_seq;
    a.token_index = token_index;
    a.T = T;
    a.K = *K;
    a.V = *V;
    a.bf16 = x_dtype == QV_BF16;
    a.cos = cos;
    a.sin = sin;
    a.places = places;
    a.axes = axes;
    a.position = position;
    if (Q) {
      a.Q = *Q;
      a.Q_out = *Q_out;
    }
    a.q_heads = q_heads;
    return hip_status(qv::launch_kv_append(a, static_cast<hipStream_t>(hip_stream)));
  } catch (...) {
    return QV_ERR_INTERNAL;
  }
}

size_t qv_paged_attention_workspace_size(int64_t B, int64_t q_heads, int64_t heads, int64_t head_dim,
                                         int64_t capacity) {
  if (B < 0 || heads <= 0 || heads > 65536 || q_heads <= 0 || q_heads > 65536 || q_heads % heads != 0 ||
      (head_dim != 64 && head_dim != 128) || capacity < 0 || capacity > kMaxInt || B > kMaxInt / q_heads)
    return 0;
  const qv::AttentionParts p = qv::paged_attention_parts(B, q_heads, heads, capacity);
  if (!attention_fits(B, q_heads, p)) return 0;
  if (!p.split) return 256;
  return round256(static_cast<size_t>(p.most * q_heads) * static_cast<size_t>(head_dim + 2) * 4 + 1);
}

qv_status qv_paged_attention(const qv_heads* Q, qv_dtype q_dtype, int64_t B, int64_t q_heads, const qv_kv_cache* cache,
                             const int32_t* page_table, int64_t max_pages, int64_t ld_table, const int32_t* lens,
                             float scale, int64_t window, const qv_heads* O, void* workspace, size_t workspace_bytes,
                             void* hip_stream) {
  try {
    qv_status st = check_cache(cache);
    if (st != QV_OK) return st;
    if (!valid_dtype(q_dtype)) return QV_ERR_DTYPE;
    st = check_table(page_table, B, max_pages, ld_table, cache);
    if (st != QV_OK) return st;
    if (q_heads <= 0 || q_heads > 65536 || q_heads % cache->heads != 0 || window < 0) return QV_ERR_SHAPE;
    if (B > kMaxInt / q_heads) return QV_ERR_UNSUPPORTED;
    if (!attention_fits(B, q_heads, qv::paged_attention_parts(B, q_heads, cache->heads, max_pages * cache->page_size)))
      return QV_ERR_UNSUPPORTED;
    if (B == 0) return QV_OK;
    if (!Q || !O || !lens) return QV_ERR_NULL;
    if (!aligned(lens, 4)) return QV_ERR_ALIGN;
    const qv_heads* rows[] = {Q, O};
    for (const qv_heads* h : rows) {
      st = check_heads(h, q_dtype, cache->head_dim);
      if (st != QV_OK) return st;
    }
    st = check_output(O, B, q_heads, cache->head_dim);
    if (st != QV_OK) return st;
    const size_t need =
        qv_paged_attention_workspace_size(B, q_heads, cache->heads, cache->head_dim, max_pages * cache->page_size);
    if (!workspace || need == 0 || workspace_bytes < need) return QV_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return QV_ERR_ALIGN;
    qv::AttentionArgs a = {};
    a.Q = *Q;
    a.O = *O;
    a.bf16 = q_dtype == QV_BF16;
    a.B = B;
    a.q_heads = q_heads;
    a.cache = *cache;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.ld_table = ld_table;
    a.lens = lens;
    a.scale = scale;
    a.window = window;
    a.partial = static_cast<float*>(workspace);
    return hip_status(qv::launch_paged_attention(a, static_cast<hipStream_t>(hip_stream)));
  } catch (...) {
    return QV_ERR_INTERNAL;
  }
}

}  // extern "C"
