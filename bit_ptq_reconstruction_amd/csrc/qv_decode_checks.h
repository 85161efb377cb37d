// qv_decode_checks.h -- host-side argument checks that the ABI layers of the single-token entry points and of those for
// runs of tokens share.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "qv_decode.h"
#include "qv_decode_internal.h"

namespace {

constexpr int64_t kMaxDim = int64_t{1} << 40;   // as in qv_abi.cpp: byte counts stay inside int64
constexpr int64_t kMaxInt = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1;  // of a launch, along one dimension

inline bool aligned(const void* p, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(p) % to) == 0; }

inline int64_t dtype_bytes(qv_dtype t) { return t == QV_BF16 ? 2 : 4; }

inline bool valid_dtype(qv_dtype t) { return t == QV_F32 || t == QV_BF16; }

inline size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

inline qv_status hip_status(hipError_t e) { return e == hipSuccess ? QV_OK : QV_ERR_HIP; }

inline qv_status check_cache(const qv_kv_cache* c) {
  if (!c) return QV_ERR_NULL;
  if (c->dtype != QV_KV_BF16 && c->dtype != QV_KV_INT8 && (c->dtype != QV_KV_FP8 || c->scale_tokens == 0))
    return QV_ERR_DTYPE;
  if (c->num_pages < 0 || c->heads <= 0 || c->page_size <= 0 || c->head_dim <= 0) return QV_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return QV_ERR_UNSUPPORTED;
  if (c->page_size % 16 != 0 || c->page_size > 65536 || c->num_pages > kMaxInt || c->heads > 65536)
    return QV_ERR_UNSUPPORTED;
  if (c->dtype == QV_KV_FP8 && (c->scale_tokens < 0 || c->scale_tokens % 16 != 0 || c->page_size % c->scale_tokens != 0))
    return QV_ERR_UNSUPPORTED;
  if (c->page_stride < c->head_dim || c->head_stride < c->head_dim || c->token_stride < c->head_dim ||
      c->page_stride > kMaxInt || c->head_stride > kMaxInt || c->token_stride >= (int64_t{1} << 24))
    return QV_ERR_SHAPE;
  if (c->num_pages == 0) return QV_OK;
  if (!c->k_pages || !c->v_pages) return QV_ERR_NULL;
  const bool scaled = c->dtype != QV_KV_BF16;
  if (scaled && (!c->k_scale || !c->v_scale)) return QV_ERR_NULL;
  const int64_t e = scaled ? 1 : 2;
  if (!aligned(c->k_pages) || !aligned(c->v_pages) || (c->page_stride * e) % 16 != 0 ||
      (c->head_stride * e) % 16 != 0 || (c->token_stride * e) % 16 != 0)
    return QV_ERR_ALIGN;
  if (scaled && (!aligned(c->k_scale) || !aligned(c->v_scale))) return QV_ERR_ALIGN;
  return QV_OK;
}

// Rows [T][heads][D].  One token or one head needs no stride of its own.
inline qv_status check_heads(const qv_heads* h, qv_dtype t, int64_t D) {
  if (!h->data) return QV_ERR_NULL;
  if (h->token_stride < 0 || h->head_stride < D || h->token_stride > kMaxDim || h->head_stride > kMaxInt)
    return QV_ERR_SHAPE;
  if (!aligned(h->data) || (h->token_stride * dtype_bytes(t)) % 16 != 0 || (h->head_stride * dtype_bytes(t)) % 16 != 0)
    return QV_ERR_ALIGN;
  return QV_OK;
}

// Rows that are written: no two of them share memory.
inline qv_status check_output(const qv_heads* h, int64_t T, int64_t H, int64_t D) {
  return qv::rows_overlap(T, h->token_stride, H, h->head_stride, D) ? QV_ERR_SHAPE : QV_OK;
}

// Whether the attention's launches hold the batch: 256 threads to a part of a sequence, at least 128 to a query head's join.
inline bool attention_fits(int64_t B, int64_t q_heads, const qv::AttentionParts& p) {
  return p.most * p.blocks <= kMaxThreads / 256 && (!p.split || B * q_heads <= kMaxThreads / 128);
}

inline qv_status check_table(const int32_t* table, int64_t rows, int64_t max_pages, int64_t ld, const qv_kv_cache* c) {
  if (rows < 0 || max_pages < 0 || ld < max_pages || ld > kMaxDim) return QV_ERR_SHAPE;
  // places are counted in 32 bits
  if (rows > kMaxInt || max_pages > kMaxInt / c->page_size) return QV_ERR_UNSUPPORTED;
  if (rows > 0 && max_pages > 0) {
    if (!table) return QV_ERR_NULL;
    if (!aligned(table, 4)) return QV_ERR_ALIGN;
  }
  return QV_OK;
}

}  // namespace
