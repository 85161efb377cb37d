// qv_runs_abi.cpp -- the C ABI of the entry points for runs of tokens (declared in include/qv_runs.h): host-side argument
// checks, then the kernel launches on the caller's stream.  Every check runs before the first HIP call, so a rejected call
// launches nothing and touches no device state.
#include "qv_runs.h"

#include <cmath>

#include "qv_decode_checks.h"
#include "qv_runs_internal.h"

namespace {

// Whether a batch's sizes are ones that the kernels take.
bool run_sizes(int64_t T, int64_t B, int64_t max_run, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t capacity) {
  if (T < 0 || T > kMaxInt || B < 0 || max_run < 0 || max_run > T || heads <= 0 || heads > 65536 || q_heads <= 0 ||
      q_heads > 65536 || q_heads % heads != 0 || (head_dim != 64 && head_dim != 128) || capacity < 0 ||
      capacity > kMaxInt - qv::kTokensPerStep)  // the end of a step is counted in 31 bits
    return false;
  if (max_run == 0) max_run = 1;
  if (B > kMaxInt / q_heads || B * q_heads > kMaxInt / max_run) return false;
  if (B > 0 && qv::long_runs(max_run, q_heads, heads, false)) {  // 256 threads to a block, 32 to a row's join
    const qv::RunTiles t = qv::run_tiles(T, B, q_heads, heads, capacity);
    if (T > kMaxInt / q_heads / 32 || t.items * t.parts > kMaxThreads / 256 / heads) return false;
  }
  if (qv::long_runs(max_run, q_heads, heads, true)) return true;
  qv::AttentionParts p = qv::paged_attention_parts(B, q_heads * max_run, heads, capacity);
  p.most += 8;  // the blocks of a tile of rows are rounded up to eight
  return attention_fits(B, q_heads * max_run, p);
}

}  // namespace

extern "C" {

qv_status qv_page_tables(const int32_t* runs, const int32_t* lens, int64_t B, int64_t page_size, const int32_t* free_pages,
                         int64_t num_free, const int32_t* free_count, int32_t* page_table, int64_t max_pages,
                         int64_t ld_table, int32_t* starts, int32_t* lens_out, int32_t* free_left, int32_t* token_seq,
                         int32_t* token_index, int64_t* slots, int64_t T, int32_t* status, void* hip_stream) {
  try {
    if (B < 0 || T < 0 || num_free < 0 || page_size <= 0 || max_pages < 0 || ld_table < max_pages || ld_table > kMaxDim)
      return QV_ERR_SHAPE;
    if (B > kMaxInt || T > kMaxInt || num_free > kMaxInt || page_size > kMaxInt || max_pages > kMaxInt / page_size)
      return QV_ERR_UNSUPPORTED;
    if (!free_count || !starts || !free_left || (B > 0 && (!runs || !lens || !lens_out || !status)) ||
        (B > 0 && max_pages > 0 && !page_table) || (num_free > 0 && !free_pages) ||
        (T > 0 && (!token_seq || !token_index || !slots)))
      return QV_ERR_NULL;
    const void* words[] = {runs, lens, free_pages, free_count, page_table, starts, lens_out, free_left, token_seq, token_index,
                           status};
    for (const void* p : words)
      if (!aligned(p, 4)) return QV_ERR_ALIGN;
    if (!aligned(slots, 8)) return QV_ERR_ALIGN;
    qv::TablesArgs a = {runs,   lens,     B,         page_size, free_pages,  num_free, free_count, page_table, max_pages, ld_table,
                        starts, lens_out, free_left, token_seq, token_index, slots,    T,          status};
    return hip_status(qv::launch_page_tables(a, static_cast<hipStream_t>(hip_stream)));
  } catch (...) {
    return QV_ERR_INTERNAL;
  }
}

size_t qv_run_attention_workspace_size(int64_t T, int64_t B, int64_t max_run, int64_t q_heads, int64_t heads,
                                       int64_t head_dim, int64_t capacity) {
  if (!run_sizes(T, B, max_run, q_heads, heads, head_dim, capacity)) return 0;
  return round256(static_cast<size_t>(qv::run_attention_bytes(T, B, max_run, q_heads, heads, head_dim, capacity)) + 1);
}

qv_status qv_run_attention(const qv_heads* Q, qv_dtype q_dtype, int64_t T, int64_t q_heads, const int32_t* starts, int64_t B,
                           int64_t max_run, const qv_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                           int64_t ld_table, const int32_t* lens, float scale, int64_t window, int64_t sinks, int32_t causal,
                           const qv_heads* O, void* workspace, size_t workspace_bytes, void* hip_stream) {
  try {
    qv_status st = check_cache(cache);
    if (st != QV_OK) return st;
    if (!valid_dtype(q_dtype)) return QV_ERR_DTYPE;
    st = check_table(page_table, B, max_pages, ld_table, cache);
    if (st != QV_OK) return st;
    if (T < 0 || q_heads <= 0 || q_heads > 65536 || q_heads % cache->heads != 0 || window < 0 || sinks < 0 || max_run < 0 ||
        max_run > T || !std::isfinite(scale))
      return QV_ERR_SHAPE;
    if (!starts && (T != B || max_run > 1)) return QV_ERR_SHAPE;
    const int64_t capacity = max_pages * cache->page_size;
    if (!run_sizes(T, B, max_run, q_heads, cache->heads, cache->head_dim, capacity)) return QV_ERR_UNSUPPORTED;
    if (T == 0 || B == 0 || max_run == 0) return QV_OK;
    if (!Q || !O || !lens) return QV_ERR_NULL;
    if (!aligned(lens, 4) || !aligned(starts, 4)) return QV_ERR_ALIGN;
    const qv_heads* rows[] = {Q, O};
    for (const qv_heads* h : rows) {
      st = check_heads(h, q_dtype, cache->head_dim);
      if (st != QV_OK) return st;
    }
    st = check_output(O, T, q_heads, cache->head_dim);
    if (st != QV_OK) return st;
    if (!workspace ||
        workspace_bytes < qv_run_attention_workspace_size(T, B, max_run, q_heads, cache->heads, cache->head_dim, capacity))
      return QV_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return QV_ERR_ALIGN;
    qv::RunArgs a = {};
    a.base.Q = *Q;
    a.base.O = *O;
    a.base.bf16 = q_dtype == QV_BF16;
    a.base.B = B;
    a.base.q_heads = q_heads;
    a.base.cache = *cache;
    a.base.page_table = page_table;
    a.base.max_pages = max_pages;
    a.base.ld_table = ld_table;
    a.base.lens = lens;
    a.base.scale = scale;
    a.base.window = window;
    a.base.partial = static_cast<float*>(workspace);
    a.starts = starts;
    a.T = T;
    a.max_run = max_run;
    a.sinks = sinks;
    a.causal = causal != 0;
    return hip_status(qv::launch_run_attention(a, static_cast<hipStream_t>(hip_stream)));
  } catch (...) {
    return QV_ERR_INTERNAL;
  }
}

}  // extern "C"
