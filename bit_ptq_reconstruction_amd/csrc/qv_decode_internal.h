// qv_decode_internal.h -- launchers of the single-token kernels, shared between their translation
// units and the C ABI layer (qv_decode_abi.cpp), which validates every argument before calling one.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qv_decode.h"

namespace qv {

// Few rows times int4 weights.  rotate: rows are rotated (Hadamard width K in {1024, 4096}) and
// multiplied by mult[k] (NULL = 1) first; `rows32` is then scratch for M * K floats.
hipError_t launch_w4a16(const void* X, bool x_bf16, int64_t M, int64_t K, int64_t ldx, bool rotate, const float* mult,
                        const uint8_t* Wq, const float* ws, int64_t group, const float* bias, int64_t N, bool gelu,
                        void* Y, bool y_bf16, int64_t ldy, float* rows32, hipStream_t st);

// Whether two of the rows of D elements at t token_stride + h head_stride (t < T, h < H) share an element.
inline bool rows_overlap(int64_t T, int64_t token_stride, int64_t H, int64_t head_stride, int64_t D) {
  if (H > 1 && head_stride < D) return T > 0;
  if (T <= 1 || H < 1) return false;
  if (token_stride < D) return true;
  if (token_stride >= (H - 1) * head_stride + D || token_stride <= (head_stride - D) / (T - 1)) return false;  // nested
  for (int64_t h = 1; h < H; ++h) {  // the tokens on either side of head h of token 0
    const int64_t at = h * head_stride, before = at / token_stride, gap = at - before * token_stride;
    if ((before >= 1 && before < T && gap < D) || (before + 1 < T && token_stride - gap < D)) return true;
  }
  return false;
}

struct AppendArgs {
  qv_kv_cache cache;
  const int32_t* page_table;
  int64_t num_seqs, max_pages, ld_table;
  const int32_t *token_seq, *token_index;
  int64_t T;
  qv_heads K, V;
  bool bf16;
  const float *cos, *sin;
  int64_t places, axes;
  const int32_t* position;
  qv_heads Q, Q_out;
  int64_t q_heads;
};
hipError_t launch_kv_append(const AppendArgs& a, hipStream_t st);

struct AttentionArgs {
  qv_heads Q, O;
  bool bf16;
  int64_t B, q_heads;
  qv_kv_cache cache;
  const int32_t* page_table;
  int64_t max_pages, ld_table;
  const int32_t* lens;
  float scale;
  int64_t window;
  float* partial;  // scratch for the parts of split sequences
};
hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t st);

// How the batch's tokens are cut into parts of equal size: at most `many` parts of all sequences together, and one
// more of each that is not full; no sequence has more than its capacity holds.  Each part keeps head_dim + 2 floats
// for every query head.
constexpr int64_t kQueriesPerBlock = 16;    // query heads of one cache head that a block takes
constexpr int64_t kMinTokensPerPart = 128;  // a unit of work for each wave of a block
constexpr int64_t kLongPart = 1536;         // tokens from which a block's start no longer counts
constexpr int64_t kManyBlocks = 4096;       // no less than a round of them
constexpr int64_t kTokensPerTile = 16;
// Tiles of a part where all sequences together have `total`: one round of blocks (`few` parts), or more of them where each
// still has a long part (uneven lengths and starts even out), `many` at most.  No sequence has more than 2^27 tiles.
template <typename U>
constexpr int tiles_of_part(U total, U few, U many) {
  const U each = (total + few - 1) / few, at_most = (total + many - 1) / many;
  const U least = kMinTokensPerPart / kTokensPerTile, enough = kLongPart / kTokensPerTile, all = U{1} << 27;
  const U more = at_most > enough ? at_most : enough;
  const U per = each < more ? each : more;
  return (int)(per < least ? least : (per > all ? all : per));
}
struct AttentionParts {
  int64_t many, most;
  int64_t blocks;  // of a part
  bool split;  // whether a sequence can have more than one
};
inline AttentionParts paged_attention_parts(int64_t B, int64_t q_heads, int64_t heads, int64_t capacity) {
  AttentionParts p;
  p.blocks = heads * ((q_heads / heads + kQueriesPerBlock - 1) / kQueriesPerBlock);
  p.many = (kManyBlocks + p.blocks - 1) / p.blocks;
  p.split = capacity > kMinTokensPerPart;
  const int64_t full = (capacity + kMinTokensPerPart - 1) / kMinTokensPerPart;
  p.most = !p.split ? B : (B * full < p.many + B ? B * full : p.many + B);
  return p;
}

}  // namespace qv
