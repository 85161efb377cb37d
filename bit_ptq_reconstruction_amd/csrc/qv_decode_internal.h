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
  float* partial;  // scratch of paged_attention_splits() > 1
};
hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t st);

// Parts that the length is split into at most: enough for the partial results to fill the chip.
// Each part keeps head_dim + 2 floats for every query head.
constexpr int64_t kQueriesPerBlock = 16;   // query heads of one cache head that a block takes
constexpr int64_t kMinTokensPerPart = 256;  // a shorter part costs more in the join than it saves
constexpr int64_t kPartsWanted = 2048;      // 256 CUs x 8 blocks
inline int64_t paged_attention_splits(int64_t B, int64_t q_heads, int64_t heads, int64_t capacity) {
  const int64_t tiles = (q_heads / heads + kQueriesPerBlock - 1) / kQueriesPerBlock;
  const int64_t blocks = B * heads * tiles;
  int64_t n = blocks > 0 ? (kPartsWanted + blocks - 1) / blocks : 1;
  const int64_t most = (capacity + kMinTokensPerPart - 1) / kMinTokensPerPart;
  if (n > most) n = most;
  return n < 1 ? 1 : n;
}

}  // namespace qv
