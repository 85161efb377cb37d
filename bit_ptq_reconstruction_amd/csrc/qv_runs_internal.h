// qv_runs_internal.h -- launchers of the kernels for runs of tokens, shared between their translation units and the C ABI
// layer (qv_runs_abi.cpp), which validates every argument before calling one.
#pragma once
#include "qv_decode_internal.h"
#include "qv_runs.h"

namespace qv {

struct TablesArgs {
  const int32_t *runs, *lens;
  int64_t B, page_size;
  const int32_t* free_pages;
  int64_t num_free;
  const int32_t* free_count;
  int32_t* page_table;
  int64_t max_pages, ld_table;
  int32_t *starts, *lens_out, *free_left, *token_seq, *token_index;
  int64_t* slots;
  int64_t T;
  int32_t* status;
};
hipError_t launch_page_tables(const TablesArgs& a, hipStream_t st);

struct RunArgs {
  AttentionArgs base;  // B sequences; Q and O have T rows
  const int32_t* starts;
  int64_t T, max_run, sinks;
  bool causal;
};
hipError_t launch_run_attention(const RunArgs& a, hipStream_t st);
hipError_t launch_run_tiles(const RunArgs& a, hipStream_t st);  // run_tiles.hip; with starts

// Long runs go in tiles of rows, up to kRowsPerTile (query heads that share a cache head, for each token) and kTokensPerStep
// tokens at a time.
constexpr int64_t kRowsPerTile = 128, kTokensPerStep = 64;
constexpr int64_t kLeastSteps = 4;   // of a part
constexpr int64_t kMostParts = 64;
constexpr int64_t kTileCUs = 256;
struct RunTiles {
  int64_t items, parts;
};
// Tiles of rows, and into how many parts the tokens that one sees are cut.  A CU works on its blocks side by side and is well used
// with two or more, so a call takes about (blocks of the CU that has most) x (steps of a block and its start), half as much again where
// that is one block; each part costs the join as much as a step.  `seen`: tokens that a tile's rows see, at most; `room`: parts
// that the workspace holds.
// us with 1, 2, 3, 4, 5, 6, 8 and 12 parts, and as chosen: a frame over eight 205 137 143 120 134 129 126 134, 120; a chunk of two prompts
// over 4001 in FP8 164 114 114 101 98 111 108 122, 101; 8 heads of 128 with 32 queries, 256 tokens over 100000 2590 1310 882 685 740 660
// 581 637, 616, eight chunks of 128 over 4000 157 118 125 126 131 134 154 178, 125, one prompt of 2048 75 85 97 109 105 113 127 126, 75.
inline RunTiles run_tiles(int64_t T, int64_t B, int64_t q_heads, int64_t heads, int64_t seen, int64_t room = kMostParts) {
  RunTiles t;
  t.items = T * (q_heads / heads) / kRowsPerTile + B;
  t.parts = 1;
  const int64_t steps = seen / kTokensPerStep + 1, blocks = t.items * heads, most = steps / kLeastSteps;
  int64_t best = 0;
  for (int64_t p = 1; p <= room && p <= most && (p == 1 || blocks * (p - 1) < 8 * kTileCUs); ++p) {
    const int64_t on_a_cu = (blocks * p + kTileCUs - 1) / kTileCUs, each = (uint32_t)(steps + p - 1) / (uint32_t)p + 6;
    const int64_t cost = 2 * on_a_cu * each + (on_a_cu == 1 ? each : 0) + (p > 1 ? 2 * p + 12 : 0);
    if (p == 1 || cost < best) best = cost, t.parts = p;
  }
  return t;
}

// Tokens that the rows of a tile see, at most: their windows, which begin up to a tile's rows apart, and the first tokens; all of the
// run behind them where it is not causal.
inline int64_t tokens_of_tile(int64_t capacity, int64_t max_run, int64_t window, int64_t sinks, bool causal) {
  if (window == 0 || window >= capacity) return capacity;
  const int64_t seen = window + (causal ? kRowsPerTile : max_run) + (sinks < capacity ? sinks : capacity);
  return seen < capacity ? seen : capacity;
}

// Whether a call goes that way.  us, few-row kernel and tiles, over bf16: 16 runs of 5 tokens of 4 query heads over up to 8192 41 and 48,
// 32 of 8 over 4096 88 and 79, 64 of 10 over 2000 129 and 77, four of 40 (16 heads of 64) over 4000 30 and 28; over 8-bit caches, which
// the tiles convert ahead of their products, 32 to 34 and 59 to 62, 69 to 74 and 93 to 97, 98 to 109 and 96 to 102, 27 to 28 and 34 to 35.
// Heads, sequences and past are not in the rule: one run of 48, 64 or 128 tokens over 30000 with two heads gives the tiles few blocks and
// takes 23, 25 and 36 against 49 to 50 over bf16, 21 to 23, 24 to 26 and 31 to 35 against 58 to 62 over 8-bit caches.
inline bool long_runs(int64_t max_run, int64_t q_heads, int64_t heads, bool bytes) {
  return max_run > 1 && max_run * (q_heads / heads) > (bytes ? QV_RUN_FEW_ROWS_8BIT : QV_RUN_FEW_ROWS);
}

// Bytes of partial results that the launch may write, whatever the cache holds.
inline int64_t run_attention_bytes(int64_t T, int64_t B, int64_t max_run, int64_t q_heads, int64_t heads, int64_t head_dim,
                                   int64_t capacity) {
  if (max_run == 0 || B == 0) return 0;
  int64_t rows = 0;
  if (long_runs(max_run, q_heads, heads, false)) {
    const RunTiles t = run_tiles(T, B, q_heads, heads, capacity);
    if (t.parts > 1) rows = t.parts * T * q_heads;
  }
  if (!long_runs(max_run, q_heads, heads, true)) {
    const AttentionParts p = paged_attention_parts(B, q_heads * max_run, heads, capacity);
    if (p.split && p.most * q_heads * max_run > rows) rows = p.most * q_heads * max_run;
  }
  return rows * (head_dim + 2) * 4;
}

}  // namespace qv
