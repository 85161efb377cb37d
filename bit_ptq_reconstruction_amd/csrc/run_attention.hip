// run_attention.hip -- attention of short runs of tokens (and of single ones that keep first tokens in sight) over a paged
// cache: the kernels of paged_attention.h with the rows of a run in the place of a token's query heads.
//
// Bound by memory where a run has up to 16 rows to a cache head: one token of each of 32 sequences with a window of 4096 and four
// first tokens (513 MB) takes 108 + 5 us, 4.5 TB/s.  More rows go in tiles of 16, each of which reads and converts the tokens again: 16
// runs of 5 tokens of 4 query heads over up to 8192 in int8 (62 MB) 26 + 5 us.  Their blocks follow each other on one die,
// whose cache then has what the first one read: bf16 38 us instead of 49, int8 32 instead of 35.
#include "paged_attention.h"
#include "qv_runs_internal.h"

namespace qv {

hipError_t launch_run_attention(const RunArgs& in, hipStream_t st) {
  if (long_runs(in.max_run, in.base.q_heads, in.base.cache.heads, in.base.cache.dtype != QV_KV_BF16)) return launch_run_tiles(in, st);
  if (!in.starts && in.sinks == 0) return launch_paged_attention(in.base, st);  // a single token sees no token behind itself
  bool split;
  Args a = arguments(in.base, in.max_run, &split);
  a.starts = in.starts;
  a.T = (int32_t)in.T;
  a.sinks = in.sinks > 0x7fffffff ? 0x7fffffff : (int32_t)in.sinks;
  a.causal = in.causal;
  return launch<true>(a, in.base.cache.head_dim, in.base.bf16, in.base.cache.dtype, split, st);
}

}  // namespace qv
