// run_attention.hip -- attention of short runs of tokens (and of single ones that keep first tokens in sight) over a paged
// cache: the kernels of paged_attention.h with the rows of a run in the place of a token's query heads.
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
