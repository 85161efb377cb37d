// paged_attention.hip -- attention of one new token of every sequence over a paged cache of keys and
// values (bf16, int8 with a scale per token and head, or 8-bit floating point with a scale per block of tokens and head).
//
//   O[b][i] = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q_i . k_t - m),  m the running maximum
//
// One pass over the keys and values, which is all there is to move: the kernel is bound by memory.  48 sequences of up to
// 16384 tokens (8 heads of 128, 32 queries, 1.6 GB) take 270 us, 6.0 TB/s (a copy runs at 5.0; the matrix cores are busy for 8 %
// and the vector ALU for 14 % of the time); two of 99991 tokens in int8 (211 MB) take 49-50 us, 4.3 TB/s (vector ALU
// 44 %, for the conversions).  FP8 codes become bf16 two at a time in one instruction and a tile has one scale: the 48 sequences take
// 147 us (811 MB, 5.5 TB/s, vector ALU 39 %).  One frame of 1374 tokens (5.6 MB) takes 7.9 us: 5.0 for the parts' chain of loads (lengths,
// page table, keys) and 2.9 for the join.
// Every block finds its part from the lengths of all sequences, which tells from many short ones on: 256 sequences of 1374 tokens
// (16 heads of 64) run at 6.1 TB/s, 1024 of 100 tokens (8 heads of 128, 32 queries) take 181 us, 2.4 TB/s, and 4096 of 64 tokens
// 1447 us, 0.8 TB/s.
//
// A wave takes two tiles of 16 tokens at a time and the up to 16 query heads that share a cache head, and nothing leaves its
// registers between the two products:
//   S^T = K q^T     lane (r = lane % 16, c = lane / 16) loads 16 bytes of token r's key as they lie in memory; it gets
//                   the scores of tokens 4 c + i (i < 4) for query r.
//   O^T += V^T P^T  over 32 tokens, slots 8 c + 4 u + i being token 4 c + i of tile u: so a lane's own scores are its operand,
//                   in three bf16 pieces that sum to them (two would leave up to 2^-15 of each, always of its sign, while the
//                   sum that divides the result takes it whole).  The other operand is value channel D / 16 r + e of the
//                   same tokens: each lane loads D / 16 neighbouring channels of four tokens a tile and picks channel e of a
//                   pair of tokens with one byte permutation.  The result has query r in lane (r, c), channels 4 D / 16 c onwards, next
//                   to that query's maximum and sum.
// Both are v_mfma_f32_16x16x32_bf16.  The order of channels inside S and of tokens inside O is free, which is what makes the
// loads contiguous and saves any exchange between lanes.  (v_mfma_f32_16x16x4_f32 takes P unrounded and needs no pieces, but
// four times the matrix time: long int8 86 against 74 us when it was tried, large batch 300 against 278.)
// With one query to a head its probabilities stand in all 16 columns, so that every lane has those of its tokens, and the
// second product is D / 16 fp32 multiply-adds a token.
// The next unit's keys are loaded as soon as this one's scores are formed, its values as soon as this one's sum is.
//
// A row without tokens is one whose sum is zero: fmaxf passes over a score that is NaN, exp2 makes it a probability of NaN, and
// sum and result are NaN as well.
//
// The tokens of all sequences together are cut into parts of equal size, one round of the blocks that the chip holds at once,
// or more where each part still has kLongPart tokens; a second kernel joins a sequence's parts by their maxima and
// sums.  Measured with one, two and three rounds: ragged batch 60, 58, 61 us, long int8 48, 55, 59, 4 sequences up to
// 16384 in fp32 41, 42, 45, 64 of 1374 66, 83, 73; with 768 blocks whatever the kernel 61, 49, 45, 66.  kLongPart of 768, 1536
// and 3072 tokens: long int8 60, 54, 54, large batch 279, 278, 293.
#include "paged_attention.h"

namespace qv {

hipError_t launch_paged_attention(const AttentionArgs& in, hipStream_t st) {
  bool split;
  const Args a = arguments(in, 1, &split);
  return launch<false>(a, in.cache.head_dim, in.bf16, in.cache.dtype, split, st);
}

}  // namespace qv
