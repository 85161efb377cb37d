// run_tiles.hip -- attention of long runs of tokens (prompts, frames, chunks) over a paged cache.
//
//   O[s] = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q_s . k_t - m_s),  m_s a running maximum,  t what row s sees
//
// A block takes 128 rows of one cache head (a run's tokens and, within each, the query heads that share the cache head) and
// passes once over the tokens that any of them sees, 64 at a time; each of its four waves has 32 of the rows and all tokens:
//   S^T = K Q^T     32 tokens x 32 rows a matrix instruction; a lane has one row and half of the tokens, so that maximum and
//                   sum need one exchange between the halves of a wave.
//   O^T += V^T P^T  a lane's own probabilities are its operand: slot 8 h + j of 16 tokens (h = lane / 32) stands for token
//                   4 h + j (j < 4) or 4 h + j + 4, on both sides.  V is read from LDS transposed.
// Both are v_mfma_f32_32x32x16_bf16; queries stay in registers, and keys and values of the next step are on their way while one
// is worked on (two buffers, one barrier a step): bf16 straight to LDS, 8-bit codes by way of registers, converted once for the four
// waves.  In LDS a 16-byte piece of a token lies at its number xor some bits of the token's (key_xor, value_xor).
//
// bf16 queries: a probability is two bf16 pieces for the second product, each to the nearest, which leave 2^-17 of it at most and of
// either sign, of the order of its score's fp32 rounding; their sum is of the whole ones.  One piece, with two thirds of
// the matrix instructions, leaves 2^-8 and a result that is 2.1 to 2.3e-3 off in the 2-norm where its own rounding makes 1.6 to
// 1.7e-3 (us with one piece and with two: frame over eight 89 and 116 to 119, chunk in FP8 91 and 102, prompts of up to 8192 982 and 1350 to 1390).
// fp32 queries and their probabilities are three bf16 pieces that sum to them.
// The maximum that scales a row's probabilities is raised only when one passes 2^8 of it: sums are fp32, and the rest follows.
//
// Bound by the matrix cores and the vector ALU (32 exponentials, 32 multiply-adds, 32 sums and the pieces of 32 probabilities of a lane
// to 48 matrix instructions of 128 channels) together: four prompts of up to 8192 tokens (8 heads of 128, 32 queries, causal) take 1.35
// to 1.39 ms, 0.72 to 0.74 PFLOP/s with each product counted once and 1.08 to 1.12 as they are made, where a library product of 8192^3
// reaches 1.22; the matrix cores are busy for 54 % of the time, the vector ALU for 51 %.  A frame of 1374 tokens over eight (16 heads of
// 64) takes 116 to 119 us with its join, 520 to 535 TFLOP/s: with 64 channels the vector ALU has twice as much to do for a matrix
// instruction (58 and 36 % busy).  A chunk of up to 611 tokens over 4001 of the FP8 cache takes 99 to 100 us (conversions, join), fp32
// prompts of up to 1833 tokens with a window of 1000 43 us (one wave a SIMD, 1100 waves of a dozen steps).
//
// Tried with one piece to a probability (us: frame over eight, prompts of 8192): staging bf16 by way of registers and masks in every step 179, 1505; steps whose
// way depends on masks only through a branch that changes scores 133, 1089; scalar addresses for the loads to LDS 140, 962 where it was
// 138, 1029; scores formed a step ahead, behind the product of the step before, 114, 1036 where it was 103, 984; matrix and vector
// instructions dealt out in turn by the scheduler 145, 1097 where it was 140, 1061; eight waves and 256 rows to a block 119, 988 where
// it was 100, 977; four waves a SIMD for 64 channels (registers spill) 123 where it was 103.
#include <type_traits>

#include "paged_attention.h"
#include "qv_runs_internal.h"

namespace qv {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = (int)kRowsPerTile, kN = (int)kTokensPerStep;  // of a block; tokens at a time
constexpr int kThreads = 256;
constexpr float kSlack = 8.0f;  // bits by which a probability may pass 1

struct TileArgs {
  Args a;
  int64_t items;       // tiles of rows, some of them empty
  uint32_t parts;      // of an item's tokens
  uint32_t least;      // steps of a part, at least
};

// Sequence and tile of rows of an item: a sequence's tiles begin at floor(its first row / 128) + its number, which leaves
// each as many as it needs whatever the starts are.
struct Item {
  int b, tile;
  Run run;
};
__device__ __forceinline__ int64_t first_item(const Args& a, int b) {
  int s = a.starts[b];
  s = s < 0 ? 0 : (s > a.T ? a.T : s);
  return (int64_t)s * a.share / kRows + b;
}
__device__ __forceinline__ Item item_of(const Args& a, int64_t number) {
  int low = 0, high = (int)a.B;
  while (high - low > 1) {
    const int mid = (low + high) / 2;
    if (first_item(a, mid) <= number) low = mid;
    else high = mid;
  }
  const int64_t tile = number - first_item(a, low);
  Item i = {low, -1, run_of(a, low)};
  if (tile >= 0 && tile * kRows < (int64_t)i.run.n * a.share) i.tile = (int)tile;
  return i;
}

// What the rows of a tile see: [0, sinks) and [low, high), in steps of 64 tokens without those between.
struct Steps {
  int len, low, high, sinks, near, skip, count;  // count: steps
  int all_low, all_high;                         // [all_low, all_high) is what every row sees
  int per, parts;                                // steps of a part; parts that have any
  __device__ __forceinline__ int first_token(int step) const { return (step < near ? step : step + skip) * kN; }
};
__device__ __forceinline__ Steps steps_of(const TileArgs& t, const Item& i) {
  const Args& a = t.a;
  Steps s;
  const int n = a.lens[i.b];
  s.len = n < 0 ? 0 : (n > a.capacity ? a.capacity : n);
  const int rows = i.run.n * (int)a.share, first = i.tile * kRows, last = first + kRows < rows ? first + kRows - 1 : rows - 1;
  const int64_t from = (int64_t)s.len - i.run.n + first / (int)a.share, to = (int64_t)s.len - i.run.n + last / (int)a.share;
  s.high = !a.causal ? s.len : (to + 1 < 0 ? 0 : (int)(to + 1));
  s.low = a.window > 0 && from >= a.window ? (int)(from - a.window + 1) : 0;
  s.all_high = !a.causal ? s.len : (from + 1 < 0 ? 0 : (int)(from + 1));
  s.all_low = a.window > 0 && to >= a.window ? (int)(to - a.window + 1) : 0;
  s.sinks = a.sinks < s.high ? a.sinks : s.high;
  s.near = (s.sinks + kN - 1) / kN;
  s.skip = s.low / kN > s.near ? s.low / kN - s.near : 0;
  s.count = (s.high + kN - 1) / kN - s.skip;
  if (s.count < 0) s.count = 0;
  s.per = (s.count + (int)t.parts - 1) / (int)t.parts;
  if (s.per < (int)t.least) s.per = (int)t.least;
  s.parts = s.count > s.per ? (s.count + s.per - 1) / s.per : 1;
  return s;
}

__device__ __forceinline__ unsigned pack(float x, float y) {  // to nearest even
  bf16x2 p;
  p[0] = (__bf16)x;
  p[1] = (__bf16)y;
  return __builtin_bit_cast(unsigned, p);
}

// The next bf16 pieces of two numbers, truncated, which leave the numbers.
__device__ __forceinline__ unsigned cut(float& x, float& y) {
  const unsigned w = __builtin_amdgcn_perm(float_bits(y), float_bits(x), 0x07060302u);
  x -= bits_float(float_bits(x) & 0xFFFF0000u);
  y -= bits_float(float_bits(y) & 0xFFFF0000u);
  return w;
}

// The nearest bf16 pieces of two numbers, which leave the numbers.
__device__ __forceinline__ unsigned cut_nearest(float& x, float& y) {
  const unsigned w = pack(x, y);
  x -= bits_float(w << 16);
  y -= bits_float(w & 0xFFFF0000u);
  return w;
}

__device__ __forceinline__ bool odd_pair(unsigned w) {  // an infinity or NaN among two bf16 values
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ unsigned even_pair(unsigned w) {  // zeros in their place
  w = (w & 0x7F80u) == 0x7F80u ? w & 0xFFFF0000u : w;
  return (w & 0x7F800000u) == 0x7F800000u ? w & 0xFFFFu : w;
}

// What the numbers of a token's 16-byte pieces are changed by in LDS: pieces of one number of 16 neighbouring keys, and pieces
// 4 i to 4 i + 3 of four neighbouring values, lie on different banks.
template <int D>
__device__ __forceinline__ int key_xor(int token) {
  return D == 128 ? token & 15 : token >> 1 & 7;
}
template <int D>
__device__ __forceinline__ int value_xor(int token) {
  return D == 128 ? (token & 3) << 2 : (token >> 1 & 1) << 2;
}

// 16 bytes of each lane's address to LDS, side by side from byte `to` on.  The compiler does not count these loads: what reads
// them comes behind arrive().  (Its own builtin for them makes the next read of LDS wait, whatever it reads.)
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t lane_bytes, uint32_t to) {  // base and `to` the same in a wave
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(lane_bytes), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory", "m0");
}
// All loads to LDS of the block have landed, and all waves are here.
__device__ __forceinline__ void arrive() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

template <int D, typename X, int KIND>
__global__ __launch_bounds__(kThreads, sizeof(X) == 4 && D == 128 ? 1 : 2) void tiles_kernel(TileArgs t) {
  const Args& a = t.a;
  constexpr int NQ = sizeof(X) == 2 ? 1 : 3;      // bf16 pieces of a query
  constexpr int NP = sizeof(X) == 2 ? 2 : 3;      // of a probability
  constexpr int kElem = KIND == kBf16 ? 2 : 1;
  constexpr int kPieces = D * kElem / 16;         // 16-byte loads of a token
  constexpr int kPass = kN * kPieces / kThreads;  // loads of a thread
  constexpr int kTokens = kThreads / kPieces;     // tokens of one load of the block
  constexpr int kK = D / 16, kC = D / 32;
  constexpr int kRowPieces = D / 8;               // 16-byte pieces of a token in LDS
  __shared__ __attribute__((aligned(1024))) u32x4 ks[2][kN * kRowPieces], vs[2][kN * kRowPieces];
  __shared__ float k_scale[2][kN], v_scale[2][kN];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, half = lane >> 5;
  // Heads are neighbours, so that the tiles of one head, which share its keys and values, go to one of the eight dies (blocks are
  // dealt out in turn); the last tiles of a run, which see most tokens, come first.
  const uint32_t h = blockIdx.x % a.heads, id = blockIdx.x / a.heads;
  const uint32_t part = id % t.parts;
  const Item item = item_of(a, t.items - 1 - id / t.parts);
  if (item.tile < 0) return;
  const Steps steps = steps_of(t, item);
  if ((int)part >= steps.parts) return;
  const int first_step = (int)part * steps.per;
  const int last_step = first_step + steps.per < steps.count ? first_step + steps.per : steps.count;

  // The lane's row.
  const int rows = item.run.n * (int)a.share, row0 = item.tile * kRows + 32 * wave;
  const int row = row0 + r < rows ? row0 + r : rows - 1;
  const int token = row / (int)a.share, head = (int)(h * a.share) + row - token * (int)a.share;
  const int place = steps.len - item.run.n + token;  // negative where the run is longer than its sequence
  const int high = a.causal && place + 1 < steps.len ? place + 1 : steps.len;
  const int low = a.window > 0 && place >= a.window ? place - a.window + 1 : 0;
  auto sees = [&](int at) { return at < high && (at >= low || at < a.sinks); };
  // Of the wave: what all of its rows see is [all_low, all_high), what any of them does lies in [any_low, any_high) or the first tokens.
  const int last_row = row0 + 31 < rows ? row0 + 31 : rows - 1;
  const int place0 = steps.len - item.run.n + row0 / (int)a.share, place1 = steps.len - item.run.n + last_row / (int)a.share;
  const int all_high = a.causal && place0 + 1 < steps.len ? place0 + 1 : steps.len;
  const int any_high = a.causal && place1 + 1 < steps.len ? place1 + 1 : steps.len;
  const int all_low = a.window > 0 && place1 >= a.window ? place1 - a.window + 1 : 0;
  const int any_low = a.window > 0 && place0 >= a.window ? place0 - a.window + 1 : 0;
  const bool live = row0 < rows;

  const float scale = fabsf(a.scale);
  bf16x8 q[kK][NQ];
  {
    const X* const x = static_cast<const X*>(a.q) + (int64_t)(item.run.s0 + token) * a.q_ts + (int64_t)head * a.q_hs + 8 * half;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      float v[8];
      if constexpr (NQ == 1) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(x + 16 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bits_float(w[i] << 16), v[2 * i + 1] = bits_float(w[i] & 0xFFFF0000u);
      } else {
        const f32x4 lo = reinterpret_cast<const f32x4*>(x + 16 * k)[0], hi = reinterpret_cast<const f32x4*>(x + 16 * k)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
      }
      if (!(a.scale > 0.0f)) {  // the maximum is taken of scores before their scale, whose sign goes to the query
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= a.scale < 0.0f ? -1.0f : 0.0f;
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = cut(v[2 * i], v[2 * i + 1]);
        q[k][n] = __builtin_bit_cast(bf16x8, w);
      }
    }
  }
  const float c = scale > 0.0f ? scale : 1.0f;

  // Lane i knows where group i of 16 tokens of the next 16 steps begins: bytes from the cache's start, -1 without a page.
  const int32_t* const table = a.table + (int64_t)item.b * a.ld_table;
  int64_t at = -1;
  int64_t scale_at = 0;
  auto look_up = [&](int step) {  // steps `step` to step + 15
    at = -1;
    const int s = step + lane / 4;
    if (s >= last_step) return;
    const uint32_t from = (uint32_t)steps.first_token(s) + 16 * (lane % 4);
    const uint32_t entry = from / a.page_size, slot = from - entry * a.page_size;
    if ((int)from >= steps.high) return;
    const int64_t page = table[entry];
    if (page < 0 || page >= a.num_pages) return;
    at = (page * a.page_stride + h * a.head_stride + (int64_t)slot * a.token_stride) * kElem;
    if constexpr (KIND == kFp8)
      scale_at = (page * a.heads + h) * (a.page_size / a.scale_tokens) + slot / a.scale_tokens;
    else
      scale_at = (page * a.heads + h) * a.page_size + slot;
  };

  // A step's keys and values: bf16 straight into LDS, 8-bit codes by way of registers.  Where some row of the block does not see the
  // whole step, lanes of tokens that none sees read the nearest one that is seen (or anything, if that has no page).
  constexpr int kBuffer = kN * kRowPieces;  // pieces of a buffer
  constexpr int kHeld = KIND == kBf16 ? 1 : kPass;
  u32x4 kr[kHeld] = {}, vr[kHeld] = {};
  float scale_r = 0.0f;
  const int my_token = threadIdx.x / kPieces, my_piece = threadIdx.x % kPieces;
  const uint32_t token_bytes = a.token_stride * kElem;
  const int kx_write = key_xor<D>(my_token), vx_write = value_xor<D>(my_token);
  // bf16: the lane's piece in a token is the one whose place in LDS is the lane's.
  const uint32_t k_piece = 16 * (my_piece ^ kx_write), v_piece = 16 * (my_piece ^ vx_write);
  const uint32_t k_bytes = (my_token % 16) * token_bytes + k_piece, v_bytes = (my_token % 16) * token_bytes + v_piece;
  // Where a wave's pieces of the first buffer go, and the values behind the keys.
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)&ks[0][0] + 1024 * wave);
  const uint32_t values_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)&vs[0][0] + 1024 * wave) - lds0;
  auto load = [&](int step) {  // returns which groups of tokens have a page
    const int number = step - first_step, lane0 = 4 * (number % 16);
    if (number % 16 == 0) look_up(step);
    const int t0 = steps.first_token(step);
    const unsigned paged = __ballot(at >= 0) >> lane0 & 15;
    if (paged == 0) return paged;
    const bool whole = paged == 15 && t0 >= steps.all_low && t0 + kN <= steps.all_high;
    const uint32_t to = lds0 + (number & 1) * (16 * kBuffer);
    auto nearest = [&](int i) {  // where the i-th token of the thread, or the nearest one that is seen, begins
      int tk = t0 + i * kTokens + my_token;
      tk = tk < steps.high ? tk : steps.high - 1;
      if (tk < steps.low && tk >= steps.sinks) tk = steps.sinks > t0 ? steps.sinks - 1 : steps.low;
      const int64_t group = __shfl(at, lane0 + ((tk - t0) >> 4));
      return (group < 0 ? 0 : group) + (int64_t)((uint64_t)(tk & 15) * token_bytes);
    };
    if constexpr (KIND == kBf16) {
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        if (whole) {  // a group is the same in a wave, whose 64 pieces go side by side
          const int64_t from = lane_value(at, lane0 + (i * kTokens + wave * (kTokens / 4)) / 16);
          load_to_lds(a.kp + from, k_bytes, to + i * 4096);
          load_to_lds(a.vp + from, v_bytes, to + i * 4096 + values_at);
        } else {
          const int64_t from = nearest(i);
          load_to_lds(a.kp + from + k_piece, to + i * 4096);
          load_to_lds(a.vp + from + v_piece, to + i * 4096 + values_at);
        }
      }
    } else {
      // One load for both, whose address is formed on one way alone.  (Loads on two ways were merged by the compiler, with an
      // address that was set on one of them.)  Of a whole step every token is its own nearest one.
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        const int64_t from = nearest(i) + 16 * my_piece;
        kr[i] = *reinterpret_cast<const u32x4*>(a.kp + from);
        vr[i] = *reinterpret_cast<const u32x4*>(a.vp + from);
      }
    }
    if constexpr (KIND != kBf16) {
      if (wave < 2) {  // 64 scales of keys, 64 of values; of tokens that no row sees none, which may be anything
        const int64_t from = __shfl(at, lane0 + lane / 16), s = __shfl(scale_at, lane0 + lane / 16);
        const int tk = t0 + lane;
        const bool seen = tk < steps.high && (tk >= steps.low || tk < steps.sinks);
        scale_r = seen && from >= 0 ? (wave == 0 ? a.ks : a.vs)[KIND == kFp8 ? s : s + lane % 16] : 0.0f;
      }
    }
    return paged;
  };
  auto stage = [&](int step) {  // 8-bit codes as bf16
    const int buffer = (step - first_step) & 1;
    u32x4* const kt = &ks[0][0] + buffer * kBuffer + my_token * kRowPieces;
    u32x4* const vt = &vs[0][0] + buffer * kBuffer + my_token * kRowPieces;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        u32x4 k, v;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const unsigned kw = kr[i][2 * u + j], vw = vr[i][2 * u + j];
          k[2 * j] = KIND == kFp8 ? pair_of_codes<false>(kw) : pair_of_bytes<false>(kw);
          k[2 * j + 1] = KIND == kFp8 ? pair_of_codes<true>(kw) : pair_of_bytes<true>(kw);
          v[2 * j] = KIND == kFp8 ? pair_of_codes<false>(vw) : pair_of_bytes<false>(vw);
          v[2 * j + 1] = KIND == kFp8 ? pair_of_codes<true>(vw) : pair_of_bytes<true>(vw);
        }
        kt[i * kTokens * kRowPieces + ((2 * my_piece + u) ^ kx_write)] = k;
        vt[i * kTokens * kRowPieces + ((2 * my_piece + u) ^ vx_write)] = v;
      }
    if (wave < 2) (wave == 0 ? k_scale : v_scale)[buffer][lane] = scale_r;
  };

  f32x16 o[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) o[i] = f32x16{};
  float m = kLowest, l = 0.0f;  // of the lane's row, in bits; l of its half of the tokens

  // Where the lane reads operands in LDS: piece 2 k + half of token r, and four channels of token 4 half + (lane / 4) % 4.
  const int k_row = r * kRowPieces, k_xor = key_xor<D>(r);
  const int v_token = 4 * half + (lane >> 2 & 3), v_xor = value_xor<D>(v_token);
  const int v_four = 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
  int k_at[kK], v_at[kC];
#pragma unroll
  for (int k = 0; k < kK; ++k) k_at[k] = k_row + ((2 * k + half) ^ k_xor);
#pragma unroll
  for (int d = 0; d < kC; ++d) v_at[d] = 2 * (v_token * kRowPieces + ((4 * d + v_four) ^ v_xor)) + (lane & 1);  // in 8 bytes

  // One step.  `edge`: some row of the wave may not see all of it.  CAREFUL: values that are not finite, which would reach the rows
  // that do not see their token through their zero probabilities, are left out of the product and added to the rows that see them.
  auto work = [&](auto careful, bool edge, int step, int t0, unsigned paged) {
    constexpr bool CAREFUL = decltype(careful)::value;
    const int buffer = (step - first_step) & 1;
    float s[2][16];
    float top = -INFINITY;
    const u32x4* const kt = &ks[0][0] + buffer * kBuffer;
    f32x16 acc[2] = {f32x16{}, f32x16{}};
    // Keys are read a group of operands ahead of the products.
    constexpr int kGroup = D == 64 && NQ == 1 ? 4 : 2;
    bf16x8 f[2][kGroup][2];
    auto read_keys = [&](int group) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          f[group & 1][k][u] = __builtin_bit_cast(bf16x8, kt[k_at[group * kGroup + k] + 32 * u * kRowPieces]);
    };
    // While matrix instructions are to be issued the wave goes before the one that shares its SIMD.
    if constexpr (KIND == kBf16) __builtin_amdgcn_s_setprio(1);
    read_keys(0);
#pragma unroll
    for (int group = 0; group < kK / kGroup; ++group) {
      if (group + 1 < kK / kGroup) read_keys(group + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kGroup; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = NQ - 1; n >= 0; --n)
            acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[group & 1][k][u], q[group * kGroup + k][n], acc[u], 0, 0, 0);
    }
    if constexpr (KIND == kBf16) __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[u][i] = acc[u][i];
      if constexpr (KIND != kBf16) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 f = *reinterpret_cast<const f32x4*>(&k_scale[buffer][32 * u + 8 * g + 4 * half]);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[u][4 * g + i] *= f[i];
        }
      }
    }
    if (edge) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int tk = t0 + 32 * u + 8 * (i >> 2) + 4 * half + (i & 3);
          const bool seen = (tk < high) & ((tk >= low) | (tk < a.sinks)) & ((paged >> (2 * u + (i >> 3)) & 1) != 0);
          s[u][i] = seen ? s[u][i] : -INFINITY;
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
    const u32x2 both = __builtin_amdgcn_permlane32_swap(float_bits(top), float_bits(top), false, false);  // the two halves' maxima
    top = fmaxf(bits_float(both[0]), bits_float(both[1])) * c;
    if (__any(top > m + kSlack)) {
      top = fmaxf(top, m);
      const float shrink = exp2_raw(m - top);
      m = top;
      l *= shrink;
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] *= shrink;
    }
    // Probabilities of 16 tokens, numbers 8 g to 8 g + 7 of half u.
    auto probabilities = [&](int u, int g, bf16x8 (&p)[NP]) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float& y = s[u][8 * g + i];
        y = exp2_raw(fmaf(y, c, -m));
        l += y;
      }
      if constexpr (KIND != kBf16) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const f32x4 f = *reinterpret_cast<const f32x4*>(&v_scale[buffer][32 * u + 16 * g + 8 * z + 4 * half]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& y = s[u][8 * g + 4 * z + i];
            const int tk = 32 * u + 16 * g + 8 * z + 4 * half + i;
            // A scale of a token that the row does not see may be anything.
            y = !CAREFUL || (sees(t0 + tk) & ((paged >> (2 * u + g) & 1) != 0)) ? y * f[i] : 0.0f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = s[u][8 * g + i];
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = NP == 3 ? cut(x[2 * i], x[2 * i + 1]) : (n == 0 ? cut_nearest(x[2 * i], x[2 * i + 1]) : pack(x[2 * i], x[2 * i + 1]));
        p[n] = __builtin_bit_cast(bf16x8, w);
      }
    };
    s16x4* const vt = reinterpret_cast<s16x4*>(&vs[0][0] + buffer * kBuffer);
    auto values = [&](int u, int g, int d) {  // operand of 16 tokens and 32 channels
      u32x4 w;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        s16x4* const from = vt + v_at[d] + 2 * (32 * u + 16 * g + 8 * z) * kRowPieces;
        const u32x2 x = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)from));
        w[2 * z] = x[0];
        w[2 * z + 1] = x[1];
      }
      return w;
    };
    // The vector ALU works on the next 16 tokens' probabilities while the matrix cores multiply these.
    bf16x8 p[2][NP];
    u32x4 w[2][kC];
    auto read_values = [&](int n16) {
#pragma unroll
      for (int d = 0; d < kC; ++d) w[n16 & 1][d] = values(n16 >> 1, n16 & 1, d);
    };
    read_values(0);
    __builtin_amdgcn_sched_barrier(0);
    probabilities(0, 0, p[0]);
    if constexpr (KIND == kBf16) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int n16 = 0; n16 < 4; ++n16) {
      if (n16 < 3) read_values(n16 + 1);
#pragma unroll
      for (int d = 0; d < kC; ++d) {
        if constexpr (CAREFUL) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[n16 & 1][d][i] = even_pair(w[n16 & 1][d][i]);
        }
        const bf16x8 f = __builtin_bit_cast(bf16x8, w[n16 & 1][d]);
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, p[n16 & 1][n], o[d], 0, 0, 0);
      }
      if (n16 < 3) probabilities((n16 + 1) >> 1, (n16 + 1) & 1, p[(n16 + 1) & 1]);
    }
    // fp32 queries of 128 channels leave room for one wave a SIMD: its vector instructions go between its own matrix instructions (two
    // prompts of up to 4000 tokens 0.60 ms where it was 0.63; with two waves a SIMD there is nothing to gain).
    if constexpr (NP == 3 && D == 128 && KIND == kBf16 && !CAREFUL) {
#pragma unroll
      for (int i = 0; i < 3 * NP * kC; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x402, 72 / (NP * kC), 0);
      }
    }
    if constexpr (KIND == kBf16) __builtin_amdgcn_s_setprio(0);
    if constexpr (CAREFUL) {
      const u32x4* const mine = &vs[buffer][lane * kRowPieces];  // lane i looks at token i
      bool any = false;
      for (int j = 0; j < kRowPieces; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= odd_pair(mine[j][i]);
      for (uint64_t left = __ballot(any); left; left &= left - 1) {
        const int tk = __builtin_ctzll(left);
        float p = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) p = (tk >> 5) == u && ((tk >> 3 & 3) << 2 | (tk & 3)) == i ? s[u][i] : p;
        p = __shfl(p, r + 32 * (tk >> 2 & 1));
        const uint16_t* const v = reinterpret_cast<const uint16_t*>(&vs[buffer][tk * kRowPieces]);
        const int vx = value_xor<D>(tk);
        const bool seen = sees(t0 + tk) && (paged >> (tk >> 4) & 1);
#pragma unroll
        for (int d = 0; d < kC; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int ch = 32 * d + 8 * (i >> 2) + 4 * half + (i & 3);
            const unsigned w = v[((ch >> 3) ^ vx) * 8 + (ch & 7)];
            if (seen && (w & 0x7F80u) == 0x7F80u) o[d][i] = fmaf(bits_float(w << 16), p, o[d][i]);
          }
      }
    }
  };

  auto pass = [&](auto careful) {
    unsigned paged = 0, paged_next = 0;
    if (first_step < last_step) {
      paged = load(first_step);
      if constexpr (KIND != kBf16) stage(first_step);
    }
    arrive();
    for (int step = first_step; step < last_step; ++step) {
      const int t0 = steps.first_token(step);
      const bool more = step + 1 < last_step;
      if (more) paged_next = load(step + 1);
      if (live && paged != 0 && t0 < any_high && (t0 + kN > any_low || t0 < a.sinks))
        work(careful, t0 < all_low || t0 + kN > all_high || paged != 15, step, t0, paged);
      if constexpr (KIND != kBf16) {
        if (more) stage(step + 1);
      }
      paged = paged_next;
      arrive();
    }
  };
  pass(std::false_type{});
  // Again, with care, where something was not finite.
  float zero = 0.0f * l;
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) zero = fmaf(o[i][j], 0.0f, zero);
  if (__syncthreads_or(live && zero != 0.0f)) {  // NaN
    m = kLowest;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < kC; ++i) o[i] = f32x16{};
    pass(std::true_type{});
  }

  l += __shfl_xor(l, 32);
  if (!live || row0 + r >= rows) return;
  if (steps.parts == 1) {
    const float inverse = l == 0.0f ? 0.0f : 1.0f / l;  // no token: zeros
    X* const to = static_cast<X*>(a.o) + (int64_t)(item.run.s0 + token) * a.o_ts + (int64_t)head * a.o_hs + 4 * half;
#pragma unroll
    for (int d = 0; d < kC; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = l == 0.0f ? 0.0f : o[d][4 * g + i] * inverse;
        if constexpr (sizeof(X) == 2)
          *reinterpret_cast<u32x2*>(to + 32 * d + 8 * g) = u32x2{pack(v[0], v[1]), pack(v[2], v[3])};
        else
          *reinterpret_cast<f32x4*>(to + 32 * d + 8 * g) = f32x4{v[0], v[1], v[2], v[3]};
      }
  } else {
    const int64_t index = ((int64_t)part * a.T + item.run.s0 + token) * a.q_heads + head;
    float* const to = a.partial + index * D + 4 * half;
#pragma unroll
    for (int d = 0; d < kC; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4*>(to + 32 * d + 8 * g) = f32x4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
    if (half == 0) {
      float* const ml = a.partial + (int64_t)t.parts * a.T * a.q_heads * D + 2 * index;
      ml[0] = m;
      ml[1] = l;
    }
  }
}

// Parts joined: D / 4 lanes to a query head of a token, four channels each.  The lanes weigh a part each, then add the parts.
template <int D, typename X>
__global__ __launch_bounds__(256) void join_tiles_kernel(TileArgs t) {
  const Args& a = t.a;
  constexpr int kLanes = D / 4;
  const int sub = threadIdx.x % kLanes;
  const uint32_t rows_all = (uint32_t)a.T * a.q_heads;
  const uint32_t given = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes, id = given < rows_all ? given : rows_all - 1;
  const int s = (int)(id / a.q_heads), head = (int)(id % a.q_heads);
  // The sequence of row s: the last one that does not begin behind it.
  int b = 0, end = (int)a.B;
  while (end - b > 1) {
    const int mid = (b + end) / 2;
    if (a.starts[mid] <= s) b = mid;
    else end = mid;
  }
  Item item = {b, 0, run_of(a, b)};
  if (given >= rows_all || s < item.run.s0 || s - item.run.s0 >= item.run.n) return;
  item.tile = ((s - item.run.s0) * (int)a.share + head % (int)a.share) / kRows;
  const int parts = steps_of(t, item).parts;
  if (parts == 1) return;  // its one block has written the result
  const int64_t step = rows_all;
  const float* const ml = a.partial + (int64_t)t.parts * step * D + 2 * (int64_t)id;
  const f32x4* const part = reinterpret_cast<const f32x4*>(a.partial + (int64_t)id * D) + sub;
  float m = kLowest, l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  for (int first = 0; first < parts; first += kLanes) {
    const int n = parts - first < kLanes ? parts - first : kLanes;
    const f32x2 mine = sub < n ? *reinterpret_cast<const f32x2*>(ml + 2 * (first + sub) * step) : f32x2{kLowest, 0.0f};
    float top = fmaxf(m, mine[0]);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float shrink = exp2_raw(m - top), weight = exp2_raw(mine[0] - top);
    m = top;
    l = l * shrink + weight * mine[1];  // of this lane's parts
    o *= shrink;
    for (int q = 0; q < n; ++q) {
      const f32x4 x = part[(first + q) * step * (D / 4)];
      o += __shfl(weight, q, kLanes) * x;
    }
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) l += __shfl_xor(l, d);
  X* const to = static_cast<X*>(a.o) + (int64_t)s * a.o_ts + (int64_t)head * a.o_hs + 4 * sub;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = l == 0.0f ? 0.0f : o[i] / l;
  if constexpr (sizeof(X) == 2)
    *reinterpret_cast<u32x2*>(to) = u32x2{pack(v[0], v[1]), pack(v[2], v[3])};
  else
    *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
}

template <int D, typename X>
hipError_t launch_tiles(const TileArgs& t, int kind, unsigned blocks, hipStream_t st) {
  kind == kBf16   ? tiles_kernel<D, X, kBf16><<<blocks, kThreads, 0, st>>>(t)
  : kind == kInt8 ? tiles_kernel<D, X, kInt8><<<blocks, kThreads, 0, st>>>(t)
                  : tiles_kernel<D, X, kFp8><<<blocks, kThreads, 0, st>>>(t);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || t.parts == 1) return e;
  constexpr int kJoined = 256 / (D / 4);  // of a block
  join_tiles_kernel<D, X><<<(unsigned)(((int64_t)t.a.T * t.a.q_heads + kJoined - 1) / kJoined), 256, 0, st>>>(t);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_run_tiles(const RunArgs& in, hipStream_t st) {
  bool split;
  TileArgs t = {};
  t.a = arguments(in.base, in.max_run, &split);
  t.a.starts = in.starts;
  t.a.T = (int32_t)in.T;
  t.a.sinks = in.sinks > 0x7fffffff ? 0x7fffffff : (int32_t)in.sinks;
  t.a.causal = in.causal;
  RunTiles tiles = run_tiles(in.T, in.base.B, in.base.q_heads, in.base.cache.heads, t.a.capacity);  // as the workspace was sized
  const int64_t seen = tokens_of_tile(t.a.capacity, in.max_run, in.base.window, in.sinks, in.causal);
  if (seen < t.a.capacity) tiles = run_tiles(in.T, in.base.B, in.base.q_heads, in.base.cache.heads, seen, tiles.parts);
  t.items = tiles.items;
  t.parts = (uint32_t)tiles.parts;
  t.least = (uint32_t)kLeastSteps;
  const unsigned blocks = (unsigned)(tiles.items * tiles.parts * in.base.cache.heads);
  const int kind = in.base.cache.dtype;
  if (in.base.cache.head_dim == 64)
    return in.base.bf16 ? launch_tiles<64, __hip_bfloat16>(t, kind, blocks, st) : launch_tiles<64, float>(t, kind, blocks, st);
  return in.base.bf16 ? launch_tiles<128, __hip_bfloat16>(t, kind, blocks, st) : launch_tiles<128, float>(t, kind, blocks, st);
}

}  // namespace qv
