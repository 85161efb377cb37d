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
// Both are v_mfma_f32_32x32x16_bf16; queries stay in registers, keys and values go global -> registers -> LDS while the tile
// before is worked on (two buffers, one barrier a tile); 8-bit caches are converted on the way, once for the four waves.
// In LDS a 16-byte piece of a row lies at its number xor the row's: reads of one piece of eight rows, and transposed reads of
// 32 channels of four rows, then fall on different banks.
//
// bf16 queries: probabilities are rounded to bf16 for the second product (to nearest, 2^-9 of each on average and of either
// sign, as much as the result's own rounding); their sum is of the unrounded ones.  fp32 queries and their probabilities
// are three bf16 pieces that sum to them.
// The maximum that scales a row's probabilities is raised only when one passes 2^8 of it: sums are fp32, and the rest follows.
#include "paged_attention.h"
#include "qv_runs_internal.h"

namespace qv {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
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

__device__ __forceinline__ bool odd_pair(unsigned w) {  // an infinity or NaN among two bf16 values
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ unsigned even_pair(unsigned w) {  // zeros in their place
  w = (w & 0x7F80u) == 0x7F80u ? w & 0xFFFF0000u : w;
  return (w & 0x7F800000u) == 0x7F800000u ? w & 0xFFFFu : w;
}

template <int D, typename X, int KIND>
__global__ __launch_bounds__(kThreads, sizeof(X) == 4 && D == 128 ? 1 : 2) void tiles_kernel(TileArgs t) {
  const Args& a = t.a;
  constexpr int NP = sizeof(X) == 2 ? 1 : 3;      // bf16 pieces of a query and of a probability
  constexpr int kElem = KIND == kBf16 ? 2 : 1;
  constexpr int kPieces = D * kElem / 16;         // 16-byte loads of a token
  constexpr int kPass = kN * kPieces / kThreads;  // loads of a thread
  constexpr int kTokens = kThreads / kPieces;     // tokens of one load of the block
  constexpr int kK = D / 16, kC = D / 32;
  constexpr int kRowPieces = D / 8;               // 16-byte pieces of a token in LDS
  __shared__ u32x4 ks[2][kN * kRowPieces], vs[2][kN * kRowPieces];
  __shared__ float k_scale[2][kN], v_scale[2][kN];
  __shared__ unsigned odd[3][2];                  // tokens of a step with a value that is not finite

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
  bf16x8 q[kK][NP];
  {
    const X* const x = static_cast<const X*>(a.q) + (int64_t)(item.run.s0 + token) * a.q_ts + (int64_t)head * a.q_hs + 8 * half;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      float v[8];
      if constexpr (NP == 1) {
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
      for (int n = 0; n < NP; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = cut(v[2 * i], v[2 * i + 1]);
        q[k][n] = __builtin_bit_cast(bf16x8, w);
      }
    }
  }
  const float c = scale > 0.0f ? scale : 1.0f;

  // Lane i knows where group i of 16 tokens of the next 16 steps begins: an offset from the cache's start, -1 without a page.
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
    at = page * a.page_stride + h * a.head_stride + (int64_t)slot * a.token_stride;
    if constexpr (KIND == kFp8)
      scale_at = (page * a.heads + h) * (a.page_size / a.scale_tokens) + slot / a.scale_tokens;
    else
      scale_at = (page * a.heads + h) * a.page_size + slot;
  };

  // A step's keys and values on their way: this thread's pieces, and which groups of tokens have a page.
  u32x4 kr[kPass], vr[kPass];
  float scale_r = 0.0f;
  const int my_token = threadIdx.x / kPieces, my_piece = threadIdx.x % kPieces;
  const uint32_t token_bytes = a.token_stride * kElem;
  auto any_sees = [&](int tk) { return tk < steps.high && (tk >= steps.low || tk < steps.sinks); };
  auto block_edge = [&](int t0) { return t0 < steps.low || t0 + kN > steps.high; };
  auto load = [&](int step) {
    if (step % 16 == first_step % 16) look_up(step);
    const int t0 = steps.first_token(step), lane0 = 4 * ((step - first_step) % 16);
    const bool edge = block_edge(t0);
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const int tk = i * kTokens + my_token;
      const int group = (i * kTokens + wave * (kTokens / 4)) / 16;  // the same in a wave
      const int64_t from = lane_value(at, lane0 + group);
      kr[i] = vr[i] = u32x4{0, 0, 0, 0};
      if (from >= 0 && (!edge || any_sees(t0 + tk))) {
        const int64_t off = from * kElem + (uint64_t)(tk % 16) * token_bytes + 16 * my_piece;
        kr[i] = *reinterpret_cast<const u32x4*>(a.kp + off);
        vr[i] = *reinterpret_cast<const u32x4*>(a.vp + off);
      }
    }
    if constexpr (KIND != kBf16) {
      if (wave < 2) {  // 64 scales of keys, 64 of values
        const int64_t from = __shfl(at, lane0 + lane / 16), s = __shfl(scale_at, lane0 + lane / 16);
        scale_r = from >= 0 ? (wave == 0 ? a.ks : a.vs)[KIND == kFp8 ? s : s + lane % 16] : 0.0f;
      }
    }
    return __ballot(at >= 0) >> lane0 & 15;  // groups of the step that have a page
  };
  auto stage = [&](int step) {
    const int t0 = steps.first_token(step), buffer = (step - first_step) & 1, slot = (step - first_step) % 3;
    const bool edge = block_edge(t0) || a.causal || a.window > 0;
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const int tk = i * kTokens + my_token;
      u32x4* const kt = &ks[buffer][tk * kRowPieces];
      u32x4* const vt = &vs[buffer][tk * kRowPieces];
      const int kx = tk & (kRowPieces - 1), vx = D == 128 ? (tk & 3) << 2 : (tk >> 1 & 1) << 2;
      if constexpr (KIND == kBf16) {
        kt[my_piece ^ kx] = kr[i];
        vt[my_piece ^ vx] = vr[i];
        if (edge) {
          bool any = false;
#pragma unroll
          for (int j = 0; j < 4; ++j) any |= odd_pair(vr[i][j]);
          if (any) atomicOr(&odd[slot][tk >> 5], 1u << (tk & 31));
        }
      } else {
        u32x4 k[2], v[2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const unsigned kw = kr[i][j], vw = vr[i][j];
            if constexpr (KIND == kFp8) {
              k[j >> 1][2 * (j & 1) + u] = u ? pair_of_codes<true>(kw) : pair_of_codes<false>(kw);
              v[j >> 1][2 * (j & 1) + u] = u ? pair_of_codes<true>(vw) : pair_of_codes<false>(vw);
            } else {
              k[j >> 1][2 * (j & 1) + u] = u ? pair_of_bytes<true>(kw) : pair_of_bytes<false>(kw);
              v[j >> 1][2 * (j & 1) + u] = u ? pair_of_bytes<true>(vw) : pair_of_bytes<false>(vw);
            }
          }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          kt[(2 * my_piece + u) ^ kx] = k[u];
          vt[(2 * my_piece + u) ^ vx] = v[u];
        }
        if (KIND == kFp8 && edge) {
          bool any = false;
#pragma unroll
          for (int j = 0; j < 4; ++j) any |= (((vr[i][j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
          if (any) atomicOr(&odd[slot][tk >> 5], 1u << (tk & 31));
        }
      }
    }
    if constexpr (KIND != kBf16) {
      if (wave < 2) (wave == 0 ? k_scale : v_scale)[buffer][lane] = scale_r;
    }
  };

  f32x16 o[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) o[i] = f32x16{};
  float m = kLowest, l = 0.0f;  // of the lane's row, in bits; l of its half of the tokens

  if (threadIdx.x < 6) odd[threadIdx.x >> 1][threadIdx.x & 1] = 0;
  __syncthreads();
  uint64_t paged = 0, paged_next = 0;
  if (first_step < last_step) {
    paged = load(first_step);
    stage(first_step);
  }
  __syncthreads();

  for (int step = first_step; step < last_step; ++step) {
    const int buffer = (step - first_step) & 1, t0 = steps.first_token(step);
    const bool more = step + 1 < last_step;
    if (more) paged_next = load(step + 1);
    if (threadIdx.x < 2) odd[(step - first_step + 2) % 3][threadIdx.x] = 0;  // read a step ago, used in the next but one

    if (live && t0 < any_high && (t0 + kN > any_low || t0 < a.sinks)) {
      const bool edge = t0 < all_low || t0 + kN > all_high || paged != 15;
      float s[2][16];
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x16 acc = f32x16{};
        const u32x4* const kt = &ks[buffer][(32 * u + r) * kRowPieces];
        const int kx = r & (kRowPieces - 1);
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const bf16x8 f = __builtin_bit_cast(bf16x8, kt[(2 * k + half) ^ kx]);
#pragma unroll
          for (int n = NP - 1; n >= 0; --n) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[k][n], acc, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = acc[i];
        if constexpr (KIND != kBf16) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&k_scale[buffer][32 * u + 8 * g + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][4 * g + i] *= f[i];
          }
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int tk = 32 * u + 8 * (i >> 2) + 4 * half + (i & 3);
            s[u][i] = sees(t0 + tk) && (paged >> (tk >> 4) & 1) ? s[u][i] : -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
      }
      top = fmaxf(top, __shfl_xor(top, 32)) * c;
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
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[u][i] = exp2_raw(fmaf(s[u][i], c, -m));
          l += s[u][i];
        }
      if constexpr (KIND != kBf16) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&v_scale[buffer][32 * u + 8 * g + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float& p = s[u][4 * g + i];
              const int tk = 32 * u + 8 * g + 4 * half + i;
              p = !edge || (sees(t0 + tk) && (paged >> (tk >> 4) & 1)) ? p * f[i] : 0.0f;  // a scale that a row does not see may be anything
            }
          }
      }
      const uint64_t odd_tokens = edge && KIND != kInt8 ? (uint64_t)odd[(step - first_step) % 3][1] << 32 | odd[(step - first_step) % 3][0] : 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          bf16x8 p[NP];
          if constexpr (NP == 1) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack(s[u][8 * g + 2 * i], s[u][8 * g + 2 * i + 1]);
            p[0] = __builtin_bit_cast(bf16x8, w);
          } else {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = s[u][8 * g + i];
#pragma unroll
            for (int n = 0; n < NP; ++n) {
              u32x4 w;
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = cut(x[2 * i], x[2 * i + 1]);
              p[n] = __builtin_bit_cast(bf16x8, w);
            }
          }
#pragma unroll
          for (int d = 0; d < kC; ++d) {
            u32x4 w;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int tk = 32 * u + 16 * g + 8 * z + 4 * half + (lane >> 2 & 3);
              const int piece = 4 * d + 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
              const int vx = D == 128 ? (tk & 3) << 2 : (tk >> 1 & 1) << 2;
              s16x4* const from = reinterpret_cast<s16x4*>(&vs[buffer][tk * kRowPieces + (piece ^ vx)]) + (lane & 1);
              const u32x2 x = __builtin_bit_cast(
                  u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)from));
              w[2 * z] = x[0];
              w[2 * z + 1] = x[1];
            }
            if (odd_tokens) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = even_pair(w[i]);
            }
            const bf16x8 f = __builtin_bit_cast(bf16x8, w);
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, p[n], o[d], 0, 0, 0);
          }
        }
      // Values that are not finite would reach the rows that do not see their token through their zero probabilities: they
      // were left out above and are added to the rows that see them.
      for (uint64_t left = odd_tokens; left; left &= left - 1) {
        const int tk = __builtin_ctzll(left);
        float p = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) p = (tk >> 5) == u && ((tk >> 3 & 3) << 2 | (tk & 3)) == i ? s[u][i] : p;
        p = __shfl(p, r + 32 * (tk >> 2 & 1));
        const uint16_t* const v = reinterpret_cast<const uint16_t*>(&vs[buffer][tk * kRowPieces]);
        const int vx = D == 128 ? (tk & 3) << 2 : (tk >> 1 & 1) << 2;
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
    if (more) stage(step + 1);
    paged = paged_next;
    __syncthreads();
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
        if constexpr (NP == 1)
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

// Parts joined: a wave to a query head of a token.
template <int D, typename X>
__global__ __launch_bounds__(256) void join_tiles_kernel(TileArgs t) {
  const Args& a = t.a;
  constexpr int kPer = D / 64;
  const int lane = threadIdx.x & 63;
  const uint32_t id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (id >= (uint32_t)a.T * a.q_heads) return;
  const int s = (int)(id / a.q_heads), head = (int)(id % a.q_heads);
  // The sequence of row s: the last one that does not begin behind it.
  int b = 0, end = (int)a.B;
  while (end - b > 1) {
    const int mid = (b + end) / 2;
    if (a.starts[mid] <= s) b = mid;
    else end = mid;
  }
  Item item = {b, 0, run_of(a, b)};
  if (s < item.run.s0 || s - item.run.s0 >= item.run.n) return;
  const int row = (s - item.run.s0) * (int)a.share + head % (int)a.share;
  item.tile = row / kRows;
  const Steps steps = steps_of(t, item);
  if (steps.parts == 1) return;
  const int64_t step = (int64_t)a.T * a.q_heads, ml0 = (int64_t)t.parts * step * D;
  float m = kLowest, l = 0.0f, o[kPer] = {};
  for (int p = 0; p < steps.parts; ++p) m = fmaxf(m, a.partial[ml0 + 2 * (p * step + id)]);
  for (int p = 0; p < steps.parts; ++p) {
    const float w = exp2_raw(a.partial[ml0 + 2 * (p * step + id)] - m);
    l = fmaf(w, a.partial[ml0 + 2 * (p * step + id) + 1], l);
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = fmaf(w, a.partial[(p * step + id) * D + kPer * lane + i], o[i]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    store(static_cast<X*>(a.o) + (int64_t)s * a.o_ts + (int64_t)head * a.o_hs + kPer * lane + i, l == 0.0f ? 0.0f : o[i] / l);
}

template <int D, typename X>
hipError_t launch_tiles(const TileArgs& t, int kind, unsigned blocks, hipStream_t st) {
  kind == kBf16   ? tiles_kernel<D, X, kBf16><<<blocks, kThreads, 0, st>>>(t)
  : kind == kInt8 ? tiles_kernel<D, X, kInt8><<<blocks, kThreads, 0, st>>>(t)
                  : tiles_kernel<D, X, kFp8><<<blocks, kThreads, 0, st>>>(t);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || t.parts == 1) return e;
  join_tiles_kernel<D, X><<<(unsigned)(((int64_t)t.a.T * t.a.q_heads + 3) / 4), 256, 0, st>>>(t);
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
  const RunTiles tiles = run_tiles(in.T, in.base.B, in.base.q_heads, in.base.cache.heads, t.a.capacity);
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
