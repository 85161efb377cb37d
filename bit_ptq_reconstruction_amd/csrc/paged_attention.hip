// paged_attention.hip -- attention of one new token of every sequence over a paged cache of keys and
// values (bf16, or int8 with a scale per token and head).
//
//   O[b][i] = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q_i . k_t - m),  m the running maximum
//
// One pass over the keys and values, which is all there is to move: the kernel is bound by memory.  48 sequences of up to
// 16384 tokens (8 heads of 128, 32 queries, 1.6 GB) take 270 us, 6.0 TB/s (a copy runs at 5.0; the matrix cores are busy for 8 %
// and the vector ALU for 14 % of the time); two of 99991 tokens in int8 (211 MB) take 49-50 us, 4.3 TB/s (vector ALU
// 44 %, for the conversions).  One frame of 1374 tokens (5.6 MB) takes 7.9 us: 5.0 for the parts' chain of loads (lengths,
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
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qv_decode_internal.h"

namespace qv {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;  // of a block
constexpr int kTile = (int)kTokensPerTile;
constexpr int kCUs = 256, kMaxResident = 8;
static_assert(kCUs * kMaxResident <= kManyBlocks, "a round of blocks");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;  // finite, so that differences of maxima are never inf - inf

struct Args {
  const void* q;
  void* o;
  const char *kp, *vp;
  const float *ks, *vs;
  const int32_t *table, *lens;
  float* partial;  // [parts][q_heads][D], then [parts][q_heads][2] (maximum, sum)
  int64_t q_ts, q_hs, o_ts, o_hs, page_stride, head_stride, ld_table, num_pages;
  int64_t few, many;  // parts of all sequences together
  int32_t few_tiles;   // whether all sequences at their capacity have fewer than 2^31 tiles
  int32_t capacity, window;  // a window of more than 2^31 - 1 tokens is none
  uint32_t B, heads, q_heads, share, q_tiles, parts, token_stride, page_size;
  float scale;  // times log2 e
};

__device__ __forceinline__ float bits_float(unsigned u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ unsigned float_bits(float f) { return __builtin_bit_cast(unsigned, f); }

// Tokens [begin, end) that a sequence attends to and their tiles [first, last); places are counted in 31 bits.
struct Span {
  int begin, end, first, last;
};
__device__ __forceinline__ Span span_of(const Args& a, int n) {
  Span s;
  s.end = n < 0 ? 0 : (n > a.capacity ? a.capacity : n);
  s.begin = a.window > 0 && s.end > a.window ? s.end - a.window : 0;
  s.first = s.begin / kTile;
  s.last = (s.end + kTile - 1) / kTile;
  return s;
}

// Sums over the lanes up to each one, by DPP: within rows of 16 lanes, then a row's total to the rows behind it.
__device__ __forceinline__ int scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return x;
}

// Where a part lies.  The tiles of all sequences together give the size of a part; a sequence has as many as that
// takes, at least one, and the parts of all sequences are numbered through.  A wave's lanes work this
// out from the lengths, 64 sequences at a time; every result is the same in all lanes.
struct Part {
  int b, index;         // sequence and number in it
  int first_of, count;  // number of the sequence's first part among all, and how many it has
  int per_part;         // tiles
  Span span;
};
// BY_PART: of part number `which` (b = -1: there is none), else of sequence `which` (index 0).
template <bool BY_PART>
__device__ __forceinline__ Part find_part(const Args& a, int which) {
  const int lane = threadIdx.x & 63, B = (int)a.B;
  Part p;
  const int mine = lane < B ? a.lens[lane] : 0;  // of the first 64 sequences
  const Span own = span_of(a, mine);
  if (B <= 64 && a.few_tiles) {  // the totals fit 32 bits
    const uint32_t total = __builtin_amdgcn_readlane(scan(own.last - own.first), 63);
    p.per_part = __builtin_amdgcn_readfirstlane(tiles_of_part(total, (uint32_t)a.few, (uint32_t)a.many));
  } else {
    uint64_t total = own.last - own.first;
    for (int i = lane + 64; i < B; i += 64) {
      const Span s = span_of(a, a.lens[i]);
      total += s.last - s.first;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
    p.per_part = __builtin_amdgcn_readfirstlane(tiles_of_part(total, (uint64_t)a.few, (uint64_t)a.many));
  }
  int base = 0;  // parts of the sequences before
  p.b = -1;
  for (int first = 0; first < B; first += 64) {
    const int i = first + lane;
    const int n = first == 0 ? mine : (i < B ? a.lens[i] : 0);
    const Span s = span_of(a, n);
    const int tiles = s.last - s.first;
    const int count = i < B ? (tiles > p.per_part ? (int)((uint32_t)(tiles + p.per_part - 1) / (uint32_t)p.per_part) : 1) : 0;
    const int upto = scan(count);
    const uint64_t hit = BY_PART ? __ballot(i < B && base + upto > which) : __ballot(i == which);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      p.b = first + at;
      p.count = __builtin_amdgcn_readlane(count, at);
      p.first_of = base + __builtin_amdgcn_readlane(upto, at) - p.count;
      p.index = BY_PART ? which - p.first_of : 0;
      p.span = span_of(a, __builtin_amdgcn_readlane(n, at));
      break;
    }
    base += __builtin_amdgcn_readlane(upto, 63);
  }
  return p;
}

// Byte i of a dword as a signed number, in one instruction.
template <int i>
__device__ __forceinline__ float signed_byte(unsigned w) {
  float f;
  if constexpr (i == 0)
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(w));
  else if constexpr (i == 1)
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(w));
  else if constexpr (i == 2)
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(w));
  else
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(w));
  return f;
}

// Keys of one tile as loaded, and as operands of the score product.
template <int D, bool INT8>
struct Keys {
  static constexpr int kLoads = INT8 ? D / 64 : D / 32;
  u32x4 d[kLoads];
  __device__ __forceinline__ void load(const char* tile, uint32_t lane_bytes) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      d[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(tile + lane_bytes + 64 * j));
  }
  // operand f covers channels channel(f, c) .. + 7
  static __device__ __forceinline__ int channel(int f, int c) {
    return INT8 ? 64 * (f >> 1) + 16 * c + 8 * (f & 1) : 32 * f + 8 * c;
  }
  __device__ __forceinline__ bf16x8 operand(int f) const {
    if constexpr (!INT8) {
      return __builtin_bit_cast(bf16x8, d[f]);
    } else {
      u32x4 o;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned w = d[f >> 1][2 * (f & 1) + h];
        o[2 * h] = __builtin_amdgcn_perm(float_bits(signed_byte<1>(w)), float_bits(signed_byte<0>(w)), 0x07060302u);
        o[2 * h + 1] = __builtin_amdgcn_perm(float_bits(signed_byte<3>(w)), float_bits(signed_byte<2>(w)), 0x07060302u);
      }
      return __builtin_bit_cast(bf16x8, o);
    }
  }
};

// Channels kE r .. kE r + kE - 1 of one token's value.
template <int D, bool INT8>
struct Values {
  static constexpr int kE = D / 16;
  static constexpr int kBytes = kE * (INT8 ? 1 : 2);
  static constexpr int kWords = kBytes / 4;
  unsigned d[kWords];
  __device__ __forceinline__ void load(const char* tile, uint32_t lane_bytes) {
    const char* const p = tile + lane_bytes;
    if constexpr (kWords == 4) {
      const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
      d[0] = v[0], d[1] = v[1], d[2] = v[2], d[3] = v[3];
    } else if constexpr (kWords == 2) {
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
      d[0] = v[0], d[1] = v[1];
    } else {
      d[0] = __builtin_nontemporal_load(reinterpret_cast<const unsigned*>(p));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) d[i] = 0;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (INT8) {
      const unsigned w = d[e >> 2];
      return (e & 3) == 0 ? signed_byte<0>(w) : (e & 3) == 1 ? signed_byte<1>(w) : (e & 3) == 2 ? signed_byte<2>(w)
                                                                                                : signed_byte<3>(w);
    }
    return (e & 1) ? bits_float(d[e >> 1] & 0xFFFF0000u) : bits_float(d[e >> 1] << 16);
  }
  // Channel e of two tokens as a bf16 pair.
  static __device__ __forceinline__ unsigned pair(const Values& a, const Values& b, int e) {
    if constexpr (INT8) return __builtin_amdgcn_perm(float_bits(b.get(e)), float_bits(a.get(e)), 0x07060302u);
    return __builtin_amdgcn_perm(b.d[e >> 1], a.d[e >> 1], (e & 1) ? 0x07060302u : 0x05040100u);
  }
};

__device__ __forceinline__ void store(float* o, float v) { *o = v; }
__device__ __forceinline__ void store(__hip_bfloat16* o, float v) { *o = __float2bfloat16(v); }

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {  // of a uniform lane
  const int lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// W: waves of a block.  ONE: each cache head has one query, which then stands in all 16 columns of the scores, and
// every lane has the probabilities of its own four tokens: the second product is D / 16 multiply-adds a token on
// the vector ALU, a quarter of the time that the matrix cores would take for 16 columns.
template <int D, typename X, bool INT8, bool ONE, int W>
__global__ __launch_bounds__(64 * W, 2) void attention_kernel(Args a) {
  constexpr int NP = sizeof(X) == 2 ? 1 : 3;  // bf16 pieces of a query
  constexpr int kF = D / 32;                  // operands of the score product
  constexpr int kE = D / 16;
  constexpr int kElem = INT8 ? 1 : 2;
  constexpr int kU = 2;  // tiles at a time
  constexpr int NV = 3;  // bf16 pieces of a probability
  constexpr int kRowsOut = ONE ? 1 : kTile;
  __shared__ float red_o[W][kRowsOut][D + 4];
  __shared__ float red_m[W][kRowsOut], red_l[W][kRowsOut];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  uint32_t id = blockIdx.x;
  const uint32_t q_tile = id % a.q_tiles;
  id /= a.q_tiles;
  const uint32_t h = id % a.heads;
  const uint32_t number = id / a.heads;
  const Part part = find_part<true>(a, (int)number);
  if (part.b < 0) return;
  const uint32_t b = (uint32_t)part.b;
  const uint32_t q0 = q_tile * kTile;
  const int queries = ONE ? 1 : (int)(a.share - q0 < kTile ? a.share - q0 : kTile);
  const Span sp = part.span;
  const int first = sp.first + part.index * part.per_part;
  const int last = first + part.per_part < sp.last ? first + part.per_part : sp.last;

  // Lane i knows where tile i of the wave's next 64 begins: offsets from the cache's start, -1 where there is no page.
  const uint32_t tiles_per_page = a.page_size / kTile;
  const int32_t* const table = a.table + (int64_t)b * a.ld_table;
  const int mine_first = first + wave * kU;
  const int units = mine_first < last ? (last - mine_first + W * kU - 1) / (W * kU) : 0;
  int64_t at = -1, scale_at = 0;
  auto look_up = [&](int unit) {
    const int tile = mine_first + (unit + lane / kU) * (W * kU) + lane % kU;
    at = -1;
    if (tile < last) {
      const uint32_t entry = (uint32_t)tile / tiles_per_page, slot = ((uint32_t)tile % tiles_per_page) * kTile;
      const int64_t page = table[entry];
      if (page >= 0 && page < a.num_pages) {
        at = page * a.page_stride + h * a.head_stride + (int64_t)slot * a.token_stride;
        scale_at = (page * a.heads + h) * a.page_size + slot;
      }
    }
  };

  const int mine = r < queries ? r : queries - 1;
  bf16x8 q[kF][NP];
  {
    const X* row = static_cast<const X*>(a.q) + b * a.q_ts + (int64_t)(h * a.share + q0 + mine) * a.q_hs;
#pragma unroll
    for (int f = 0; f < kF; ++f) {
      const X* p = row + Keys<D, INT8>::channel(f, c);
      if constexpr (NP == 1) {
        q[f][0] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(p));
      } else {
        f32x4 v[2] = {reinterpret_cast<const f32x4*>(p)[0], reinterpret_cast<const f32x4*>(p)[1]};
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          u32x4 o;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const float x = v[s >> 1][2 * (s & 1)], y = v[s >> 1][2 * (s & 1) + 1];
            o[s] = __builtin_amdgcn_perm(float_bits(y), float_bits(x), 0x07060302u);
            v[s >> 1][2 * (s & 1)] = x - bits_float(float_bits(x) & 0xFFFF0000u);
            v[s >> 1][2 * (s & 1) + 1] = y - bits_float(float_bits(y) & 0xFFFF0000u);
          }
          q[f][n] = __builtin_bit_cast(bf16x8, o);
        }
      }
    }
  }

  Keys<D, INT8> k[kU];
  Values<D, INT8> v[kU][4];
  f32x4 ks[kU], vs[kU];
  const uint32_t token_bytes = a.token_stride * kElem;
  const uint32_t key_lane = r * token_bytes + 16 * c, value_lane = r * Values<D, INT8>::kBytes;
  auto edge = [&](int tile) { return tile * kTile < sp.begin || tile * kTile + kTile > sp.end; };
  // Tokens before `begin` and from `end` on are not read: their lanes read the nearest one inside.
  auto inside = [&](int tile, int t) {
    const int lo = sp.begin - tile * kTile, hi = sp.end - 1 - tile * kTile;
    return (uint32_t)(t < lo ? lo : (t > hi ? hi : t));
  };
  auto load_keys = [&](int u, int tile, int64_t at_u, int64_t scale_u) {
    uint32_t lane_bytes = key_lane;
    if (edge(tile)) lane_bytes = inside(tile, r) * token_bytes + 16 * c;
    k[u].load(a.kp + at_u * kElem, lane_bytes);
    if constexpr (INT8) ks[u] = *reinterpret_cast<const f32x4*>(a.ks + scale_u + 4 * c);
  };
  auto load_values = [&](int u, int tile, int64_t at_u, int64_t scale_u) {
    uint32_t lane_bytes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) lane_bytes[i] = (4 * c + i) * token_bytes + value_lane;
    if (edge(tile)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lane_bytes[i] = inside(tile, 4 * c + i) * token_bytes + value_lane;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[u][i].load(a.vp + at_u * kElem, lane_bytes[i]);
    if constexpr (INT8) vs[u] = *reinterpret_cast<const f32x4*>(a.vs + scale_u + 4 * c);
  };

  f32x4 o[ONE ? 1 : kE];
  float o1[ONE ? kE : 1];
  if constexpr (ONE) {
#pragma unroll
    for (int e = 0; e < kE; ++e) o1[e] = 0.0f;
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = f32x4{0, 0, 0, 0};
  }
  float m = kLowest, l = 0.0f;  // of query r; l of this lane's tokens

  int64_t here[kU], next[kU], scale_next[kU];
  if (units > 0) {
    look_up(0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      here[u] = lane_value(at, u);
      const int64_t sc = INT8 ? lane_value(scale_at, u) : 0;
      if (here[u] >= 0) {
        load_keys(u, mine_first + u, here[u], sc);
        load_values(u, mine_first + u, here[u], sc);
      }
    }
  }
  for (int unit = 0; unit < units; ++unit) {
    const int tile0 = mine_first + unit * (W * kU), tile1 = tile0 + W * kU;
    const bool more = unit + 1 < units;
    float s[kU][4];  // -inf: the token takes no part
    float top = m;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (here[u] < 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] = -INFINITY;
        continue;
      }
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int f = 0; f < kF; ++f) {
        const bf16x8 kf = k[u].operand(f);
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[f][n], acc, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u][i] = INT8 ? acc[i] * (a.scale * ks[u][i]) : acc[i] * a.scale;
      const int t0 = (tile0 + u) * kTile;
      if (edge(tile0 + u)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[u][i] = t0 + 4 * c + i >= sp.begin && t0 + 4 * c + i < sp.end ? s[u][i] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[u][i]);
    }
    // The next unit's keys are on their way while this one's probabilities and sums are formed.
    if (more) {
      if (((unit + 1) * kU) % 64 == 0) look_up(unit + 1);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = ((unit + 1) * kU + u) % 64;
        next[u] = lane_value(at, i);
        scale_next[u] = INT8 ? lane_value(scale_at, i) : 0;
        if (next[u] >= 0) load_keys(u, tile1 + u, next[u], scale_next[u]);
      }
    }
    if (__any(top > m)) {  // otherwise the maxima stand
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float shrink = exp2_raw(m - top);
      m = top;
      l *= shrink;
      if constexpr (ONE) {
#pragma unroll
        for (int e = 0; e < kE; ++e) o1[e] *= shrink;
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[e][i] *= shrink;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float p = exp2_raw(s[u][i] - m);
        l += p;
        if constexpr (INT8) p = s[u][i] != -INFINITY ? p * vs[u][i] : 0.0f;  // behind a sequence's end a scale may be anything
        s[u][i] = p;
      }
      if (here[u] < 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i].clear();
      }
    }
    if constexpr (ONE) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < kE; ++e) o1[e] = fmaf(v[u][i].get(e), s[u][i], o1[e]);
    } else {
      bf16x8 p[NV];  // slots 8 c + 4 u + i of the sum: token 4 c + i of tile u
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        u32x4 w;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          float &x = s[z >> 1][2 * (z & 1)], &y = s[z >> 1][2 * (z & 1) + 1];
          w[z] = __builtin_amdgcn_perm(float_bits(y), float_bits(x), 0x07060302u);
          x -= bits_float(float_bits(x) & 0xFFFF0000u);
          y -= bits_float(float_bits(y) & 0xFFFF0000u);
        }
        p[n] = __builtin_bit_cast(bf16x8, w);
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        u32x4 w;
#pragma unroll
        for (int z = 0; z < 4; ++z) w[z] = Values<D, INT8>::pair(v[z >> 1][2 * (z & 1)], v[z >> 1][2 * (z & 1) + 1], e);
        const bf16x8 vf = __builtin_bit_cast(bf16x8, w);
#pragma unroll
        for (int n = NV - 1; n >= 0; --n) o[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, p[n], o[e], 0, 0, 0);
      }
    }
    if (more) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (next[u] >= 0) load_values(u, tile1 + u, next[u], scale_next[u]);
        here[u] = next[u];
      }
    }
  }

  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (c == 0 && r < kRowsOut) {
    red_m[wave][r] = m;
    red_l[wave][r] = l;
  }
  if constexpr (ONE) {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      o1[e] += __shfl_xor(o1[e], 16);
      o1[e] += __shfl_xor(o1[e], 32);
      if (c == 0) red_o[wave][0][kE * r + e] = o1[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) red_o[wave][r][kE * (4 * c + i) + e] = o[e][i];
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < queries * D; idx += 64 * W) {
    const int j = idx / D, d = idx % D;
    float top = red_m[0][j];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, red_m[w][j]);
    float sum = 0.0f, val = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = exp2_raw(red_m[w][j] - top);
      sum += f * red_l[w][j];
      val += f * red_o[w][j][d];
    }
    const uint32_t head = h * a.share + q0 + j;
    if (part.count == 1) {
      store(static_cast<X*>(a.o) + b * a.o_ts + (int64_t)head * a.o_hs + d, sum == 0.0f ? 0.0f : val / sum);
    } else {
      const int64_t to = (int64_t)number * a.q_heads + head;
      a.partial[to * D + d] = val;
      if (d == 0) {
        float* ml = a.partial + (int64_t)a.parts * a.q_heads * D + 2 * to;
        ml[0] = top;
        ml[1] = sum;
      }
    }
  }
}

// Parts joined: one block of W waves to a query head.  Every wave weighs all parts by itself (lane p of 64 at a time), adds
// every W-th of them, and the waves' sums meet once in LDS.
template <int D, typename X, int W>
__global__ __launch_bounds__(64 * W) void join_kernel(Args a) {
  constexpr int kPer = D / 64;  // channels of a lane
  __shared__ float sums[W][D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t b = blockIdx.x / a.q_heads, head = blockIdx.x % a.q_heads;
  const Part part = find_part<false>(a, (int)b);
  const int parts = part.count;
  if (parts == 1) return;  // its one block has written the result
  const int64_t at = (int64_t)part.first_of * a.q_heads + head;
  const int64_t step = a.q_heads;
  const float* const ml = a.partial + (int64_t)a.parts * a.q_heads * D + 2 * at;
  const float* const val = a.partial + at * D + kPer * lane;

  float m = kLowest, l = 0.0f, o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
  for (int first = 0; first < parts; first += 64) {
    const int p = first + lane, n = parts - first < 64 ? parts - first : 64;
    const float pm = p < parts ? ml[2 * p * step] : kLowest, pl = p < parts ? ml[2 * p * step + 1] : 0.0f;
    float part_o[64 / W][kPer];  // on their way while the weights are formed
#pragma unroll
    for (int i = 0; i < 64 / W; ++i) {
      const int q = i * W + wave;
      if (q >= n) break;
#pragma unroll
      for (int e = 0; e < kPer; ++e) part_o[i][e] = val[(first + q) * step * D + e];
    }
    float top = fmaxf(m, pm);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float shrink = exp2_raw(m - top), weight = p < parts ? exp2_raw(pm - top) : 0.0f;
    m = top;
    l = l * shrink + weight * pl;  // of this lane's parts
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] *= shrink;
#pragma unroll
    for (int i = 0; i < 64 / W; ++i) {
      const int q = i * W + wave;
      if (q >= n) break;
      const float w = bits_float(__builtin_amdgcn_readlane(float_bits(weight), q));
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] += w * part_o[i][e];
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
#pragma unroll
  for (int i = 0; i < kPer; ++i) sums[wave][kPer * lane + i] = o[i];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 64 * W) {
    float x = sums[0][d];
#pragma unroll
    for (int w = 1; w < W; ++w) x += sums[w][d];
    store(static_cast<X*>(a.o) + b * a.o_ts + (int64_t)head * a.o_hs + d, l == 0.0f ? 0.0f : x / l);
  }
}

template <int D, typename X, bool INT8>
hipError_t launch(Args a, bool split, hipStream_t st) {
  void (*const kernel)(Args) =
      a.share == 1 ? attention_kernel<D, X, INT8, true, kWaves> : attention_kernel<D, X, INT8, false, kWaves>;
  static std::atomic<int> resident_blocks[2];  // on a CU, by kernel; 0: not asked for yet; every device is alike
  std::atomic<int>& resident = resident_blocks[a.share == 1];
  int n = resident.load(std::memory_order_relaxed);
  if (n == 0) {
    const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 64 * kWaves, 0);
    if (e != hipSuccess) return e;
    n = n < 1 ? 1 : (n > kMaxResident ? kMaxResident : n);
    resident.store(n, std::memory_order_relaxed);
  }
  // One round of blocks, less half a part a sequence, since the last part of each is half full on average.
  const int64_t each = (int64_t)a.heads * a.q_tiles, round = (int64_t)n * kCUs / each;
  a.few = round - a.B / 2 > round / 2 ? round - a.B / 2 : round / 2;
  if (a.few < 1) a.few = 1;
  const unsigned blocks = a.parts * a.heads * a.q_tiles;
  kernel<<<blocks, 64 * kWaves, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !split) return e;
  // Many heads fill the chip with two waves each; few heads have many parts, which eight waves read at once (us, two and
  // eight waves: ragged batch 60.1 and 60.9, large batch 270.4 and 272.4, long int8 60.1 and 49.9).
  if (a.B * a.q_heads > 2 * kCUs)
    join_kernel<D, X, 2><<<a.B * a.q_heads, 128, 0, st>>>(a);
  else
    join_kernel<D, X, 8><<<a.B * a.q_heads, 512, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_attention(const AttentionArgs& in, hipStream_t st) {
  const qv_kv_cache& c = in.cache;
  Args a = {};
  a.q = in.Q.data;
  a.o = const_cast<void*>(in.O.data);
  a.kp = static_cast<const char*>(c.k_pages);
  a.vp = static_cast<const char*>(c.v_pages);
  a.ks = c.k_scale;
  a.vs = c.v_scale;
  a.table = in.page_table;
  a.lens = in.lens;
  a.partial = in.partial;
  a.q_ts = in.Q.token_stride;
  a.q_hs = in.Q.head_stride;
  a.o_ts = in.O.token_stride;
  a.o_hs = in.O.head_stride;
  a.page_stride = c.page_stride;
  a.head_stride = c.head_stride;
  a.ld_table = in.ld_table;
  a.num_pages = c.num_pages;
  a.capacity = (int32_t)(in.max_pages * c.page_size);
  a.window = in.window > 0x7fffffff ? 0 : (int32_t)in.window;
  a.B = (uint32_t)in.B;
  a.heads = (uint32_t)c.heads;
  a.q_heads = (uint32_t)in.q_heads;
  a.share = (uint32_t)(in.q_heads / c.heads);
  a.q_tiles = (a.share + kTile - 1) / kTile;
  const AttentionParts parts = paged_attention_parts(in.B, in.q_heads, c.heads, a.capacity);
  a.many = parts.many;
  a.few_tiles = (in.max_pages * c.page_size + kTile) / kTile * in.B < (int64_t{1} << 31) - kManyBlocks;
  a.parts = (uint32_t)parts.most;
  a.token_stride = (uint32_t)c.token_stride;
  a.page_size = (uint32_t)c.page_size;
  a.scale = in.scale * kLog2e;
  const bool q8 = c.dtype == QV_KV_INT8;
  if (c.head_dim == 64) {
    if (in.bf16)
      return q8 ? launch<64, __hip_bfloat16, true>(a, parts.split, st)
                : launch<64, __hip_bfloat16, false>(a, parts.split, st);
    return q8 ? launch<64, float, true>(a, parts.split, st) : launch<64, float, false>(a, parts.split, st);
  }
  if (in.bf16)
    return q8 ? launch<128, __hip_bfloat16, true>(a, parts.split, st)
              : launch<128, __hip_bfloat16, false>(a, parts.split, st);
  return q8 ? launch<128, float, true>(a, parts.split, st) : launch<128, float, false>(a, parts.split, st);
}

}  // namespace qv
