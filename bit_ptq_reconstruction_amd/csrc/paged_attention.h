// paged_attention.h -- the attention of a few rows over a paged cache: one new token of every sequence (paged_attention.hip)
// and short runs of them (run_attention.hip).  paged_attention.hip says how it works.
#pragma once
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
constexpr int kBf16 = QV_KV_BF16, kInt8 = QV_KV_INT8, kFp8 = QV_KV_FP8;  // what a cache holds
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
  uint32_t scale_tokens;  // of a scale (FP8 caches)
  // Runs of tokens (RUN); without `starts` each sequence has one.
  const int32_t* starts;
  int32_t T, sinks, causal;
  uint32_t max_run;
};

// A sequence's run of tokens: rows s0 .. s0 + n - 1 of Q, which are its last n.
struct Run {
  int s0, n;
};
__device__ __forceinline__ Run run_of(const Args& a, int b) {
  if (!a.starts) return {b, 1};
  int s0 = a.starts[b], s1 = a.starts[b + 1];
  s0 = s0 < 0 ? 0 : (s0 > a.T ? a.T : s0);
  s1 = s1 < s0 ? s0 : (s1 > a.T ? a.T : s1);
  return {s0, s1 - s0 < (int)a.max_run ? s1 - s0 : (int)a.max_run};
}

__device__ __forceinline__ float bits_float(unsigned u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ unsigned float_bits(float f) { return __builtin_bit_cast(unsigned, f); }

// Tokens [begin, end) that a sequence attends to and their tiles [first, last); places are counted in 31 bits.
// RUN: the tokens that any query of the run sees, [0, sinks) and [begin, end).  Tiles are then counted without those between:
// number v is tile v up to `near`, and v + skip from there on.
struct Span {
  int begin, end, first, last;
  int sinks, near, skip;
  __device__ __forceinline__ int tile(int v) const { return v < near ? v : v + skip; }
};
template <bool RUN>
__device__ __forceinline__ Span span_of(const Args& a, int n, int b) {
  Span s;
  s.end = n < 0 ? 0 : (n > a.capacity ? a.capacity : n);
  if constexpr (!RUN) {
    s.begin = a.window > 0 && s.end > a.window ? s.end - a.window : 0;
    s.first = s.begin / kTile;
    s.last = (s.end + kTile - 1) / kTile;
    s.sinks = s.near = s.skip = 0;
  } else {
    const int run = run_of(a, b).n;
    const int64_t low = (int64_t)s.end - run - a.window + 1;  // of the first query's window
    s.begin = a.window > 0 && low > 0 ? (int)low : 0;
    s.sinks = a.sinks < s.end ? a.sinks : s.end;
    s.near = (s.sinks + kTile - 1) / kTile;
    s.skip = s.begin / kTile > s.near ? s.begin / kTile - s.near : 0;
    s.first = 0;
    s.last = run > 0 ? (s.end + kTile - 1) / kTile - s.skip : 0;
  }
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
template <bool BY_PART, bool RUN>
__device__ __forceinline__ Part find_part(const Args& a, int which) {
  const int lane = threadIdx.x & 63, B = (int)a.B;
  Part p;
  const int mine = lane < B ? a.lens[lane] : 0;  // of the first 64 sequences
  const Span own = span_of<RUN>(a, mine, lane < B ? lane : 0);
  if (B <= 64 && a.few_tiles) {  // the totals fit 32 bits
    const uint32_t total = __builtin_amdgcn_readlane(scan(own.last - own.first), 63);
    p.per_part = __builtin_amdgcn_readfirstlane(tiles_of_part(total, (uint32_t)a.few, (uint32_t)a.many));
  } else {
    uint64_t total = own.last - own.first;
    for (int i = lane + 64; i < B; i += 64) {
      const Span s = span_of<RUN>(a, a.lens[i], i);
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
    const Span s = first == 0 ? own : span_of<RUN>(a, n, i < B ? i : 0);
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
      p.span = span_of<RUN>(a, __builtin_amdgcn_readlane(n, at), first + at);
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

// Two signed bytes of a dword (its low or high half) as a bf16 pair, exactly.
template <bool HIGH>
__device__ __forceinline__ unsigned pair_of_bytes(unsigned w) {
  const float x = HIGH ? signed_byte<2>(w) : signed_byte<0>(w), y = HIGH ? signed_byte<3>(w) : signed_byte<1>(w);
  return __builtin_amdgcn_perm(float_bits(y), float_bits(x), 0x07060302u);
}

// Two 8-bit floating-point codes of a dword (its low or high half) as a bf16 pair.
template <bool HIGH>
__device__ __forceinline__ unsigned pair_of_codes(unsigned w) {
  return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}

// RUN: several blocks read the same tokens one behind the other, so these stay in the cache.
template <bool RUN, typename T>
__device__ __forceinline__ T load_once(const char* p) {
  return RUN ? *reinterpret_cast<const T*>(p) : __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
}

// Keys of one tile as loaded, and as operands of the score product.
template <int D, int KIND, bool RUN>
struct Keys {
  static constexpr bool kBytes = KIND != kBf16;
  static constexpr int kLoads = kBytes ? D / 64 : D / 32;
  u32x4 d[kLoads];
  __device__ __forceinline__ void load(const char* tile, uint32_t lane_bytes) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      d[j] = load_once<RUN, u32x4>(tile + lane_bytes + 64 * j);
  }
  // operand f covers channels channel(f, c) .. + 7
  static __device__ __forceinline__ int channel(int f, int c) {
    return kBytes ? 64 * (f >> 1) + 16 * c + 8 * (f & 1) : 32 * f + 8 * c;
  }
  __device__ __forceinline__ bf16x8 operand(int f) const {
    if constexpr (KIND == kBf16) {
      return __builtin_bit_cast(bf16x8, d[f]);
    } else if constexpr (KIND == kFp8) {
      const unsigned w0 = d[f >> 1][2 * (f & 1)], w1 = d[f >> 1][2 * (f & 1) + 1];
      return __builtin_bit_cast(bf16x8, u32x4{pair_of_codes<false>(w0), pair_of_codes<true>(w0), pair_of_codes<false>(w1),
                                              pair_of_codes<true>(w1)});
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
template <int D, int KIND, bool RUN>
struct Values {
  static constexpr int kE = D / 16;
  static constexpr int kBytes = kE * (KIND != kBf16 ? 1 : 2);
  static constexpr int kWords = kBytes / 4;
  unsigned d[kWords];
  __device__ __forceinline__ void load(const char* tile, uint32_t lane_bytes) {
    const char* const p = tile + lane_bytes;
    if constexpr (kWords == 4) {
      const u32x4 v = load_once<RUN, u32x4>(p);
      d[0] = v[0], d[1] = v[1], d[2] = v[2], d[3] = v[3];
    } else if constexpr (kWords == 2) {
      const u32x2 v = load_once<RUN, u32x2>(p);
      d[0] = v[0], d[1] = v[1];
    } else {
      d[0] = load_once<RUN, unsigned>(p);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) d[i] = 0;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (KIND == kFp8) {
      const unsigned w = d[e >> 2];
      return (e & 3) == 0   ? __builtin_amdgcn_cvt_f32_fp8(w, 0)
             : (e & 3) == 1 ? __builtin_amdgcn_cvt_f32_fp8(w, 1)
             : (e & 3) == 2 ? __builtin_amdgcn_cvt_f32_fp8(w, 2)
                            : __builtin_amdgcn_cvt_f32_fp8(w, 3);
    } else if constexpr (KIND == kInt8) {
      const unsigned w = d[e >> 2];
      return (e & 3) == 0 ? signed_byte<0>(w) : (e & 3) == 1 ? signed_byte<1>(w) : (e & 3) == 2 ? signed_byte<2>(w)
                                                                                                : signed_byte<3>(w);
    }
    return (e & 1) ? bits_float(d[e >> 1] & 0xFFFF0000u) : bits_float(d[e >> 1] << 16);
  }
  // Whether one of them is not finite.
  __device__ __forceinline__ bool odd() const {
    bool any = false;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (KIND == kFp8) {  // NaN is 0x7F with either sign, and there are no infinities
        const unsigned w = (d[i] & 0x7F7F7F7Fu) + 0x01010101u;
        any |= (w & 0x80808080u) != 0;
      } else {
        any |= (d[i] & 0x7F80u) == 0x7F80u || (d[i] & 0x7F800000u) == 0x7F800000u;
      }
    }
    return any;
  }
  // Channel d of the token whose value is at `row`.
  static __device__ __forceinline__ float of(const char* row, int d) {
    if constexpr (KIND == kFp8) return __builtin_amdgcn_cvt_f32_fp8((unsigned)(uint8_t)row[d], 0);
    return bits_float((unsigned)reinterpret_cast<const uint16_t*>(row)[d] << 16);
  }
  // Channel e of two tokens as a bf16 pair.
  static __device__ __forceinline__ unsigned pair(const Values& a, const Values& b, int e) {
    if constexpr (KIND == kInt8) return __builtin_amdgcn_perm(float_bits(b.get(e)), float_bits(a.get(e)), 0x07060302u);
    if constexpr (KIND == kFp8) {  // codes of channels e and e + 1 (e even) side by side; the permutation serves both
      const unsigned w = __builtin_amdgcn_perm(b.d[e >> 2], a.d[e >> 2], (e & 2) ? 0x07030602u : 0x05010400u);
      return (e & 1) ? pair_of_codes<true>(w) : pair_of_codes<false>(w);
    }
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
//
// RUN: a sequence has up to max_run new tokens, and the rows that share a cache head are its tokens' query heads, token
// by token.  Each row sees its own part of the sequence's span: what another row sees is read and masked.
template <int D, typename X, int KIND, bool ONE, int W, bool RUN>
__global__ __launch_bounds__(64 * W, 2) void attention_kernel(Args a) {
  constexpr int NP = sizeof(X) == 2 ? 1 : 3;  // bf16 pieces of a query
  constexpr int kF = D / 32;                  // operands of the score product
  constexpr int kE = D / 16;
  constexpr bool INT8 = KIND == kInt8, FP8 = KIND == kFp8;
  constexpr int kElem = KIND == kBf16 ? 2 : 1;
  constexpr int kU = 2;  // tiles at a time
  constexpr int NV = 3;  // bf16 pieces of a probability
  constexpr int kRowsOut = ONE ? 1 : kTile;
  __shared__ float red_o[W][kRowsOut][D + 4];
  __shared__ float red_m[W][kRowsOut], red_l[W][kRowsOut];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  uint32_t id = blockIdx.x, q_tile;
  if constexpr (RUN) {  // blocks are dealt out to eight dies in turn: the tiles of a part and head, which read the same, go to one
    const uint32_t lot = id / (8 * a.q_tiles), in_lot = id % (8 * a.q_tiles);
    q_tile = in_lot / 8;
    id = 8 * lot + in_lot % 8;
  } else {
    q_tile = id % a.q_tiles;
    id /= a.q_tiles;
  }
  const uint32_t h = id % a.heads;
  const uint32_t number = id / a.heads;
  const Part part = find_part<true, RUN>(a, (int)number);
  if (part.b < 0) return;
  const uint32_t b = (uint32_t)part.b;
  const uint32_t q0 = q_tile * kTile;
  const Run run = RUN ? run_of(a, (int)b) : Run{(int)b, 1};
  const uint32_t rows = RUN ? run.n * a.share : a.share;
  if (RUN && q0 >= rows) return;
  const int queries = ONE ? 1 : (int)(rows - q0 < kTile ? rows - q0 : kTile);
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
    int tile = mine_first + (unit + lane / kU) * (W * kU) + lane % kU;
    at = -1;
    if (tile < last) {
      if constexpr (RUN) tile = sp.tile(tile);
      const uint32_t entry = (uint32_t)tile / tiles_per_page, slot = ((uint32_t)tile % tiles_per_page) * kTile;
      const int64_t page = table[entry];
      if (page >= 0 && page < a.num_pages) {
        at = page * a.page_stride + h * a.head_stride + (int64_t)slot * a.token_stride;
        if constexpr (FP8)
          scale_at = (page * a.heads + h) * (a.page_size / a.scale_tokens) + slot / a.scale_tokens;
        else
          scale_at = (page * a.heads + h) * a.page_size + slot;
      }
    }
  };

  const int mine = r < queries ? r : queries - 1;
  bf16x8 q[kF][NP];
  // RUN: query r sees [0, sinks) and [low, high).
  int low = 0, high = 0;
  {
    uint32_t token = 0, head = q0 + mine;
    if constexpr (RUN) {
      token = head / a.share;
      head -= token * a.share;
      const int place = sp.end - run.n + (int)token;  // negative where the run is longer than its sequence
      high = a.causal && place + 1 < sp.end ? place + 1 : sp.end;
      low = a.window > 0 && place >= a.window ? place - a.window + 1 : 0;
    }
    const X* row = static_cast<const X*>(a.q) + (int64_t)(run.s0 + token) * a.q_ts + (int64_t)(h * a.share + head) * a.q_hs;
#pragma unroll
    for (int f = 0; f < kF; ++f) {
      const X* p = row + Keys<D, KIND, RUN>::channel(f, c);
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

  Keys<D, KIND, RUN> k[kU];
  Values<D, KIND, RUN> v[kU][4];
  f32x4 ks[kU], vs[kU];
  float ks1[kU], vs1[kU];  // FP8: of the tile's block
  const uint32_t token_bytes = a.token_stride * kElem;
  const uint32_t key_lane = r * token_bytes + 16 * c, value_lane = r * Values<D, KIND, RUN>::kBytes;
  // Of tile number v: whether there is a token in it that some row does not see.
  const int all_low = RUN && a.window > 0 ? sp.end - a.window : sp.begin, all_high = RUN && a.causal ? sp.end - run.n + 1 : sp.end;
  auto edge = [&](int v) {
    const int tile = RUN ? sp.tile(v) : v;
    return tile * kTile < all_low || tile * kTile + kTile > all_high;
  };
  // Tokens that no row sees are not read: their lanes read the nearest one inside.
  auto inside = [&](int v, int t) {
    const int tile = RUN ? sp.tile(v) : v;
    const int lo = sp.begin - tile * kTile, hi = sp.end - 1 - tile * kTile;
    t = t > hi ? hi : t;
    if constexpr (RUN) {
      const int sinks = sp.sinks - tile * kTile;
      return (uint32_t)(t < lo && t >= sinks ? (sinks > 0 ? sinks - 1 : lo) : t);
    }
    return (uint32_t)(t < lo ? lo : t);
  };
  auto sees = [&](int t) { return t < high && (t >= low || t < a.sinks); };  // RUN
  auto load_keys = [&](int u, int tile, int64_t at_u, int64_t scale_u) {
    uint32_t lane_bytes = key_lane;
    if (edge(tile)) lane_bytes = inside(tile, r) * token_bytes + 16 * c;
    k[u].load(a.kp + at_u * kElem, lane_bytes);
    if constexpr (INT8) ks[u] = *reinterpret_cast<const f32x4*>(a.ks + scale_u + 4 * c);
    if constexpr (FP8) ks1[u] = a.ks[scale_u];
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
    if constexpr (FP8) vs1[u] = a.vs[scale_u];
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
  float s[kU][4];  // scores (-inf: the token takes no part), then probabilities
  // RUN: a value that is not finite would reach the rows that do not see its token through their zero probabilities.
  // Such tokens are taken out of the second product and added to the rows that see them alone.
  auto take_out = [&](int tile0) {
    if constexpr (RUN && !ONE && KIND != kInt8) {
      bool odd = false;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (here[u] >= 0 && edge(tile0 + u)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) odd |= v[u][i].odd();
        }
      if (!__any(odd)) return;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (here[u] < 0 || !edge(tile0 + u)) continue;
        const int t0 = sp.tile(tile0 + u) * kTile;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t lanes = __ballot(v[u][i].odd());
          if ((lanes >> (16 * c)) & 0xFFFF) v[u][i].clear();
          for (int g = 0; g < 4; ++g) {  // token 4 g + i
            if (!((lanes >> (16 * g)) & 0xFFFF)) continue;
            const float p = __shfl(s[u][i], 16 * g + r);
            const char* const row = a.vp + here[u] * kElem + inside(tile0 + u, 4 * g + i) * (uint64_t)token_bytes;
            if (!sees(t0 + 4 * g + i)) continue;
#pragma unroll
            for (int e = 0; e < kE; ++e)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[e][j] = fmaf(Values<D, KIND, RUN>::of(row, kE * (4 * c + j) + e), p, o[e][j]);
          }
        }
      }
    }
  };
  if (units > 0) {
    look_up(0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      here[u] = lane_value(at, u);
      const int64_t sc = KIND != kBf16 ? lane_value(scale_at, u) : 0;
      if (here[u] >= 0) {
        load_keys(u, mine_first + u, here[u], sc);
        load_values(u, mine_first + u, here[u], sc);
      }
    }
  }
  for (int unit = 0; unit < units; ++unit) {
    const int tile0 = mine_first + unit * (W * kU), tile1 = tile0 + W * kU;
    const bool more = unit + 1 < units;
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
      for (int i = 0; i < 4; ++i)
        s[u][i] = INT8 ? acc[i] * (a.scale * ks[u][i]) : (FP8 ? acc[i] * (a.scale * ks1[u]) : acc[i] * a.scale);
      const int t0 = (RUN ? sp.tile(tile0 + u) : tile0 + u) * kTile;
      if (edge(tile0 + u)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 4 * c + i;
          s[u][i] = (RUN ? sees(t) : t >= sp.begin && t < sp.end) ? s[u][i] : -INFINITY;
        }
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
        scale_next[u] = KIND != kBf16 ? lane_value(scale_at, i) : 0;
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
        if constexpr (FP8) p = s[u][i] != -INFINITY ? p * vs1[u] : 0.0f;
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
      if constexpr (RUN && KIND != kInt8) {
        if (a.max_run > 1) take_out(tile0);
      }
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
        for (int z = 0; z < 4; ++z) w[z] = Values<D, KIND, RUN>::pair(v[z >> 1][2 * (z & 1)], v[z >> 1][2 * (z & 1) + 1], e);
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
    uint32_t token = 0, head = q0 + j;
    if constexpr (RUN) {
      token = head / a.share;
      head -= token * a.share;
    }
    head += h * a.share;
    if (part.count == 1) {
      store(static_cast<X*>(a.o) + (int64_t)(run.s0 + token) * a.o_ts + (int64_t)head * a.o_hs + d, sum == 0.0f ? 0.0f : val / sum);
    } else {
      const int64_t rows_of_part = RUN ? (int64_t)a.q_heads * a.max_run : a.q_heads;
      const int64_t to = number * rows_of_part + token * a.q_heads + head;
      a.partial[to * D + d] = val;
      if (d == 0) {
        float* ml = a.partial + a.parts * rows_of_part * D + 2 * to;
        ml[0] = top;
        ml[1] = sum;
      }
    }
  }
}

// Parts joined: one block of W waves to a query head of a token.  Every wave weighs all parts by itself (lane p of 64 at a time), adds
// every W-th of them, and the waves' sums meet once in LDS.
template <int D, typename X, int W, bool RUN>
__global__ __launch_bounds__(64 * W) void join_kernel(Args a) {
  constexpr int kPer = D / 64;  // channels of a lane
  __shared__ float sums[W][D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t step = RUN ? a.q_heads * a.max_run : a.q_heads;
  const uint32_t b = blockIdx.x / step, row = blockIdx.x % step, token = RUN ? row / a.q_heads : 0, head = row - token * a.q_heads;
  const Part part = find_part<false, RUN>(a, (int)b);
  const int parts = part.count;
  if (parts == 1) return;  // its one block has written the result
  const Run run = RUN ? run_of(a, (int)b) : Run{(int)b, 1};
  if (RUN && (int)token >= run.n) return;
  const int64_t at = (int64_t)part.first_of * step + row;
  const float* const ml = a.partial + (int64_t)a.parts * step * D + 2 * at;
  const float* const val = a.partial + at * D + kPer * lane;

  float m = kLowest, l = 0.0f, o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
  for (int first = 0; first < parts; first += 64) {
    const int p = first + lane, n = parts - first < 64 ? parts - first : 64;
    const float pm = p < parts ? ml[(int64_t)2 * p * step] : kLowest, pl = p < parts ? ml[(int64_t)2 * p * step + 1] : 0.0f;
    float part_o[64 / W][kPer];  // on their way while the weights are formed
#pragma unroll
    for (int i = 0; i < 64 / W; ++i) {
      const int q = i * W + wave;
      if (q >= n) break;
#pragma unroll
      for (int e = 0; e < kPer; ++e) part_o[i][e] = val[(int64_t)(first + q) * step * D + e];
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
    store(static_cast<X*>(a.o) + (int64_t)(run.s0 + token) * a.o_ts + (int64_t)head * a.o_hs + d, l == 0.0f ? 0.0f : x / l);
  }
}

template <int D, typename X, int KIND, bool RUN>
hipError_t launch(Args a, bool split, hipStream_t st) {
  void (*const kernel)(Args) =
      a.share * a.max_run == 1 ? attention_kernel<D, X, KIND, true, kWaves, RUN> : attention_kernel<D, X, KIND, false, kWaves, RUN>;
  static std::atomic<int> resident_blocks[2];  // on a CU, by kernel; 0: not asked for yet; every device is alike
  std::atomic<int>& resident = resident_blocks[a.share * a.max_run == 1];
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
  const unsigned each_tile = a.parts * a.heads, blocks = (RUN ? (each_tile + 7) / 8 * 8 : each_tile) * a.q_tiles;
  kernel<<<blocks, 64 * kWaves, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !split) return e;
  // Many heads fill the chip with two waves each; few heads have many parts, which eight waves read at once (us, two and
  // eight waves: ragged batch 60.1 and 60.9, large batch 270.4 and 272.4, long int8 60.1 and 49.9).
  const unsigned rows = a.B * a.q_heads * a.max_run;
  if (rows > 2 * kCUs)
    join_kernel<D, X, 2, RUN><<<rows, 128, 0, st>>>(a);
  else
    join_kernel<D, X, 8, RUN><<<rows, 512, 0, st>>>(a);
  return hipGetLastError();
}

// The kernels' arguments, for runs of up to `max_run` tokens of each sequence.
Args arguments(const AttentionArgs& in, int64_t max_run, bool* split) {
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
  a.max_run = (uint32_t)max_run;
  a.q_tiles = (a.share * a.max_run + kTile - 1) / kTile;
  const AttentionParts parts = paged_attention_parts(in.B, in.q_heads * max_run, c.heads, a.capacity);
  *split = parts.split;
  a.many = parts.many;
  a.few_tiles = (in.max_pages * c.page_size + kTile) / kTile * in.B < (int64_t{1} << 31) - kManyBlocks;
  a.parts = (uint32_t)parts.most;
  a.token_stride = (uint32_t)c.token_stride;
  a.page_size = (uint32_t)c.page_size;
  a.scale = in.scale * kLog2e;
  a.scale_tokens = (uint32_t)c.scale_tokens;
  return a;
}

template <int D, typename X, bool RUN>
hipError_t launch(const Args& a, int kind, bool split, hipStream_t st) {
  return kind == kBf16   ? launch<D, X, kBf16, RUN>(a, split, st)
         : kind == kInt8 ? launch<D, X, kInt8, RUN>(a, split, st)
                         : launch<D, X, kFp8, RUN>(a, split, st);
}

template <bool RUN>
hipError_t launch(const Args& a, int64_t head_dim, bool bf16, int kind, bool split, hipStream_t st) {
  if (head_dim == 64)
    return bf16 ? launch<64, __hip_bfloat16, RUN>(a, kind, split, st) : launch<64, float, RUN>(a, kind, split, st);
  return bf16 ? launch<128, __hip_bfloat16, RUN>(a, kind, split, st) : launch<128, float, RUN>(a, kind, split, st);
}

}  // namespace

}  // namespace qv
