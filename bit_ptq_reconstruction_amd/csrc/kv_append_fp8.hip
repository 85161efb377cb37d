// kv_append_fp8.hip -- keys and values of new tokens into a paged cache of 8-bit floating-point codes with one scale for
// each block of tokens and head; keys and queries are rotated by position on the way.
//
//   s = 2^e, e the least (-126 at least) with max |x'| <= 448 * 2^e over the block's new values,   code = rne(x' / s)
//   an open block: s = max(s_before, s), and where it grows   code = rne(code * s_before / s)   for the places before
//
// 448 is the format's largest value.  With powers of two, quotients and products are exact, so a code is rounded once when it is
// made and again only where its block's scale grows and it becomes subnormal; the relative precision of a floating-point
// code does not depend on where in its binade the scale puts it.
//
// A wave owns a block of one head: it finds the run of the call's tokens that lie in the block, their maximum, the scale, and
// writes.  So no two waves touch a block and nothing is atomic.  The wave of a block's first token in the call (its leader)
// does this; waves look through a window of tokens for leaders.  A lane holds 8 low and 8 high channels of one token, both
// sides of its pairs.  The first tokens of a block (32 of 64 channels or 16 of 128) stay in registers between maximum and codes;
// their loads go out before the block's page is known.
//
// Bound by memory for prompts: 10992 tokens of 48 heads of 64 in blocks of 32 (116 MB) take 31 us, 3.7 TB/s (read twice and a
// token at a time it took 41).  One token of each of 24 sequences takes 6.0 us: a launch and the chain place -> page -> scale -> code.
#include "append_rows.h"

namespace qv {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInfinity = 0x7F800000u;

struct Args {
  Rows q, k, v, qo;
  char *kp, *vp;
  float *ks, *vs;
  const int32_t *table, *seq, *index, *position;
  const float *cos, *sin;
  int64_t num_pages, page_stride, head_stride, token_stride, ld_table;
  int64_t T, first;  // tokens of the call; the first one of this launch
  int32_t num_seqs, max_pages, page_size, heads, q_heads, places, axes, block;
  uint32_t count;              // tokens of this launch
  uint32_t window;             // tokens that a wave looks through
  uint32_t kv_waves, q_waves;  // of this launch
  uint32_t q_groups;           // waves of a token's queries
};

// A lane's channels of a token: 8 of the first and 8 of the second half of an axis' block.
template <int D>
struct Part {
  int axis, j, half, low, high;
  __device__ __forceinline__ Part(const Args& a, int part) {
    half = D / 2 >> (a.axes - 1);
    axis = part >= half / 8 ? 1 : 0;
    j = 8 * part - axis * half;
    low = axis * 2 * half + j;
    high = low + half;
  }
};

// Whether token t's position lies in the tables, and its place on the lane's axis.
template <int D>
__device__ __forceinline__ bool known_place(const Args& a, const Part<D>& part, int64_t t, int* p) {
  *p = 0;
  if (!a.cos) return true;
  if (a.position) {
    const int p0 = a.position[t * a.axes], p1 = a.position[t * a.axes + a.axes - 1];
    *p = part.axis ? p1 : p0;
    return p0 >= 0 && p0 < a.places && p1 >= 0 && p1 < a.places;
  }
  *p = a.index[t];
  return *p >= 0 && *p < a.places;
}

// The lane's channels of a row as they lie in memory.
template <typename X>
struct Raw {
  u32x4 d[sizeof(X)];  // low channels, then high ones
  __device__ __forceinline__ void load(const X* row, int low, int high) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(X) / 2; ++i) {
      d[i] = reinterpret_cast<const u32x4*>(row + low)[i];
      d[sizeof(X) / 2 + i] = reinterpret_cast<const u32x4*>(row + high)[i];
    }
  }
  __device__ __forceinline__ void get(int first, float (&v)[8]) const {
    if constexpr (sizeof(X) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bits_float(d[first][i] << 16);
        v[2 * i + 1] = bits_float(d[first][i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = bits_float(d[2 * first + (i >> 2)][i & 3]);
    }
  }
};

// The scale by which a largest magnitude (its bits, finite) is at most 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_of(uint32_t top) {
  const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u);
  return bits_float((uint32_t)((e < -126 ? -126 : e) + 127) << 23);
}

__device__ __forceinline__ bool power_of_two(float s) { return (float_bits(s) & 0x7FFFFFu) == 0; }

__device__ __forceinline__ unsigned code4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Codes of x / s.  What is not finite becomes NaN (the conversion would take an infinity as the largest value).
__device__ __forceinline__ void store8(char* p, const float (&x)[8], float s, float inverse, bool exact) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = exact ? x[i] * inverse : x[i] / s;
    if ((float_bits(x[i]) & kInfinity) == kInfinity) y[i] = __builtin_nanf("");
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(code4(y[0], y[1], y[2], y[3]), code4(y[4], y[5], y[6], y[7]));
}

// The codes of 16 channels times a ratio, rounded again.
__device__ __forceinline__ void rescale16(char* p, float ratio) {
  u32x4 w = *reinterpret_cast<u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned c = w[i];
    w[i] = code4(__builtin_amdgcn_cvt_f32_fp8(c, 0) * ratio, __builtin_amdgcn_cvt_f32_fp8(c, 1) * ratio,
                 __builtin_amdgcn_cvt_f32_fp8(c, 2) * ratio, __builtin_amdgcn_cvt_f32_fp8(c, 3) * ratio);
  }
  *reinterpret_cast<u32x4*>(p) = w;
}

template <int D, typename X>
struct Append {
  static constexpr int kParts = D / 16;        // lanes of a token
  static constexpr int kStep = 64 / kParts;    // tokens at a time
  static constexpr int kKept = 2;              // steps that stay in registers
  const Args& a;
  const int lane;
  const Part<D> part;

  __device__ __forceinline__ explicit Append(const Args& args)
      : a(args), lane(threadIdx.x & 63), part(args, (threadIdx.x & 63) % kParts) {}

  __device__ __forceinline__ int64_t sequence(int64_t t) const { return a.seq ? (int64_t)a.seq[t] : t; }

  // Whether token t is the first of the call in its block.
  __device__ __forceinline__ bool leads(int64_t t) const {
    if (!a.seq) return true;  // one token to a sequence
    const uint32_t place = (uint32_t)a.index[t];
    return t == 0 || place % (uint32_t)a.block == 0 || sequence(t - 1) != sequence(t) || (uint32_t)a.index[t - 1] + 1 != place;
  }

  __device__ __forceinline__ const X* row(const Rows& src, int head, int64_t t) const {
    return static_cast<const X*>(src.data) + t * src.ts + head * src.hs;
  }
  // Token t's channels, turned if they are a key's or query's; false: its position is unknown.
  __device__ __forceinline__ bool values(const Raw<X>& raw, bool turned, int64_t t, float (&lo)[8], float (&hi)[8]) const {
    raw.get(0, lo);
    raw.get(1, hi);
    int p;
    const bool known = known_place(a, part, t, &p);
    if (a.cos && known && turned) {
      float c[8], s[8];
      load8(a.cos + (int64_t)p * part.half + part.j, c);
      load8(a.sin + (int64_t)p * part.half + part.j, s);
      turn(lo, hi, c, s);
    }
    return known;
  }

  // The block that token t leads (if it does), for one head of the keys or values.
  __device__ __forceinline__ void block(int64_t t, bool key, int head) const {
    const Rows& src = key ? a.k : a.v;
    const uint32_t mine = lane / kParts;
    Raw<X> raw[kKept];  // on their way while the place is found
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int64_t s = t + mine + i * kStep;
      if (s < a.T) raw[i].load(row(src, head, s), part.low, part.high);
    }
    // Places and sequences of this token and those behind it, a lane each.
    const int64_t mine_t = t + lane < a.T ? t + lane : a.T - 1;
    const int32_t my_place = a.index[mine_t], my_seq = a.seq ? a.seq[mine_t] : 0;
    if (!leads(t)) return;
    const uint32_t size = (uint32_t)a.block;
    const int place = __builtin_amdgcn_readfirstlane(my_place);
    const int64_t seq = a.seq ? (int64_t)__builtin_amdgcn_readfirstlane(my_seq) : t;
    if (place < 0 || seq < 0 || seq >= a.num_seqs) return;
    const uint32_t entry = (uint32_t)place / (uint32_t)a.page_size, slot = (uint32_t)place % (uint32_t)a.page_size;
    if (entry >= (uint32_t)a.max_pages) return;
    const int64_t page = a.table[seq * a.ld_table + entry];
    const uint32_t at = slot % size, most = size - at;

    uint32_t n = 1;  // tokens of the call that lie in the block
    if (a.seq) {
      const uint32_t ahead = lane;
      uint64_t missing = ~__ballot(ahead < most && t + lane < a.T && my_seq == seq && (uint32_t)my_place == (uint32_t)place + ahead);
      n = missing ? __builtin_ctzll(missing) : 64;
      while (!missing) {
        const uint32_t j = n + lane;
        const bool ok = j < most && t + j < a.T && a.seq[t + j] == seq && (uint32_t)a.index[t + j] == (uint32_t)place + j;
        missing = ~__ballot(ok);
        n += missing ? __builtin_ctzll(missing) : 64;
      }
    }
    if (page < 0 || page >= a.num_pages) return;
    float* const held = (key ? a.ks : a.vs) + (page * a.heads + head) * (a.page_size / size) + slot / size;
    const float before = at ? *held : 0.0f;

    uint32_t top = 0;
    auto largest = [&](const float (&x)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = float_bits(x[i]) & 0x7FFFFFFFu;
        if (b < kInfinity && b > top) top = b;
      }
    };
    float lo[kKept][8], hi[kKept][8];
    bool stored[kKept];
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const uint32_t j = mine + i * kStep;
      stored[i] = j < n && values(raw[i], key, t + j, lo[i], hi[i]);
      if (stored[i]) largest(lo[i]), largest(hi[i]);
    }
    for (uint32_t j = kKept * kStep + mine; j < n; j += kStep) {  // these are read again below
      Raw<X> x;
      float l[8], h[8];
      x.load(row(src, head, t + j), part.low, part.high);
      if (values(x, key, t + j, l, h)) largest(l), largest(h);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const float s = at ? fmaxf(before, scale_of(top)) : scale_of(top);
    const bool exact = power_of_two(s);
    const float inverse = 1.0f / s;

    char* const start = (key ? a.kp : a.vp) + page * a.page_stride + head * a.head_stride + (int64_t)(slot - at) * a.token_stride;
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      if (!stored[i]) continue;
      char* const to = start + (int64_t)(at + mine + i * kStep) * a.token_stride;
      store8(to + part.low, lo[i], s, inverse, exact);
      store8(to + part.high, hi[i], s, inverse, exact);
    }
    for (uint32_t j = kKept * kStep + mine; j < n; j += kStep) {
      Raw<X> x;
      float l[8], h[8];
      x.load(row(src, head, t + j), part.low, part.high);
      if (!values(x, key, t + j, l, h)) continue;
      char* const to = start + (int64_t)(at + j) * a.token_stride;
      store8(to + part.low, l, s, inverse, exact);
      store8(to + part.high, h, s, inverse, exact);
    }
    if (at && before != s) {
      const float ratio = before / s;
      for (uint32_t j = mine; j < at; j += kStep) rescale16(start + (int64_t)j * a.token_stride + 16 * (lane % kParts), ratio);
    }
    if (lane == 0) *held = s;
  }

  __device__ __forceinline__ void query(int64_t t, int head) const {
    if (head >= a.q_heads) return;
    float lo[8], hi[8];
    Raw<X> x;
    x.load(row(a.q, head, t), part.low, part.high);
    if (!values(x, true, t, lo, hi)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) lo[i] = hi[i] = __builtin_nanf("");
    }
    X* const o = static_cast<X*>(const_cast<void*>(a.qo.data)) + t * a.qo.ts + head * a.qo.hs;
    qv::store8(o + part.low, lo);
    qv::store8(o + part.high, hi);
  }
};

template <int D, typename X>
__global__ __launch_bounds__(kThreads) void append_fp8_kernel(Args a) {
  const Append<D, X> append(a);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + threadIdx.x / 64);
  if (wave < a.kv_waves) {
    const uint32_t heads = 2 * a.heads, first = wave / heads * a.window, which = wave % heads;
    const uint32_t end = first + a.window < a.count ? first + a.window : a.count;
    const bool key = which < (uint32_t)a.heads;
    const int head = key ? which : which - a.heads;
    if (a.window == 1) {
      append.block(a.first + first, key, head);
    } else {
      const bool leads = first + append.lane < end && append.leads(a.first + first + append.lane);
      for (uint64_t left = __ballot(leads); left; left &= left - 1) append.block(a.first + first + __builtin_ctzll(left), key, head);
    }
  } else if (wave - a.kv_waves < a.q_waves) {
    const uint32_t id = wave - a.kv_waves;
    append.query(a.first + id / a.q_groups, id % a.q_groups * Append<D, X>::kStep + append.lane / Append<D, X>::kParts);
  }
}

}  // namespace

hipError_t launch_kv_append_fp8(const AppendArgs& in, hipStream_t st) {
  const qv_kv_cache& c = in.cache;
  Args a = {};
  a.q = rows_of(in.Q);
  a.k = rows_of(in.K);
  a.v = rows_of(in.V);
  a.qo = rows_of(in.Q_out);
  a.kp = static_cast<char*>(c.k_pages);
  a.vp = static_cast<char*>(c.v_pages);
  a.ks = c.k_scale;
  a.vs = c.v_scale;
  a.table = in.page_table;
  a.seq = in.token_seq;
  a.index = in.token_index;
  a.position = in.position;
  a.cos = in.cos;
  a.sin = in.sin;
  a.num_pages = c.num_pages;
  a.page_stride = c.page_stride;
  a.head_stride = c.head_stride;
  a.token_stride = c.token_stride;
  a.ld_table = in.ld_table;
  a.T = in.T;
  a.num_seqs = (int32_t)in.num_seqs;
  a.max_pages = (int32_t)in.max_pages;
  a.page_size = (int32_t)c.page_size;
  a.heads = (int32_t)c.heads;
  a.q_heads = (int32_t)in.q_heads;
  a.places = (int32_t)in.places;
  a.axes = (int32_t)in.axes;
  a.block = c.scale_tokens;
  const int64_t step = 64 / (c.head_dim / 16);
  a.q_groups = (uint32_t)((in.q_heads + step - 1) / step);
  // A wave for each token while that does not fill the chip, so that single tokens of many sequences go side by side; then
  // windows of up to a block (and 64), since only one wave in a block's tokens finds a leader.
  a.window = 1;
  while (a.window < 64 && 2 * a.window <= (uint32_t)a.block && in.T * 2 * c.heads / a.window > 8192) a.window *= 2;
  // A launch counts its waves in 32 bits; longer runs of tokens go in several.
  const int64_t per_token = 2 * c.heads + a.q_groups;
  const int64_t most = (int64_t{1} << 25) / per_token / 64 * 64 > 0 ? (int64_t{1} << 25) / per_token / 64 * 64 : 64;
  for (int64_t t = 0; t < in.T; t += most) {
    a.first = t;
    a.count = (uint32_t)(in.T - t < most ? in.T - t : most);
    a.kv_waves = (uint32_t)((a.count + a.window - 1) / a.window * 2 * c.heads);
    a.q_waves = a.count * a.q_groups;
    const unsigned blocks = (unsigned)(((int64_t)a.kv_waves + a.q_waves + kThreads / 64 - 1) / (kThreads / 64));
    if (c.head_dim == 64)
      in.bf16 ? append_fp8_kernel<64, __hip_bfloat16><<<blocks, kThreads, 0, st>>>(a)
              : append_fp8_kernel<64, float><<<blocks, kThreads, 0, st>>>(a);
    else
      in.bf16 ? append_fp8_kernel<128, __hip_bfloat16><<<blocks, kThreads, 0, st>>>(a)
              : append_fp8_kernel<128, float><<<blocks, kThreads, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qv
