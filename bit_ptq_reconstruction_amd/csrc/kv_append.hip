// kv_append.hip -- keys and values of new tokens into a paged cache, keys and queries rotated by
// position on the way.
//
//   a' = a cos - b sin,  b' = b cos + a sin   on the pairs (x[j], x[j + w/2]) of each axis' block of w channels
//   int8: scale = max |x'| / 127 over the head's channels, code = clamp(rne(x' / scale))
//
// Each value is read once and written once with a few operations between, so the kernel is bound by
// memory: 10992 tokens of 48 heads of 64 (138 MB with the tables) take 32 us, 4.3 TB/s against a copy's 5.0; one token of each of 24
// sequences takes 3.2 us, a launch; 1833 fp32 tokens into int8 (40 MB) 12 us, 3.4 TB/s, launch included.
// A thread holds 8 low and 8 high channels of one head of one token: both sides of its 8
// pairs, in 16-byte loads and stores.  The D / 16 threads of a head are neighbours in a wave, so the int8
// scale is a maximum over 4 or 8 lanes.
//
// Every product and sum is rounded by itself (no fused multiply-add) and quotients are correctly rounded,
// so codes and bf16 values are those of the formula evaluated step by step in fp32.
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qv_decode_internal.h"

namespace qv {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

struct Rows {
  const void* data;
  int64_t ts, hs;
};

struct Args {
  Rows q, k, v, qo;
  char *kp, *vp;
  float *ks, *vs;
  const int32_t *table, *seq, *index, *position;
  const float *cos, *sin;
  int64_t num_pages, page_stride, head_stride, token_stride, ld_table;
  int32_t num_seqs, max_pages, page_size, heads, q_heads, places, axes;
  uint32_t groups;       // threads of a token and part
  uint32_t threads;      // of this launch: tokens * groups * D / 16
  int64_t first;         // its first token
};

__device__ __forceinline__ float bits_float(unsigned u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ unsigned float_bits(float f) { return __builtin_bit_cast(unsigned, f); }

__device__ __forceinline__ void load8(const __hip_bfloat16* p, float (&v)[8]) {
  const u32x4 d = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned w = d[i];
    v[2 * i] = bits_float(w << 16);
    v[2 * i + 1] = bits_float(w & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}

__device__ __forceinline__ unsigned bf16_bits(float f) {
  return __builtin_bit_cast(unsigned short, __float2bfloat16(f));
}
__device__ __forceinline__ void store8(__hip_bfloat16* p, const float (&v)[8]) {
  u32x4 d;
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
  *reinterpret_cast<u32x4*>(p) = d;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}
// Codes of the correctly rounded quotients v / scale (scale 0 or NaN: zeros).  The product with the reciprocal is off by at most
// 127 * 2^-23 and the quotient by 127 * 2^-24, 2.3e-5 together: only values nearer than 3e-5 to a half need the
// division itself (0.4 % of the waves' elements).
__device__ __forceinline__ void store8(int8_t* p, const float (&v)[8], float scale, float inverse) {
  unsigned w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = v[i] * inverse;
    float q = rintf(t);
    if (fabsf(t - q) > 0.49997f) q = rintf(v[i] / scale);
    q = inverse > 0.0f ? fminf(fmaxf(q, -128.0f), 127.0f) : 0.0f;
    w[i >> 2] |= ((unsigned)(int)q & 255u) << (8 * (i & 3));
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// The pairs (a, b) turned by their angles; __fmul_rn and its like do not keep the compiler from fusing.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = a[i], w = b[i];
    a[i] = u * c[i] - w * s[i];
    b[i] = w * c[i] + u * s[i];
  }
}

// R: heads of a thread, all of one token and `groups` apart, so that neighbouring threads have neighbouring heads; they
// share the token's place and its cosines and sines.
template <int D, typename X, bool INT8, int R>
__global__ __launch_bounds__(kThreads) void append_kernel(Args a) {
  constexpr int kParts = D / 16;
  const uint32_t at = blockIdx.x * kThreads + threadIdx.x;
  const bool live = at < a.threads;
  const uint32_t id = live ? at : a.threads - 1;  // a head's threads stay together for the scale
  const int part = id % kParts;
  const uint32_t in_run = id / kParts / a.groups;  // token of this launch
  const int64_t t = a.first + in_run;
  const int group = (int)(id / kParts - in_run * a.groups), slots = a.q_heads + 2 * a.heads;

  // The part's low and high channels: 8 of the first and 8 of the second half of an axis' block.
  const int half = D / 2 >> (a.axes - 1), per_axis = half / 8;
  const int axis = part >= per_axis ? 1 : 0, j = 8 * (part - axis * per_axis);
  const int lo_c = axis * 2 * half + j, hi_c = lo_c + half;

  float lo[R][8], hi[R][8];
  int kind[R], head[R];  // 0 query, 1 key, 2 value, 3 nothing
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int h = group + i * a.groups;
    kind[i] = !live || h >= slots ? 3 : (h < a.q_heads ? 0 : (h < a.q_heads + a.heads ? 1 : 2));
    head[i] = h - (kind[i] == 0 ? 0 : (kind[i] == 1 ? a.q_heads : a.q_heads + a.heads));
    if (kind[i] == 3) head[i] = 0;  // reads the first value: a scale's lanes stay together
    const Rows src = kind[i] == 0 ? a.q : (kind[i] == 1 ? a.k : a.v);
    const X* x = static_cast<const X*>(src.data) + t * src.ts + head[i] * src.hs;
    load8(x + lo_c, lo[i]);
    load8(x + hi_c, hi[i]);
  }

  const int place = a.index[t];
  const int64_t seq = a.seq ? a.seq[t] : t;
  bool known = true;  // the position lies in the tables
  float c[8], s[8];
  if (a.cos) {
    int p = place;
    if (a.position) {
      const int p0 = a.position[t * a.axes], p1 = a.position[t * a.axes + a.axes - 1];
      known = p0 >= 0 && p0 < a.places && p1 >= 0 && p1 < a.places;
      p = axis ? p1 : p0;
    } else {
      known = p >= 0 && p < a.places;
    }
    const int64_t from = known ? (int64_t)p * half + j : 0;
    if (a.places > 0) {
      load8(a.cos + from, c);
      load8(a.sin + from, s);
    }
  }
  bool stored = known && seq >= 0 && seq < a.num_seqs && place >= 0;
  const int entry = (int)((uint32_t)place / (uint32_t)a.page_size), slot = place - entry * a.page_size;
  stored = stored && entry < a.max_pages;
  const int64_t page = stored ? a.table[seq * a.ld_table + entry] : -1;
  stored = stored && page >= 0 && page < a.num_pages;

#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (a.cos && known && kind[i] <= 1) turn(lo[i], hi[i], c, s);
    if (kind[i] == 0) {
      if (!known) {
#pragma unroll
        for (int n = 0; n < 8; ++n) lo[i][n] = hi[i][n] = __builtin_nanf("");
      }
      X* o = static_cast<X*>(const_cast<void*>(a.qo.data)) + t * a.qo.ts + head[i] * a.qo.hs;
      store8(o + lo_c, lo[i]);
      store8(o + hi_c, hi[i]);
    }
    float scale = 0.0f;
    if constexpr (INT8) {
      // The maximum as bits, which for magnitudes have the order of the values, infinities and then NaN above all.
      unsigned bits = 0;
#pragma unroll
      for (int n = 0; n < 8; ++n) bits = max(bits, max(float_bits(lo[i][n]) & 0x7FFFFFFFu, float_bits(hi[i][n]) & 0x7FFFFFFFu));
#pragma unroll
      for (int d = 1; d < kParts; d <<= 1) bits = max(bits, (unsigned)__shfl_xor((int)bits, d));
      scale = bits_float(bits) / 127.0f;
      if (scale < 1.17549435e-38f) scale = 0.0f;  // zero and subnormal scales
      if (bits >= 0x7F800000u) scale = __builtin_nanf("");
    }
    if (!stored || kind[i] == 0 || kind[i] == 3) continue;
    const int64_t to = page * a.page_stride + head[i] * a.head_stride + slot * a.token_stride;
    char* base = kind[i] == 1 ? a.kp : a.vp;
    if constexpr (!INT8) {
      __hip_bfloat16* o = reinterpret_cast<__hip_bfloat16*>(base) + to;
      store8(o + lo_c, lo[i]);
      store8(o + hi_c, hi[i]);
    } else {
      int8_t* o = reinterpret_cast<int8_t*>(base) + to;
      const float inverse = scale > 0.0f ? 1.0f / scale : 0.0f;  // 0: every code is 0, of NaN and infinities too
      store8(o + lo_c, lo[i], scale, inverse);
      store8(o + hi_c, hi[i], scale, inverse);
      if (part == 0) (kind[i] == 1 ? a.ks : a.vs)[(page * a.heads + head[i]) * a.page_size + slot] = scale;
    }
  }
}

Rows rows_of(const qv_heads& h) { return {h.data, h.token_stride, h.head_stride}; }

}  // namespace

hipError_t launch_kv_append(const AppendArgs& in, hipStream_t st) {
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
  a.num_seqs = (int32_t)in.num_seqs;
  a.max_pages = (int32_t)in.max_pages;
  a.page_size = (int32_t)c.page_size;
  a.heads = (int32_t)c.heads;
  a.q_heads = (int32_t)in.q_heads;
  a.places = (int32_t)in.places;
  a.axes = (int32_t)in.axes;
  const int64_t slots = in.q_heads + 2 * c.heads;
  // One head a thread until the chip is full twice over, then two (24 tokens of 48 heads: 3.2 against 3.6 us; 16000 of 48
  // heads of 128: 80.6 against 76.2 us).
  const int r = in.T * slots * (c.head_dim / 16) >= (int64_t{1} << 20) ? 2 : 1;
  a.groups = (uint32_t)((slots + r - 1) / r);
  const int64_t per_token = a.groups * (c.head_dim / 16);
  // A launch counts its threads in 32 bits; longer runs of tokens go in several.
  const int64_t most = ((int64_t{1} << 30) / per_token) > 0 ? (int64_t{1} << 30) / per_token : 1;
  for (int64_t t = 0; t < in.T; t += most) {
    const int64_t n = in.T - t < most ? in.T - t : most;
    a.first = t;
    a.threads = (uint32_t)(n * per_token);
    const unsigned blocks = (a.threads + kThreads - 1) / kThreads;
    const bool q8 = c.dtype == QV_KV_INT8;
#define QV_APPEND(D, R)                                                                          \
  if (in.bf16)                                                                                   \
    q8 ? append_kernel<D, __hip_bfloat16, true, R><<<blocks, kThreads, 0, st>>>(a)               \
       : append_kernel<D, __hip_bfloat16, false, R><<<blocks, kThreads, 0, st>>>(a);             \
  else                                                                                           \
    q8 ? append_kernel<D, float, true, R><<<blocks, kThreads, 0, st>>>(a)                        \
       : append_kernel<D, float, false, R><<<blocks, kThreads, 0, st>>>(a)
    if (c.head_dim == 64 && r == 1) {
      QV_APPEND(64, 1);
    } else if (c.head_dim == 64) {
      QV_APPEND(64, 2);
    } else if (r == 1) {
      QV_APPEND(128, 1);
    } else {
      QV_APPEND(128, 2);
    }
#undef QV_APPEND
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qv
