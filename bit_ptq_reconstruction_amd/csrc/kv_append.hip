// kv_append.hip -- keys and values of new tokens into a paged cache, keys and queries rotated by
// position on the way.
//
//   a' = a cos - b sin,  b' = b cos + a sin   on the pairs (x[j], x[j + w/2]) of each axis' block of w channels
//   int8: scale = max |x'| / 127 over the head's channels, code = clamp(rne(x' / scale))
//
// Each value is read once and written once with a few operations between, so the kernel is bound by
// memory.  A thread holds 8 low and 8 high channels of one head of one token: both sides of its 8
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
  uint32_t threads;      // of this launch: tokens * (q_heads + 2 heads) * D / 16
  int64_t first;         // its first token
};

__device__ __forceinline__ float bits_float(unsigned u) { return __builtin_bit_cast(float, u); }

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
__device__ __forceinline__ void store8(int8_t* p, const float (&v)[8], float scale) {
  unsigned w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = scale > 0.0f ? fminf(fmaxf(rintf(v[i] / scale), -128.0f), 127.0f) : 0.0f;
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

template <int D, typename X, bool INT8>
__global__ __launch_bounds__(kThreads) void append_kernel(Args a) {
  constexpr int kParts = D / 16;
  const uint32_t at = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t per_token = (a.q_heads + 2 * a.heads) * kParts;
  const bool live = at < a.threads;
  const uint32_t id = live ? at : a.threads - 1;  // a head's threads stay together for the scale
  const int64_t t = a.first + id / per_token;
  const uint32_t in_token = id % per_token;
  const int part = in_token % kParts;
  int h = in_token / kParts;
  // kind: 0 query, 1 key, 2 value
  const int kind = h < a.q_heads ? 0 : (h < a.q_heads + a.heads ? 1 : 2);
  h -= kind == 0 ? 0 : (kind == 1 ? a.q_heads : a.q_heads + a.heads);
  const Rows src = kind == 0 ? a.q : (kind == 1 ? a.k : a.v);

  // The part's low and high channels: 8 of the first and 8 of the second half of an axis' block.
  const int half = D / 2 / a.axes, per_axis = half / 8;
  const int axis = part / per_axis, j = 8 * (part % per_axis);
  const int lo_c = axis * 2 * half + j, hi_c = lo_c + half;
  const X* x = static_cast<const X*>(src.data) + t * src.ts + h * src.hs;
  float lo[8], hi[8];
  load8(x + lo_c, lo);
  load8(x + hi_c, hi);

  const int place = a.index[t];
  bool known = true;  // the position lies in the tables
  if (a.cos) {
    const int p = a.position ? a.position[t * a.axes + axis] : place;
    if (a.position) {
      for (int i = 0; i < a.axes; ++i) {
        const int q = a.position[t * a.axes + i];
        known = known && q >= 0 && q < a.places;
      }
    } else {
      known = p >= 0 && p < a.places;
    }
    if (kind != 2 && known) {
      float c[8], s[8];
      load8(a.cos + (int64_t)p * half + j, c);
      load8(a.sin + (int64_t)p * half + j, s);
      turn(lo, hi, c, s);
    }
  }
  if (kind == 0) {
    if (!live) return;
    if (!known) {
#pragma unroll
      for (int i = 0; i < 8; ++i) lo[i] = hi[i] = __builtin_nanf("");
    }
    X* o = static_cast<X*>(const_cast<void*>(a.qo.data)) + t * a.qo.ts + h * a.qo.hs;
    store8(o + lo_c, lo);
    store8(o + hi_c, hi);
    return;
  }

  const int64_t seq = a.seq ? a.seq[t] : t;
  bool stored = live && known && seq >= 0 && seq < a.num_seqs && place >= 0;
  const int entry = place / a.page_size, slot = place % a.page_size;
  stored = stored && entry < a.max_pages;
  const int64_t page = stored ? a.table[seq * a.ld_table + entry] : -1;
  stored = stored && page >= 0 && page < a.num_pages;

  const int64_t to = page * a.page_stride + h * a.head_stride + slot * a.token_stride;
  char* base = kind == 1 ? a.kp : a.vp;
  if constexpr (!INT8) {
    if (!stored) return;
    __hip_bfloat16* o = reinterpret_cast<__hip_bfloat16*>(base) + to;
    store8(o + lo_c, lo);
    store8(o + hi_c, hi);
  } else {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
#pragma unroll
    for (int d = 1; d < kParts; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (!stored) return;
    float scale = top / 127.0f;
    if (!(scale >= 1.17549435e-38f)) scale = 0.0f;  // zero and subnormal scales
    int8_t* o = reinterpret_cast<int8_t*>(base) + to;
    store8(o + lo_c, lo, scale);
    store8(o + hi_c, hi, scale);
    if (part == 0) (kind == 1 ? a.ks : a.vs)[(page * a.heads + h) * a.page_size + slot] = scale;
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
  const int64_t per_token = (in.q_heads + 2 * c.heads) * (c.head_dim / 16);
  // A launch counts its threads in 32 bits; longer runs of tokens go in several.
  const int64_t most = ((int64_t{1} << 30) / per_token) > 0 ? (int64_t{1} << 30) / per_token : 1;
  for (int64_t t = 0; t < in.T; t += most) {
    const int64_t n = in.T - t < most ? in.T - t : most;
    a.first = t;
    a.threads = (uint32_t)(n * per_token);
    const unsigned blocks = (a.threads + kThreads - 1) / kThreads;
    const bool q8 = c.dtype == QV_KV_INT8;
#define QV_APPEND(D)                                                                             \
  if (in.bf16)                                                                                   \
    q8 ? append_kernel<D, __hip_bfloat16, true><<<blocks, kThreads, 0, st>>>(a)                  \
       : append_kernel<D, __hip_bfloat16, false><<<blocks, kThreads, 0, st>>>(a);                \
  else                                                                                           \
    q8 ? append_kernel<D, float, true><<<blocks, kThreads, 0, st>>>(a)                           \
       : append_kernel<D, float, false><<<blocks, kThreads, 0, st>>>(a)
    if (c.head_dim == 64) {
      QV_APPEND(64);
    } else {
      QV_APPEND(128);
    }
#undef QV_APPEND
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qv
