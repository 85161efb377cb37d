// append_rows.h -- rows of heads as the append's kernels read, turn and write them.
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qv_decode_internal.h"

namespace qv {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct Rows {
  const void* data;
  int64_t ts, hs;
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

inline Rows rows_of(const qv_heads& h) { return {h.data, h.token_stride, h.head_stride}; }

}  // namespace

hipError_t launch_kv_append_fp8(const AppendArgs& in, hipStream_t st);  // kv_append_fp8.hip

}  // namespace qv
