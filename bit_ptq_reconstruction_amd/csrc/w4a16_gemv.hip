// w4a16_gemv.hip -- few rows of unquantized activations times int4 weights with group scales, with the
// Hadamard rotation and smoothing of the activations on the way.
//
//   Y[m][n] = sum_g s[n][g] * (sum_{k in g} x[m][k] q[n][k]) (+ bias) (+ GELU),  q in [-8, 7]
//
// With a few rows the weights' N K / 2 bytes are all there is to move, so the kernel is bound by memory
// (by latency for the smallest layers); the arithmetic only has to keep up with it.
//
// Products run on the matrix cores, 16 rows x 16 channels x 32 codes at a time, whatever M is: one
// v_mfma_f32_16x16x32_bf16 replaces 512 multiply-adds for 16 cycles, and the vector ALU is left with
// the unpacking.  Both operands are exact in bf16:
//   - with fp32 results a code is converted by itself (v_cvt_off_f32_i4 gives q / 16, and the upper halves
//     of two are packed: 19 instructions for 8 codes).
//   - with bf16 results a code q becomes 24 + q in [16, 31], i.e. the bits 0x4180 | (q + 8) << 3: one shift
//     and one and-or for two codes, 9 instructions for 8.  The surplus 24 * sum_k x[m][k] is formed by one more
//     MFMA against ones and taken off each group's sum.  The larger partial sums triple the fp32
//     rounding error, from 3e-7 of the result to 1e-6, which a bf16 result does not show and an fp32 one does.
//   - an activation is a sum of NP bf16 pieces (the top 16 bits, then the top 16 bits of the rest, ...):
//     one piece is exact for bf16 rows, two keep 16 bits for rotated or fp32 rows with a bf16 result
//     (2^-16 against the result's own 2^-9), three keep all 24 bits for fp32 results.
// A lane's 16-byte load holds 32 codes of one channel, and code i of dword j is contracted in MFMA j;
// the order of k inside the sum is free, so activations are read to match: lane (row r, quarter c)
// takes k = 32 c + 8 j + i of the 128-code window.
//
// A block takes 16 NT channels; its waves take the 128-code windows in turn and their sums are
// added over LDS.
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qv_decode_internal.h"

namespace qv {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 16;     // activation rows of a block (the MFMA's M)
constexpr int kWindow = 128;  // codes of a window: one 16-byte load by each quarter of a wave

// Rotated rows lie in LDS as floats with 8 floats of padding after every 64, so that the strided reads
// of the transform's passes and the fragment reads of the four quarters fall in different banks.
__host__ __device__ constexpr int padded(int k) { return k + 8 * (k >> 6); }

// Eight activations as loaded.
template <typename X>
struct Eight;
template <>
struct Eight<__hip_bfloat16> {
  u32x4 d;
};
template <>
struct Eight<float> {
  f32x4 d[2];
};

__device__ __forceinline__ void load_eight(const __hip_bfloat16* p, Eight<__hip_bfloat16>& v) {
  v.d = *reinterpret_cast<const u32x4*>(p);
}
__device__ __forceinline__ void load_eight(const float* p, Eight<float>& v) {
  v.d[0] = *reinterpret_cast<const f32x4*>(p);
  v.d[1] = *reinterpret_cast<const f32x4*>(p + 4);
}

__device__ __forceinline__ float bits_float(unsigned u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ unsigned float_bits(float f) { return __builtin_bit_cast(unsigned, f); }

// The NP pieces of eight activations in the codes' order: dword s holds elements s and s + 4.
template <int NP>
__device__ __forceinline__ void pieces(const Eight<__hip_bfloat16>& v, bf16x8 (&f)[NP]) {
  static_assert(NP == 1, "bf16 rows are one piece");
  u32x4 o;
  o[0] = __builtin_amdgcn_perm(v.d[2], v.d[0], 0x05040100u);
  o[1] = __builtin_amdgcn_perm(v.d[2], v.d[0], 0x07060302u);
  o[2] = __builtin_amdgcn_perm(v.d[3], v.d[1], 0x05040100u);
  o[3] = __builtin_amdgcn_perm(v.d[3], v.d[1], 0x07060302u);
  f[0] = __builtin_bit_cast(bf16x8, o);
}
template <int NP>
__device__ __forceinline__ void pieces(const Eight<float>& v, bf16x8 (&f)[NP]) {
  f32x4 lo = v.d[0], hi = v.d[1];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    u32x4 o;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float a = lo[s], b = hi[s];
      const unsigned ua = float_bits(a), ub = float_bits(b);
      o[s] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
      if (p + 1 < NP) {  // exact: the piece is the value's top bits
        lo[s] = a - bits_float(ua & 0xFFFF0000u);
        hi[s] = b - bits_float(ub & 0xFFFF0000u);
      }
    }
    f[p] = __builtin_bit_cast(bf16x8, o);
  }
}

// Eight codes -> q / 16 in bf16, exactly, dword s holding codes s and s + 4.
__device__ __forceinline__ bf16x8 widen_exact(unsigned w) {
  u32x4 o;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const float a = __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (4 * s)));
    const float b = __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (4 * s + 16)));
    o[s] = __builtin_amdgcn_perm(float_bits(b), float_bits(a), 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8, o);
}

// Eight codes -> 24 + q in bf16, dword s holding codes s and s + 4.
__device__ __forceinline__ bf16x8 widen(unsigned w) {
  const unsigned u = w ^ 0x88888888u;  // q + 8 in each nibble
  u32x4 o;
  o[0] = ((u << 3) & 0x00780078u) | 0x41804180u;
  o[1] = ((u >> 1) & 0x00780078u) | 0x41804180u;
  o[2] = ((u >> 5) & 0x00780078u) | 0x41804180u;
  o[3] = ((u >> 9) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8, o);
}

__device__ __forceinline__ float gelu(float y) { return 0.5f * y * erfcf(-y * 0.70710678118654752f); }

// Sylvester-order Hadamard transform of one row by K / 8 threads (t of them counted here), times mult / sqrt(K):
// log2(K) butterfly stages, three in registers per pass over LDS.  Called by every thread of a block.
template <int K, typename X>
__device__ __forceinline__ void rotate_row(const X* __restrict__ x, const float* __restrict__ mult, float* row, int t) {
  static_assert(K == 1024 || K == 4096, "Hadamard width");
  constexpr float kNorm = K == 1024 ? 0.03125f : 0.015625f;
  float v[8];
  auto butterflies = [&](int from) {  // index bits of the register number, from bit `from`
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
      if (h < from) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if ((j & h) == 0) {
          const float a = v[j], b = v[j + h];
          v[j] = a + b;
          v[j + h] = a - b;
        }
      }
    }
  };
  {  // bits 0-2
    Eight<X> e;
    load_eight(x + 8 * t, e);
    if constexpr (sizeof(X) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned w = e.d[i];
        v[2 * i] = bits_float(w << 16);
        v[2 * i + 1] = bits_float(w & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = e.d[i >> 2][i & 3];
    }
    butterflies(1);
    f32x4* p = reinterpret_cast<f32x4*>(row + padded(8 * t));
    p[0] = f32x4{v[0], v[1], v[2], v[3]};
    p[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
  __syncthreads();
#pragma unroll
  for (int bit = 3; bit <= 6; bit += 3) {  // bits 3-5, then 6-8
    const int low = t & ((1 << bit) - 1), high = t >> bit;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = row[padded(low + (j << bit) + (high << (bit + 3)))];
    butterflies(1);
#pragma unroll
    for (int j = 0; j < 8; ++j) row[padded(low + (j << bit) + (high << (bit + 3)))] = v[j];
    __syncthreads();
  }
  constexpr int kStep = K / 8;  // bits 9-11 at K = 4096; at K = 1024 only bit 9, the last of the three
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = row[padded(t + j * kStep)];
  butterflies(K == 1024 ? 4 : 1);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int k = t + j * kStep;
    row[padded(k)] = v[j] * (mult ? kNorm * mult[k] : kNorm);
  }
}

template <typename X>
struct Args {
  const X* x;
  const float* mult;
  const uint8_t* wq;
  const float* ws;
  const float* bias;
  void* y;
  int64_t M, ldx, ldy;
  int N, K, group;
  int gelu, y_bf16;
};

// EXACT: fp32 results, codes converted exactly.  KROT: 0: rows are read from memory as they are; else the Hadamard width K, and the block rotates
// its rows into LDS first.
template <typename X, int NP, bool EXACT, int NT, int KROT>
__global__ __launch_bounds__(kThreads) void w4a16_kernel(Args<X> a) {
  extern __shared__ f32x4 lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, c = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT);
  const int64_t m0 = (int64_t)blockIdx.y * kRows;
  const int rows = (int)(a.M - m0 < kRows ? a.M - m0 : kRows);
  const int windows = a.K / kWindow, groups = a.K / a.group;

  const uint8_t* wrow[NT];
  const float* srow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    int n = n0 + 16 * t + r;
    n = n < a.N ? n : a.N - 1;
    wrow[t] = a.wq + (int64_t)n * (a.K / 2) + 16 * c;
    srow[t] = a.ws + (int64_t)n * groups;
  }
  u32x4 w[NT];
  float s[NT];
  auto load_weights = [&](int win) {
    const int g = win * kWindow / a.group;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w[t] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow[t] + (int64_t)win * (kWindow / 2)));
      s[t] = srow[t][g];
    }
  };
  if (wave < windows) load_weights(wave);

  float* const rot = reinterpret_cast<float*>(lds);
  constexpr int kRowFloats = KROT ? padded(KROT) : 1;
  if constexpr (KROT != 0) {
    constexpr int kAtOnce = 8 * kThreads / KROT;  // rows in one go
    const int part = threadIdx.x / (KROT / 8), t = threadIdx.x % (KROT / 8);
    for (int m = 0; m < rows; m += kAtOnce) {
      const int mine = m + part < rows ? m + part : rows - 1;
      rotate_row<KROT, X>(a.x + (m0 + mine) * a.ldx, a.mult, rot + (m + part) * kRowFloats, t);
    }
    __syncthreads();
  }
  const int row = r < rows ? r : rows - 1;
  const X* const xrow = a.x + (m0 + row) * a.ldx + 32 * c;
  const float* const lrow = rot + row * kRowFloats;

  f32x4 y[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) y[t] = f32x4{0, 0, 0, 0};
  bf16x8 ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;

  for (int win = wave; win < windows; win += kWaves) {
    u32x4 wc[NT];
    float sc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) wc[t] = w[t], sc[t] = s[t];
    f32x4 acc[NT], sum = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    bf16x8 xf[4][NP];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (KROT != 0) {
        Eight<float> e;
        load_eight(lrow + padded(win * kWindow + 32 * c) + 8 * j, e);
        pieces<NP>(e, xf[j]);
      } else {
        Eight<X> e;
        load_eight(xrow + win * kWindow + 8 * j, e);
        pieces<NP>(e, xf[j]);
      }
    }
    if (win + kWaves < windows) load_weights(win + kWaves);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!EXACT) {
#pragma unroll
        for (int p = 0; p < NP; ++p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j][p], ones, sum, 0, 0, 0);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16x8 wf = EXACT ? widen_exact(wc[t][j]) : widen(wc[t][j]);
#pragma unroll
        for (int p = 0; p < NP; ++p) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j][p], wf, acc[t], 0, 0, 0);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[t][i] += EXACT ? 16.0f * sc[t] * acc[t][i] : sc[t] * (acc[t][i] - 24.0f * sum[i]);
  }

  // Element (m, n) of tile t at [wave][t][m][n].
  float* const red = rot + (KROT ? ((rows + 3) & ~3) * kRowFloats : 0);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(wave * NT + t) * 256 + (4 * c + i) * 16 + r] = y[t][i];
  __syncthreads();
  for (int idx = threadIdx.x; idx < 256 * NT; idx += kThreads) {
    const int t = idx >> 8, m = (idx >> 4) & 15, n = n0 + 16 * t + (idx & 15);
    if (m >= rows || n >= a.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += red[k * NT * 256 + idx];
    if (a.bias) v += a.bias[n];
    if (a.gelu) v = gelu(v);
    const int64_t at = (m0 + m) * a.ldy + n;
    if (a.y_bf16)
      reinterpret_cast<__hip_bfloat16*>(a.y)[at] = __float2bfloat16(v);
    else
      reinterpret_cast<float*>(a.y)[at] = v;
  }
}

// Rows rotated and smoothed into memory as fp32, one block of K / 8 threads to a row.
template <int K, typename X>
__global__ __launch_bounds__(K / 8) void rotate_rows_kernel(const X* __restrict__ x, int64_t ldx,
                                                            const float* __restrict__ mult, float* __restrict__ out) {
  __shared__ f32x4 row4[padded(K) / 4];
  float* row = reinterpret_cast<float*>(row4);
  const int t = threadIdx.x;
  rotate_row<K, X>(x + (int64_t)blockIdx.x * ldx, mult, row, t);
  __syncthreads();
  f32x4* o = reinterpret_cast<f32x4*>(out + (int64_t)blockIdx.x * K + 8 * t);
  const f32x4* p = reinterpret_cast<const f32x4*>(row + padded(8 * t));
  o[0] = p[0];
  o[1] = p[1];
}

template <typename X, int NP, bool EXACT, int NT, int KROT>
hipError_t launch_kernel(const Args<X>& a, hipStream_t st) {
  const unsigned gx = (unsigned)((a.N + 16 * NT - 1) / (16 * NT));
  const int rows = (int)(a.M < kRows ? a.M : kRows);
  size_t bytes = (size_t)kWaves * NT * 256 * 4;
  if (KROT) bytes += (size_t)((rows + 3) & ~3) * padded(KROT ? KROT : 1) * 4;
  // grid.y holds 65535 blocks: longer runs go in several launches
  const int64_t step = (int64_t)65535 * kRows;
  for (int64_t m = 0; m < a.M; m += step) {
    Args<X> b = a;
    b.x += m * a.ldx;
    b.M = a.M - m < step ? a.M - m : step;
    b.y = static_cast<char*>(a.y) + m * a.ldy * (a.y_bf16 ? 2 : 4);
    w4a16_kernel<X, NP, EXACT, NT, KROT><<<dim3(gx, (unsigned)((b.M + kRows - 1) / kRows)), kThreads, bytes, st>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename X, int NP, bool EXACT, int KROT>
hipError_t by_tiles(const Args<X>& a, hipStream_t st) {
  return launch_kernel<X, NP, EXACT, 1, KROT>(a, st);
}

// Pieces by the types: rows that are bf16 are one piece; others two or, for fp32 results, three.
template <typename X, int KROT>
hipError_t by_types(const Args<X>& a, hipStream_t st) {
  if constexpr (sizeof(X) == 2 && KROT == 0)
    return a.y_bf16 ? by_tiles<X, 1, false, KROT>(a, st) : by_tiles<X, 1, true, KROT>(a, st);
  else
    return a.y_bf16 ? by_tiles<X, 2, false, KROT>(a, st) : by_tiles<X, 3, true, KROT>(a, st);
}

template <typename X>
hipError_t rotate_rows(const X* x, int64_t M, int64_t K, int64_t ldx, const float* mult, float* out, hipStream_t st) {
  if (K == 1024)
    rotate_rows_kernel<1024, X><<<(unsigned)M, 128, 0, st>>>(x, ldx, mult, out);
  else
    rotate_rows_kernel<4096, X><<<(unsigned)M, 512, 0, st>>>(x, ldx, mult, out);
  return hipGetLastError();
}

template <typename X>
hipError_t launch(Args<X> a, bool rotate, float* rows32, hipStream_t st) {
  if (!rotate) return by_types<X, 0>(a, st);
  if (a.K == 1024 && a.M <= 4) return by_types<X, 1024>(a, st);
  if (a.K == 4096 && a.M == 1) return by_types<X, 4096>(a, st);
  const hipError_t e = rotate_rows<X>(a.x, a.M, a.K, a.ldx, a.mult, rows32, st);
  if (e != hipSuccess) return e;
  const Args<float> b = {rows32, nullptr, a.wq, a.ws, a.bias, a.y, a.M, a.K, a.ldy, a.N, a.K, a.group, a.gelu, a.y_bf16};
  return by_types<float, 0>(b, st);
}

}  // namespace

hipError_t launch_w4a16(const void* X, bool x_bf16, int64_t M, int64_t K, int64_t ldx, bool rotate, const float* mult,
                        const uint8_t* Wq, const float* ws, int64_t group, const float* bias, int64_t N, bool gelu,
                        void* Y, bool y_bf16, int64_t ldy, float* rows32, hipStream_t st) {
  if (x_bf16) {
    const Args<__hip_bfloat16> a = {static_cast<const __hip_bfloat16*>(X), mult, Wq, ws, bias, Y, M, ldx, ldy, (int)N,
                                    (int)K, (int)group, gelu, y_bf16};
    return launch(a, rotate, rows32, st);
  }
  const Args<float> a = {static_cast<const float*>(X), mult, Wq, ws, bias, Y, M, ldx, ldy, (int)N, (int)K, (int)group,
                         gelu, y_bf16};
  return launch(a, rotate, rows32, st);
}

}  // namespace qv
