// w4a16_gemv.hip -- few rows of unquantized activations times int4 weights with group scales, with the
// Hadamard rotation and smoothing of the activations on the way.
//
//   Y[m][n] = sum_g s[n][g] * (sum_{k in g} x[m][k] q[n][k]) (+ bias) (+ GELU),  q in [-8, 7]
//
// With a few rows the weights' N K / 2 bytes are all there is to move.  Small layers are bound by latency (a 1024 x
// 1024 layer takes 3.1 us unrotated and 4.5 us rotated for one row, in a graph whose empty nodes take about 2.5), large
// ones by the cache-line requests of a CU: 16 rows x 8192 x 16384 take 20-21 us, 72 MB at 3.4-3.7 TB/s (a copy's rate, 5.0
// TB/s, would be 14.4 us and the launch; fp32 rows, three pieces each, take 28.5 us, and one row 24).  There, without the
// scales' loads the kernel was 10 % faster, without the rows' 10 %, with codes read in pieces of 1 KB 10 %, while more loads in flight (two or four windows instead of one) changed
// nothing; hence fewer and fuller requests below.
//
// Products run on the matrix cores, 16 rows x 16 channels x 32 codes at a time, whatever M is: one
// v_mfma_f32_16x16x32_bf16 replaces 512 multiply-adds for 16 cycles, and the vector ALU is left with
// the unpacking.  Both operands are exact in bf16:
//   - a code is converted by itself (v_cvt_off_f32_i4 gives q / 16, and the upper halves of two are packed: 13
//     instructions for 8 codes).  24 + q, whose bits are one shift and one and-or for two codes (9 for 8), with
//     24 sum_k x[m][k] taken off each group's sum, would round every sum at the size of 24 |x|: a large activation against
//     a code of zero has to add nothing.
//   - an activation is a sum of NP bf16 pieces (the top 16 bits, then the top 16 bits of the rest, ...):
//     one piece is exact for bf16 rows, three are for fp32 and rotated rows (all 24 bits, whatever the result's type: two
//     would leave up to 2^-15 of each, all of one sign).
// A lane's 16-byte load holds 32 codes of one channel, and code i of dword j is contracted in MFMA j;
// the order of k inside the sum is free, so activations are read to match: lane (row r, quarter c)
// takes k = 32 c + 8 j + i of the 128-code window.
//
// The eight waves of a block take a run of windows each, and their sums are added over LDS.  The channels of a
// block go by the layer's width, so that one round of blocks fills the 256 CUs (us, one row of bf16):
//   K = 4096, N = 4096: 16 channels 5.1, 32 6.9, 64 10.6;   N = 8192: 8.4, 7.5, 10.9;   K = 8192, N = 16384: 21.3, 17.8, 19.1
//   and with 16 rows 25.2, 20.8, 20.7.  Fewer channels than 16 (narrow layers, K >= 2048): N = 1000, K = 4096, 16 rows, 16
//   channels 5.3, 4 channels 4.9; fp32, one rotated row 6.4 and 5.6.
// Rows beyond 16 count as blocks in that; where 16 to a block would take several rounds, bf16 rows go 32 to a block, which
// then unpacks each code for both halves: 32 rows x 4096 x 16384 in 22.8 and 16.0 us, 4096 x 4000 in 8.3 and 7.7.
// Rows are rotated by every block for itself, or by a kernel before.  Where blocks take turns on a CU, each rotates the rows
// again, so the rule goes by rounds of blocks as well (us, rotated in the block and before, bf16 rows):
//   K = 1024, 1 and 12 rows    N = 1024 4.6, 5.8 and 6.3, 6.4    N = 16384 (one round) 7.1, 8.5 and 9.3, 9.9
//                              N = 32768 15.5, 14.9 and 18.3, 16.2
//   K = 4096, N = 1024         1 row 5.8, 9.1    5 rows 9.4, 9.7
//             N = 32768        1 row 27.9, 30.7    3 rows 30.8, 31.6    4 rows 32.2, 31.7
//             N = 65536        1 row 56.4, 60.1    2 rows 59.4, 60.6    3 rows 62.1, 61.0
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fwht_regs.h"
#include "qv_decode_internal.h"

namespace qv {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 16;     // activation rows of a tile (the MFMA's M)
constexpr int kWindow = 128;  // codes of a window: one 16-byte load by each quarter of a wave

// Variants by size (measured above).
constexpr int64_t kCUs = 256;
constexpr int kFused1024 = 12, kFused4096 = 5;  // rows up to which every block rotates them by itself

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

// The low nibble of byte i of a dword -> q / 16, in one instruction.
template <int i>
__device__ __forceinline__ unsigned low_code(unsigned w) {
  unsigned f;
  if constexpr (i == 0)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(w));
  else if constexpr (i == 1)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(w));
  else if constexpr (i == 2)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(w));
  else
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(w));
  return f;
}

// Eight codes -> q / 16 in bf16, exactly, dword s holding codes s and s + 4.
__device__ __forceinline__ bf16x8 widen(unsigned w) {
  const unsigned odd = w >> 4;  // codes 1, 3, 5, 7 in the low nibbles
  u32x4 o;
  o[0] = __builtin_amdgcn_perm(low_code<2>(w), low_code<0>(w), 0x07060302u);
  o[1] = __builtin_amdgcn_perm(low_code<2>(odd), low_code<0>(odd), 0x07060302u);
  o[2] = __builtin_amdgcn_perm(low_code<3>(w), low_code<1>(w), 0x07060302u);
  o[3] = __builtin_amdgcn_perm(low_code<3>(odd), low_code<1>(odd), 0x07060302u);
  return __builtin_bit_cast(bf16x8, o);
}

__device__ __forceinline__ float gelu(float y) { return 0.5f * y * erfcf(-y * 0.70710678118654752f); }

// One butterfly stage across the lanes of a 16-lane row, self + sigma * partner, over 8 registers (see fwht_regs.h).
#define QV_DPP8(CTRL, R, S)                                                                                       \
  asm volatile(                                                                                                   \
      "s_nop 1\n\t"                                                                                               \
      "v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                         \
      "s_nop 1"                                                                                                   \
      : "+v"(R[0]), "+v"(R[1]), "+v"(R[2]), "+v"(R[3]), "+v"(R[4]), "+v"(R[5]), "+v"(R[6]), "+v"(R[7])            \
      : "v"(S))

// Sylvester-order Hadamard transform of up to B rows, each by K / 8 threads (t of them counted here), times
// mult / sqrt(K).  A wave holds 512 neighbouring elements, 8 a lane, and runs the stages of their 9 index
// bits in registers: bits 0-2 in the lane, 3-6 by DPP (the lanes' order and the sign that these stages leave
// are those of fwht_regs.h), 7 and 8 by changing lane bits 4 and 5 over with register bits 0 and 1.  The row then goes
// through LDS once and the remaining bits are in registers again.  The rows go side by side, so that they share the
// barriers.  What a thread reads from memory is loaded ahead; run() is called by every thread of a block.
template <int K, typename X, int B>
struct RotateRows {
  static_assert(K == 1024 || K == 4096, "Hadamard width");
  static constexpr float kNorm = K == 1024 ? 0.03125f : 0.015625f;
  static constexpr int kStep = K / 8;
  Eight<X> e[B];
  float f[8];

  __device__ __forceinline__ void load(int b, const X* __restrict__ x, int t) {
    load_eight(x + 8 * (chunk_of_lane16(t & 15) | (t & ~15)), e[b]);
  }
  __device__ __forceinline__ void load_mult(const float* __restrict__ mult, int t) {
    const float norm = (__builtin_popcount((t >> 3) & 15) & 1) ? -kNorm : kNorm;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = mult ? norm * mult[t + j * kStep] : norm;
  }

  // Butterflies over bits of the register number, bit values `from` to `to`.
  template <int from, int to>
  __device__ __forceinline__ static void butterflies(float (&v)[8]) {
#pragma unroll
    for (int h = from; h <= to; h <<= 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if ((j & h) == 0) {
          const float a = v[j], b = v[j + h];
          v[j] = a + b;
          v[j + h] = a - b;
        }
      }
    }
  }

  // Row b goes through LDS at row + b * stride; put(b, k, x) takes its results.  Rows from `count` on are left out (the
  // same in every thread).
  template <typename Put>
  __device__ __forceinline__ void run(float* row, int stride, int count, int t, Put put) const {
    const int lane = t & 63;
    // element of register 0 after the exchanges; register bits 0, 1, 2 are element bits 7, 8, 2
    float* const own = row + padded((t & ~63) * 8) + 8 * chunk_of_lane16(lane & 15) + 8 * (chunk_of_lane16(lane & 15) >> 3) +
                       ((lane >> 4) & 1) + 2 * ((lane >> 5) & 1);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (b >= count) break;
      float v[8];
      if constexpr (sizeof(X) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned w = e[b].d[i];
          v[2 * i] = bits_float(w << 16);
          v[2 * i + 1] = bits_float(w & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e[b].d[i >> 2][i & 3];
      }
      butterflies<1, 4>(v);
      QV_DPP8("quad_perm:[1,0,3,2]", v, stage_sigma(lane, 0));
      QV_DPP8("quad_perm:[2,3,0,1]", v, stage_sigma(lane, 1));
      QV_DPP8("row_ror:8", v, stage_sigma(lane, 2));
      QV_DPP8("row_mirror", v, stage_sigma(lane, 3));
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const auto x = __builtin_amdgcn_permlane16_swap(float_bits(v[j]), float_bits(v[j + 1]), false, false);
        const unsigned x0 = x[0], x1 = x[1];
        v[j] = bits_float(x0);
        v[j + 1] = bits_float(x1);
      }
      butterflies<1, 1>(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j & 2) continue;
        const auto x = __builtin_amdgcn_permlane32_swap(float_bits(v[j]), float_bits(v[j + 2]), false, false);
        const unsigned x0 = x[0], x1 = x[1];
        v[j] = bits_float(x0);
        v[j + 2] = bits_float(x1);
      }
      butterflies<2, 2>(v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        own[b * stride + padded(128) * (j & 1) + padded(256) * ((j >> 1) & 1) + 4 * (j >> 2)] = v[j];
    }
    __syncthreads();
    // bits 9-11 at K = 4096; at K = 1024 only bit 9, the last of the three
    float v[B][8];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (b >= count) break;
      const float* const x = row + b * stride + padded(t);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[b][j] = x[j * padded(kStep)];
      butterflies<K == 1024 ? 4 : 1, 4>(v[b]);
    }
    __syncthreads();  // the pieces may take the rows' place
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (b >= count) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) put(b, t + j * kStep, v[b][j] * f[j]);
    }
  }
};

// The NP pieces of activation k of a row, where the codes' order wants them: elements s and s + 4 of eight are neighbours.
// Piece p of the row lies p * stride further.
template <int NP>
__device__ __forceinline__ void put_pieces(uint16_t* row, int stride, int k, float x) {
  uint16_t* const to = row + (k & ~7) + 2 * (k & 3) + ((k >> 2) & 1);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const unsigned u = float_bits(x);
    to[p * stride] = (uint16_t)(u >> 16);
    x -= bits_float(u & 0xFFFF0000u);  // exact: the piece is the value's top bits
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
  int N, K, group, group_shift;  // a window's group: its first code >> group_shift
  int gelu, y_bf16;
};

// MT: tiles of 16 rows of a block.  NT: tiles of 16 channels.
// S: with few channels a tile has 16 / S of them and a load S windows, so that more blocks share the codes.
// SRC: where a wave's operands of the rows come from.
enum Source {
  kStaged,            // memory, through an LDS region of the wave's own, so that a row's window is read in one piece
  kRot1024, kRot4096  // LDS: the block rotates its rows into it first
};
template <int SRC>
constexpr int kWidth = SRC == kRot1024 ? 1024 : (SRC == kRot4096 ? 4096 : 0);

// LDS that a rotated row takes: as floats on its way, as pieces of K + 8 values in the end (the padding keeps 16 rows'
// operands in different banks).
template <int K, int NP>
__host__ __device__ constexpr int rotated_bytes() {
  return NP * (K + 8) * 2 > padded(K) * 4 ? NP * (K + 8) * 2 : padded(K) * 4;
}

// Rows that a block's rotation writes: at K = 1024 it takes four at a time.
template <int K>
__host__ __device__ constexpr int rotated_rows(int rows) {
  return K == 1024 ? (rows + 3) & ~3 : rows;
}

template <typename X, int NP, int MT, int NT, int S, int SRC>
__global__ __launch_bounds__(kThreads) void w4a16_kernel(Args<X> a) {
  static_assert(NT == 1 || S == 1, "few channels or many");
  static_assert(MT == 1 || (S == 1 && SRC == kStaged), "more than 16 rows come from memory");
  constexpr int kDepth = NT == 1 ? 4 : 2;  // loads in flight of each tile
  constexpr int kChannels = 16 / S;        // of a tile
  constexpr int K = kWidth<SRC>;
  extern __shared__ f32x4 lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int sub = S == 1 ? 0 : r / kChannels;  // which of S windows this lane loads
  const int n0 = blockIdx.x * (kChannels * NT);
  const int64_t m0 = (int64_t)blockIdx.y * (MT * kRows);
  const int rows = (int)(a.M - m0 < MT * kRows ? a.M - m0 : MT * kRows);
  const int windows = a.K / kWindow, groups = a.K / a.group;
  // Rotation: `kAtOnce` rows side by side, as often as there are rows.
  constexpr int kHadamard = K ? K : 1024;  // unused without a rotation
  constexpr int kAtOnce = 8 * kThreads / kHadamard, kBatch = kAtOnce == 1 ? kFused4096 : (kFused1024 + 3) / 4;
  const int part = threadIdx.x / (kHadamard / 8), in_row = threadIdx.x % (kHadamard / 8);
  RotateRows<kHadamard, X, kBatch> rotation;
  if constexpr (K != 0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int m = i * kAtOnce + part;
      if (i * kAtOnce < rows) rotation.load(i, a.x + (m0 + (m < rows ? m : rows - 1)) * a.ldx, in_row);
    }
    rotation.load_mult(a.mult, in_row);
  }

  // A wave's windows follow each other, so that both halves of a 128-byte line are asked for together.
  const int share = (windows + S * kWaves - 1) / (S * kWaves) * S;
  const int begin = wave * share, end = begin + share < windows ? begin + share : windows;

  const uint8_t* const wbase = a.wq + (int64_t)n0 * (a.K / 2);
  const float* const sbase = a.ws + (int64_t)n0 * groups;
  uint32_t wrow[NT], srow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int in_tile = S == 1 ? r : r % kChannels;
    const int n = n0 + 16 * t + in_tile < a.N ? 16 * t + in_tile : a.N - 1 - n0;
    wrow[t] = (uint32_t)n * (a.K / 2) + 16 * c;
    srow[t] = (uint32_t)n * groups;
  }
  u32x4 w[kDepth][NT];
  auto load_codes = [&](int d, int win) {
    const int mine = S == 1 || win + sub < windows ? win + sub : windows - 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      w[d][t] = *reinterpret_cast<const u32x4*>(wbase + wrow[t] + (uint32_t)mine * (kWindow / 2));
  };
  // Scales of 4 S windows at a time: quarter c of the wave loads those of the load first + c.
  float s[NT];
  auto load_scales = [&](int first) {
    const int win = first + S * c + sub;
    const uint32_t g = (uint32_t)((win < end ? win : end - 1) * kWindow) >> a.group_shift;
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t] = S == 1 || win < end ? sbase[srow[t] + g] : 0.0f;
  };
  if (begin < end) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (begin + d * S < end) load_codes(d, begin + d * S);
    load_scales(begin);
  }

  char* const room = reinterpret_cast<char*>(lds);
  constexpr int kPieceRow = K + 8;
  uint16_t* const split_rows = reinterpret_cast<uint16_t*>(room);
  if constexpr (K != 0) {
    rotation.run(reinterpret_cast<float*>(room) + part * padded(K), kAtOnce * padded(K), (rows + kAtOnce - 1) / kAtOnce,
                 in_row, [&](int b, int k, float x) {
                   put_pieces<NP>(split_rows + (b * kAtOnce + part) * NP * kPieceRow, kPieceRow, k, x);
                 });
  }
  int row[MT];
#pragma unroll
  for (int u = 0; u < MT; ++u) row[u] = kRows * u + r < rows ? kRows * u + r : rows - 1;

  // Staged rows: a wave reads its window of every row in one piece, 16 bytes a lane, and holds the next
  // one while it works; 16 bytes of padding a row keep the 16 rows' fragments in different banks.
  constexpr int kPerLoad = 16 / (int)sizeof(X);      // activations
  constexpr int kLanesPerRow = kWindow / kPerLoad;   // 16 (bf16) or 32 (fp32)
  constexpr int kRowsPerLoad = 64 / kLanesPerRow;
  constexpr int kLoads = MT * kRows / kRowsPerLoad;
  constexpr int kStageRow = kWindow + kPerLoad;      // activations
  X* const stage = reinterpret_cast<X*>(room) + wave * (rows * kStageRow);
  const int stage_row = lane / kLanesPerRow, stage_k = (lane % kLanesPerRow) * kPerLoad;
  u32x4 xs[K == 0 ? kLoads : 1];
  auto load_stage = [&](int win) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i * kRowsPerLoad >= rows) break;
      const int m = i * kRowsPerLoad + stage_row;
      xs[i] = *reinterpret_cast<const u32x4*>(a.x + (m0 + (m < rows ? m : rows - 1)) * a.ldx + win * kWindow + stage_k);
    }
  };
  if constexpr (K == 0) {
    if (begin < end) load_stage(begin);
  }
  if constexpr (K != 0) __syncthreads();

  f32x4 y[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u) y[t][u] = f32x4{0, 0, 0, 0};

  // The rows' operands of a window.
  bf16x8 xf[MT][4][NP];
  auto take_rows = [&](int win) {
    if constexpr (K == 0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (i * kRowsPerLoad >= rows) break;
        const int m = i * kRowsPerLoad + stage_row;
        if (m < rows) *reinterpret_cast<u32x4*>(stage + m * kStageRow + stage_k) = xs[i];
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (win + 1 < end) load_stage(win + 1);
    }
#pragma unroll
    for (int u = 0; u < MT; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (K != 0) {
#pragma unroll
          for (int p = 0; p < NP; ++p)
            xf[u][j][p] = *reinterpret_cast<const bf16x8*>(split_rows + (row[u] * NP + p) * kPieceRow + win * kWindow +
                                                           32 * c + 8 * j);
        } else {
          Eight<X> e;
          load_eight(stage + row[u] * kStageRow + 32 * c + 8 * j, e);
          pieces<NP>(e, xf[u][j]);
        }
      }
    }
    if constexpr (K == 0) __builtin_amdgcn_wave_barrier();
  };
  auto product = [&](const u32x4& codes, f32x4 (&acc)[MT]) {
#pragma unroll
    for (int u = 0; u < MT; ++u) acc[u] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 wf = widen(codes[j]);
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int p = 0; p < NP; ++p)
          acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[u][j][p], wf, acc[u], 0, 0, 0);
    }
  };
  auto add = [&](f32x4& to, float f, const f32x4& acc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] += 16.0f * f * acc[i];
  };

  for (int first = begin; first < end; first += 4 * S) {
    float sc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) sc[t] = s[t];
    if (first + 4 * S < end) load_scales(first + 4 * S);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int win = first + d * S;
      if (win >= end) break;
      f32x4 acc[NT][MT];
      if constexpr (S == 1) {
        take_rows(win);
#pragma unroll
        for (int t = 0; t < NT; ++t) product(w[d % kDepth][t], acc[t]);
      } else {
        // A load's columns belong to S windows: each window's product is taken with all of them and its own are kept.
        bf16x8 wf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) wf[j] = widen(w[d][0][j]);
        acc[0][0] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < S; ++u) {
          if (win + u >= end) break;
          take_rows(win + u);
          f32x4 x = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int p = 0; p < NP; ++p) x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[0][j][p], wf[j], x, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[0][0][i] = sub == u ? x[i] : acc[0][0][i];
        }
      }
      if (win + kDepth * S < end) load_codes(d % kDepth, win + kDepth * S);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f = __shfl(sc[t], r + 16 * d);
#pragma unroll
        for (int u = 0; u < MT; ++u) add(y[t][u], f, acc[t][u]);
      }
    }
  }

  // Element (m, n) of channel tile t and row tile u at [wave][t][u][m][n].
  if constexpr (K == 0) __syncthreads();  // the sums take the staging regions' place
  float* const red = reinterpret_cast<float*>(room + (K ? rotated_rows<K>(rows) * rotated_bytes<K, NP>() : 0));
  constexpr int kTiles = NT * MT;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[((wave * NT + t) * MT + u) * 256 + (4 * c + i) * 16 + r] = y[t][u][i];
  __syncthreads();
  for (int idx = threadIdx.x; idx < 256 * kTiles; idx += kThreads) {
    const int t = idx / (256 * MT), m = (idx >> 4) & (16 * MT - 1), n = n0 + 16 * t + (idx & 15);
    if (m >= rows || n >= a.N || (S > 1 && (idx & 15) >= kChannels)) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
#pragma unroll
      for (int u = 0; u < S; ++u) v += red[k * kTiles * 256 + idx + u * kChannels];
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
  const int t = threadIdx.x;
  RotateRows<K, X, 1> rotation;
  rotation.load(0, x + (int64_t)blockIdx.x * ldx, t);
  rotation.load_mult(mult, t);
  float* const to = out + (int64_t)blockIdx.x * K;
  rotation.run(reinterpret_cast<float*>(row4), 0, 1, t, [&](int, int k, float v) { to[k] = v; });
}

template <typename X, int NP, int MT, int NT, int S, int SRC>
hipError_t launch_kernel(const Args<X>& a, hipStream_t st) {
  constexpr int K = kWidth<SRC>;
  constexpr int kBlock = 16 / S * NT;  // channels
  const unsigned gx = (unsigned)((a.N + kBlock - 1) / kBlock);
  const int rows = (int)(a.M < MT * kRows ? a.M : MT * kRows);
  size_t bytes = (size_t)kWaves * NT * MT * 256 * 4;
  if (K) {
    bytes += (size_t)rotated_rows<K>(rows) * rotated_bytes<K, NP>();
  } else {
    const size_t staged = (size_t)kWaves * rows * (kWindow * sizeof(X) + 16);
    if (bytes < staged) bytes = staged;
  }
  if (bytes > 65536) {
    static std::atomic<uint64_t> raised{0};  // a bit for each device whose limit was raised for this kernel
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(&w4a16_kernel<X, NP, MT, NT, S, SRC>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
      if (e != hipSuccess) return e;
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  // grid.y holds 65535 blocks: longer runs go in several launches
  const int64_t step = (int64_t)65535 * MT * kRows;
  for (int64_t m = 0; m < a.M; m += step) {
    Args<X> b = a;
    b.x += m * a.ldx;
    b.M = a.M - m < step ? a.M - m : step;
    b.y = static_cast<char*>(a.y) + m * a.ldy * (a.y_bf16 ? 2 : 4);
    w4a16_kernel<X, NP, MT, NT, S, SRC>
        <<<dim3(gx, (unsigned)((b.M + MT * kRows - 1) / (MT * kRows))), kThreads, bytes, st>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename X, int NP, int SRC>
hipError_t by_tiles(const Args<X>& a, hipStream_t st) {
  // The fewest channels a block with which one round of blocks holds the layer, 64 at most.
  auto fits = [&](int rows, int channels, int blocks_a_cu = 1) {
    return ((a.M + rows - 1) / rows) * ((a.N + channels - 1) / channels) <= blocks_a_cu * kCUs;
  };
  // Rows of one piece (more do not fit the registers) go 32 to a block where 16 would take several rounds.
  if constexpr (SRC == kStaged && NP == 1) {
    if (a.M > kRows && !fits(kRows, 16)) {
      if (fits(2 * kRows, 16)) return launch_kernel<X, NP, 2, 1, 1, SRC>(a, st);
      if (fits(2 * kRows, 32)) return launch_kernel<X, NP, 2, 2, 1, SRC>(a, st);
      return launch_kernel<X, NP, 2, 4, 1, SRC>(a, st);
    }
  }
  // Two blocks of 32 channels share a CU where their registers (bf16 rows) and LDS (rotated rows) allow it; with more than
  // a few rows, reading the rows twice costs more than that gives: K = 4096, N = 16384, rows read and 1, 8, 16 of them 10.6, 11.5,
  // 12.9 us (64 channels: 11.8, 12.2, 12.9), rotated and 1, 2, 3 of them 13.3, 14.4, 20.5 us (15.1, 15.7, 16.5).
  const bool two = sizeof(X) == 2 && a.M <= (SRC == kStaged ? 8 : (SRC == kRot1024 ? 3 : 2));
  if (!fits(kRows, 32, two ? 2 : 1)) return launch_kernel<X, NP, 1, 4, 1, SRC>(a, st);
  if (!fits(kRows, 16)) return launch_kernel<X, NP, 1, 2, 1, SRC>(a, st);
  if constexpr (SRC != kRot1024) {  // K = 1024 has 8 windows, one for each wave
    if (a.K >= 4 * kWaves * kWindow && fits(kRows, 4)) return launch_kernel<X, NP, 1, 1, 4, SRC>(a, st);
    if (a.K >= 2 * kWaves * kWindow && fits(kRows, 8)) return launch_kernel<X, NP, 1, 1, 2, SRC>(a, st);
  }
  return launch_kernel<X, NP, 1, 1, 1, SRC>(a, st);
}

// Pieces by the type: rows that are bf16 are one piece, others three.
template <typename X, int SRC>
hipError_t by_types(const Args<X>& a, hipStream_t st) {
  return by_tiles<X, sizeof(X) == 2 && kWidth<SRC> == 0 ? 1 : 3, SRC>(a, st);
}

template <typename X>
hipError_t launch(const Args<X>& a, bool rotate, float* rows32, hipStream_t st) {
  if (!rotate) return by_types<X, kStaged>(a, st);
  const int64_t rounds = (a.N + 64 * kCUs - 1) / (64 * kCUs);  // of blocks of 64 channels
  const int64_t fused = a.K == 1024 ? (rounds == 1 ? kFused1024 : 0) : (rounds == 1 ? kFused4096 : (rounds == 2 ? 3 : 2));
  if (a.M <= fused) return a.K == 1024 ? by_types<X, kRot1024>(a, st) : by_types<X, kRot4096>(a, st);
  constexpr int64_t kStep = int64_t{1} << 20;  // rows of a launch, which holds fewer than 2^32 threads
  for (int64_t m = 0; m < a.M; m += kStep) {
    const unsigned rows = (unsigned)(a.M - m < kStep ? a.M - m : kStep);
    if (a.K == 1024)
      rotate_rows_kernel<1024, X><<<rows, 128, 0, st>>>(a.x + m * a.ldx, a.ldx, a.mult, rows32 + m * a.K);
    else
      rotate_rows_kernel<4096, X><<<rows, 512, 0, st>>>(a.x + m * a.ldx, a.ldx, a.mult, rows32 + m * a.K);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const Args<float> b = {rows32, nullptr, a.wq, a.ws, a.bias, a.y, a.M, a.K, a.ldy, a.N, a.K, a.group,
                         a.group_shift, a.gelu, a.y_bf16};
  return by_types<float, kStaged>(b, st);
}

}  // namespace

hipError_t launch_w4a16(const void* X, bool x_bf16, int64_t M, int64_t K, int64_t ldx, bool rotate, const float* mult,
                        const uint8_t* Wq, const float* ws, int64_t group, const float* bias, int64_t N, bool gelu,
                        void* Y, bool y_bf16, int64_t ldy, float* rows32, hipStream_t st) {
  // group is 128, 256 or 512, or K: one group
  const int shift = group == K ? 30 : (group == 128 ? 7 : (group == 256 ? 8 : 9));
  if (x_bf16) {
    const Args<__hip_bfloat16> a = {static_cast<const __hip_bfloat16*>(X), mult, Wq, ws, bias, Y, M, ldx, ldy, (int)N,
                                    (int)K, (int)group, shift, gelu, y_bf16};
    return launch(a, rotate, rows32, st);
  }
  const Args<float> a = {static_cast<const float*>(X), mult, Wq, ws, bias, Y, M, ldx, ldy, (int)N, (int)K, (int)group,
                         shift, gelu, y_bf16};
  return launch(a, rotate, rows32, st);
}

}  // namespace qv
