// Weights in 4-bit groups: what the products of few rows and of many share.
#pragma once
#include "bsq_device.h"
#include "bsq_internal.h"
#include "bsq_lds.h"

namespace bsqd {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

__device__ __forceinline__ float from_bf16(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// The activations' type in the matrix instructions: bf16 as they come, float32 as
// two fp16 parts of a scaled row.
template <typename X>
struct Mfma;
template <>
struct Mfma<uint16_t> {
  typedef bf16x8 V;
  static constexpr int parts = 1;
  static constexpr uint32_t ones = 0x3F803F80u;
  static __device__ __forceinline__ __bf16 near(float v) { return (__bf16)v; }
  static __device__ __forceinline__ f32x4 mul16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mul32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
  }
  template <bool HIGH>
  static __device__ __forceinline__ uint32_t pair(uint32_t bytes) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 512.0f, HIGH));
  }
};
template <>
struct Mfma<float> {
  typedef f16x8 V;
  static constexpr int parts = 2;
  static constexpr uint32_t ones = 0x3C003C00u;
  static __device__ __forceinline__ _Float16 near(float v) { return (_Float16)v; }
  static __device__ __forceinline__ f32x4 mul16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mul32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
  }
  template <bool HIGH>
  static __device__ __forceinline__ uint32_t pair(uint32_t bytes) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 512.0f, HIGH));
  }
};

// Eight codes (the lowest nibble first) as integers of that type. A byte below
// 16 is, read as E4M3, itself times 2^-9: its subnormals and its first binade
// have the same step.
template <typename X>
__device__ __forceinline__ u32x4 codes_of(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = w >> 4 & 0x0F0F0F0Fu;
  const uint32_t a = __builtin_amdgcn_perm(odd, even, 0x05010400u), b = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  return (u32x4){Mfma<X>::template pair<false>(a), Mfma<X>::template pair<true>(a), Mfma<X>::template pair<false>(b),
                 Mfma<X>::template pair<true>(b)};
}

// float32 activations as two fp16 parts: a row (or what a workgroup has of it) is
// scaled by the power of two that brings its largest value to [2^14, 2^15), which
// is exact, and each value is cut into its nearest fp16 and the nearest of the
// rest: 22 bits, down to 2^-16 of the largest; below that to 2^-39 of it. (Three
// bf16 parts would keep all 24 bits for half as many matrix instructions again;
// the float32 sums are off by more than the two bits.) Biased exponent of the
// factor for rows whose largest magnitude has these bits; rows with a NaN or an
// infinity go as they are.
__device__ __forceinline__ uint32_t row_factor(uint32_t most) {
  if (most >= 0x7F800000u) return 127;
  const int up = 141 - (int)(most >> 23);
  return (uint32_t)(127 + (up < 126 ? up : 126));
}
__device__ __forceinline__ float of_exponent(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, float f, u32x4& hi, u32x4& lo) {
  f16x8 h, l;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = (j < 4 ? a[j & 3] : b[j & 3]) * f;
    h[j] = (_Float16)y;
    l[j] = (_Float16)(y - (float)h[j]);
  }
  hi = __builtin_bit_cast(u32x4, h);
  lo = __builtin_bit_cast(u32x4, l);
}

}  // namespace bsqd

namespace bsqh {

// ---------------------------------------------------------------- few rows
constexpr int kFWaves = 8, kFThreads = 64 * kFWaves;
constexpr int kDeep = 3, kChunk = 256;
enum { kZeros, kPlain, kRagged };
constexpr int kFewLds = 163840 - 512, kFewRed = 2 * kFWaves * 1024;  // a CU's LDS but for the rows' largest values
constexpr int kFewHalf = 81920 - 512;
constexpr int kSlabLds = 131072;  // of x, but for the rows' 16 bytes more

// A row of k values of x in LDS: whole loads, and 16 bytes against bank conflicts.
__host__ __device__ constexpr int64_t few_pitch(int64_t k, int64_t size) { return (k * size + 1023) / 1024 * 1024 + 16; }
// Sums of x by groups, [group][row].
__host__ __device__ constexpr int64_t few_table(int64_t k, int64_t group, int mt) {
  return (k + kChunk - 1) / kChunk * (kChunk / group) * mt * 64;
}
__host__ inline int64_t share_bytes(int64_t M, int64_t K, int64_t group, int64_t size) {
  return M * few_pitch(K, size) + few_table(K, group, 1) + kFewRed;
}

// A launch of up to 16 rows (share), or of 16 mt rows by slabs of K, whose sums go
// to `parts` where there are several.
struct Int4Few {
  const void* x;
  int dtype;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  int64_t group;
  const float* bias;
  int64_t M, N, K;
  int mt;
  int64_t slab;
  int splits;
  float* parts;
  int64_t pitch_out;
  void* out;
  int out_f32;
};
void int4_share(const Int4Few& c, hipStream_t s);
void int4_slabs(const Int4Few& c, hipStream_t s);

}  // namespace bsqh
