// Weights in 4-bit integers with a scale, and a zero point, for each group of
// 32, 64 or 128 neighbours along K; products with unquantized activations.
//
//   w[n, k] = (q[n, k] - z[n, g]) s[n, g],  g = k / group, q and z in 0..15, z = 8 where there are no zero points
//   y[m, n] = sum_k x[m, k] w[n, k] + bias[n]
//
// The products compute with integers, which bf16 holds exactly, and bring the
// scale in once a group, in float32:
//   y[m, n] = sum_g s[n, g] sum_(k in g) (q[n, k] - z[n, g]) x[m, k]
// so that float32 sums are the only roundings before the output's. float32
// activations go as three bf16 parts whose sum they are (24 bits in 8 + 8 + 8).
#include <type_traits>

#include "bsq_device.h"
#include "bsq_internal.h"
#include "bsq_lds.h"

using namespace bsqd;

namespace {

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

// ---------------------------------------------------------------- quantizer
constexpr int kQThreads = 256;

__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = a[j];
  }
}
__device__ __forceinline__ void load16(const uint16_t* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const u32x4 a = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[8 * i + 2 * j] = bf16_lo(a[j]), v[8 * i + 2 * j + 1] = bf16_hi(a[j]);
  }
}

// rint(v / s), half to even, as if the quotient were exact: the reciprocal's
// product is off by far less than a half, and the remainder v - t s, which one
// fused operation gives exactly (s has 8 significant bits, t has 4), tells
// whether a neighbour is nearer.
__device__ __forceinline__ float rounded_quotient(float v, float s, float inv) {
  float t = rintf(v * inv);
  const float r = __builtin_fmaf(-t, s, v), half = 0.5f * s;
  if (r > half) t += 1.0f;
  else if (r < -half) t -= 1.0f;
  else if (fabsf(r) == half && ((int)t & 1)) t += r > 0.0f ? 1.0f : -1.0f;
  return t;
}

// A lane holds 16 neighbours; G / 16 lanes share a group. The weights are one
// long array of groups: K is whole groups. Bound by memory.
template <typename T, int G>
__global__ __launch_bounds__(kQThreads) void k_quant_int4(const T* __restrict__ w, int64_t units, int symmetric,
                                                         u32x2* __restrict__ codes, uint16_t* __restrict__ scales,
                                                         uint8_t* __restrict__ zeros) {
  constexpr int L = G / 16;
  const int64_t u = (int64_t)blockIdx.x * kQThreads + threadIdx.x;
  const bool ok = u < units;  // the lanes of a group end together
  float v[16];
  load16(w + (ok ? u : 0) * 16, v);
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    lo = __builtin_elementwise_minimum(lo, v[i]);  // NaN if one is
    hi = __builtin_elementwise_maximum(hi, v[i]);
  }
#pragma unroll
  for (int o = 1; o < L; o *= 2) {
    lo = __builtin_elementwise_minimum(lo, __shfl_xor(lo, o, 64));
    hi = __builtin_elementwise_maximum(hi, __shfl_xor(hi, o, 64));
  }
  float range;
  if (symmetric) range = __builtin_elementwise_maximum(-lo, hi) / 7.0f;
  else range = (float)(((double)hi - (double)lo) / 15.0);  // the difference of two floats may need 64 bits
  uint32_t b = __builtin_bit_cast(uint16_t, (__bf16)range);
  if (!(range < __builtin_inff())) b = 0x7FC0;  // NaN or an infinity in the group: no codes stand for it
  else if (b < 0x0080) b = 0x3F80;              // below the normal range: all codes stand for 0
  const float s = from_bf16((uint16_t)b), inv = 1.0f / s;
  float z = 8.0f;
  if (!symmetric) z = fminf(fmaxf(rounded_quotient(-lo, s, inv), 0.0f), 15.0f);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = fminf(fmaxf(rounded_quotient(v[i], s, inv) + z, 0.0f), 15.0f);
    c[i / 8] |= (uint32_t)(int)q << (4 * (i % 8));
  }
  if (!ok) return;
  codes[u] = (u32x2){c[0], c[1]};
  if (u % L == 0) {
    scales[u / L] = (uint16_t)b;
    if (zeros) zeros[u / L] = (uint8_t)(int)z;
  }
}

// Pieces of 16 bytes of the output, neighbouring lanes side by side: bound by
// memory (a lane's four pieces side by side took 22 us for 2048 x 7168 float32).
constexpr int kDPieces = 4;
template <typename T>
__global__ __launch_bounds__(kQThreads) void k_dequant_int4(const uint8_t* __restrict__ codes,
                                                           const uint16_t* __restrict__ scales,
                                                           const uint8_t* __restrict__ zeros, int64_t pieces, int shift,
                                                           T* __restrict__ out) {
  constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < kDPieces; ++i) {
    const int64_t p = ((int64_t)blockIdx.x * kDPieces + i) * kQThreads + threadIdx.x;
    if (p >= pieces) return;
    uint32_t c = 0;
    __builtin_memcpy(&c, __builtin_assume_aligned(codes + p * (E / 2), E / 2), E / 2);
    const int64_t g = p * E >> shift;
    const float s = from_bf16(scales[g]), z = zeros ? (float)zeros[g] : 8.0f;
    float v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = ((float)(c >> (4 * j) & 15u) - z) * s;
    if constexpr (E == 4) {
      *reinterpret_cast<f32x4*>(out + p * E) = (f32x4){v[0], v[1], v[2], v[3]};
    } else {
      bf16x8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (__bf16)v[j];
      *reinterpret_cast<bf16x8*>(out + p * E) = o;
    }
  }
}

// ---------------------------------------------------------------- operands
// Eight codes (the lowest nibble first) as bf16 integers. A byte below 16 is,
// read as E4M3, itself times 2^-9: its subnormals and its first binade have the
// same step.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = w >> 4 & 0x0F0F0F0Fu;
  const uint32_t a = __builtin_amdgcn_perm(odd, even, 0x05010400u), b = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  union {
    bf16x2 p[4];
    bf16x8 v;
  } r;
  r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, false);
  r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, true);
  r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, false);
  r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, true);
  return r.v;
}

// Eight activations as bf16 parts, the smallest part first.
template <typename X>
struct Parts;
template <>
struct Parts<uint16_t> {
  static constexpr int n = 1;
  bf16x8 p[1];
  __device__ __forceinline__ void load(const uint8_t* at) { p[0] = *reinterpret_cast<const bf16x8*>(at); }
};
template <>
struct Parts<float> {
  static constexpr int n = 3;
  bf16x8 p[3];
  __device__ __forceinline__ void load(const uint8_t* at) {
    const f32x4 a = reinterpret_cast<const f32x4*>(at)[0], b = reinterpret_cast<const f32x4*>(at)[1];
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[2];
      v[0] = i < 2 ? a[2 * (i & 1)] : b[2 * (i & 1)];
      v[1] = i < 2 ? a[2 * (i & 1) + 1] : b[2 * (i & 1) + 1];
#pragma unroll
      for (int part = 2; part >= 0; --part) {  // cut off the upper 16 bits: the rest is exact
        const uint32_t u0 = __float_as_uint(v[0]), u1 = __float_as_uint(v[1]);
        w[part][i] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
        v[0] -= __uint_as_float(u0 & 0xFFFF0000u);
        v[1] -= __uint_as_float(u1 & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int part = 0; part < 3; ++part) p[part] = __builtin_bit_cast(bf16x8, (u32x4){w[part][0], w[part][1], w[part][2], w[part][3]});
  }
};

// ---------------------------------------------------------------- few rows
// Up to 16 rows of activations, which stay in LDS: bound by reading the weights
// once. A workgroup of eight waves takes tiles of 16 weight rows one after the
// other; its waves share K, in chunks of 128, of which each keeps kDeep on their
// way in registers, across tiles. The partial sums meet in LDS.
//
// Lane l holds row l % 16's codes [32 p, 32 p + 32) of a chunk, p = l / 16, as
// one 16-byte load. Matrix instruction i multiplies one word of each lane: 32
// codes of the chunk. Groups of 128 take them as they lie; for shorter groups
// lanes exchange words first, so that the 32 codes are of one group.
//
// Zero points: sum (q - z) x = sum q x - z sum x, the second sum by the same
// instruction with ones.
constexpr int kFWaves = 8, kFThreads = 64 * kFWaves;
constexpr int kFewRows = 16;
constexpr int kDeep = 4;
constexpr int kFewLds = 163840, kFewRed = 2 * kFWaves * 1024;

template <typename X>
__host__ __device__ constexpr int64_t few_pitch(int64_t K) {  // a row of x: whole loads, and 16 bytes against bank conflicts
  return (K * (int64_t)sizeof(X) + 1023) / 1024 * 1024 + 16;
}

template <int G>
__device__ __forceinline__ void regroup(u32x4& w) {
  if constexpr (G == 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[2], w[3], false, false);
    w = (u32x4){a[0], b[0], a[1], b[1]};
  } else if constexpr (G == 32) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = (u32x4){c[0], c[1], d[0], d[1]};
  }
}
// Where in the chunk the eight codes begin that lane group p holds in word i after regroup().
template <int G>
__device__ __forceinline__ int place_of(int p, int i) {
  if constexpr (G == 128) return p * 32 + i * 8;
  else if constexpr (G == 64) return (i >> 1) * 64 + (p & 1) * 32 + (p >> 1) * 8 + (i & 1) * 16;
  else return i * 32 + p * 8;
}

struct Chunk {
  u32x4 w;
  uint32_t s[2], z;  // scales and zero points of its groups, the first lowest
};

// BYTES of LDS: half of a CU's where that does, for two workgroups a CU.
template <typename X, typename T, int G, int BYTES>
__global__ __launch_bounds__(kFThreads) void k_linear_int4_few(const X* __restrict__ x, const uint8_t* __restrict__ codes,
                                                              const uint16_t* __restrict__ scales,
                                                              const uint8_t* __restrict__ zeros,
                                                              const float* __restrict__ bias, int M, int64_t N, int K,
                                                              T* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[BYTES];
  f32x4* red = reinterpret_cast<f32x4*>(lds);  // [2][waves][64]
  uint8_t* xs = lds + kFewRed;
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63, col = lane & 15, p = lane >> 4;
  const int pitch = (int)few_pitch<X>(K), row_loads = pitch / 1024;
  {
    const rsrc_words d = descriptor(x, (uint32_t)M * K * (uint32_t)sizeof(X));
    const uint32_t base = lds_offset(xs), row_bytes = (uint32_t)K * sizeof(X);
    for (int i = wave; i < M * row_loads; i += kFWaves) {
      const int r = i / row_loads, c = i - r * row_loads;
      const uint32_t at = c * 1024 + lane * 16;
      load_to_lds<16>(d, buffer_at(true, at < row_bytes, (uint32_t)r * row_bytes + at, 0), base + r * pitch + c * 1024);
    }
  }
  const int64_t tiles = (N + 15) / 16;
  const int chunks = (K + 127) / 128, KG = K / G;
  const int c0 = chunks * wave / kFWaves, nc = chunks * (wave + 1) / kFWaves - c0;
  constexpr int GP = 128 / G;  // groups of a chunk
  int64_t ft = blockIdx.x;     // the tile and the chunk that are asked for next
  int fc = 0;
  const uint8_t* at_w;
  const uint16_t* at_s;
  const uint8_t* at_z;
  auto aim = [&] {  // this lane's row of the tile
    int64_t n = ft * 16 + col;
    if (n >= N) n = N - 1;
    at_w = codes + n * (K / 2) + c0 * 64 + p * 16;
    at_s = scales + n * KG + c0 * GP;
    at_z = zeros ? zeros + n * KG + c0 * GP : nullptr;
  };
  auto fetch = [&](Chunk& f) {
    const int c = c0 + fc;
    if (c * 128 + p * 32 < K) f.w = *reinterpret_cast<const u32x4*>(at_w + fc * 64);
    else f.w = (u32x4){0, 0, 0, 0};
    f.s[0] = f.s[1] = 0;
    f.z = 0x08080808u;
    const int g = fc * GP;
    if (GP == 1 || (c + 1) * GP <= KG) {
      __builtin_memcpy(f.s, at_s + g, 2 * GP);
      if (zeros) __builtin_memcpy(&f.z, at_z + g, GP);
    } else {  // the last groups of a row
#pragma unroll
      for (int j = 0; j < GP; ++j)
        if (c * GP + j < KG) {
          f.s[j / 2] |= (uint32_t)at_s[g + j] << (16 * (j & 1));
          if (zeros) f.z = (f.z & ~(0xFFu << (8 * j))) | (uint32_t)at_z[g + j] << (8 * j);
        }
    }
    if (++fc == nc) {
      fc = 0;
      ft += gridDim.x;
      if (ft < tiles) aim();
    }
  };
  Chunk ring[kDeep];
  if (nc) {
    aim();
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
      if (ft < tiles) fetch(ring[d]);
  }
  wait_loads<0>();
  __syncthreads();
  const int row = col < M ? col : 0;  // lanes past M repeat row 0
  const uint8_t* mine = xs + row * pitch;
  const bf16x8 ones = __builtin_bit_cast(bf16x8, (u32x4){0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  f32x4 acc = {0, 0, 0, 0};
  auto multiply = [&](Chunk f, int c) {
    regroup<G>(f.w);
    const bool whole = c * 128 + 128 <= K;
#pragma unroll
    for (int j = 0; j < GP; ++j) {
      f32x4 sum = {0, 0, 0, 0}, of_x = {0, 0, 0, 0};
#pragma unroll
      for (int i = j * (4 / GP); i < (j + 1) * (4 / GP); ++i) {
        const int k = c * 128 + place_of<G>(p, i);
        Parts<X> a;
        a.load(mine + k * sizeof(X));
        const bf16x8 b = codes_bf16(f.w[i]);
#pragma unroll
        for (int part = 0; part < Parts<X>::n; ++part) {
          if (!whole && k >= K) a.p[part] = __builtin_bit_cast(bf16x8, (u32x4){0, 0, 0, 0});  // past the row: anything may lie there
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[part], b, sum, 0, 0, 0);
          of_x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[part], ones, of_x, 0, 0, 0);
        }
      }
      const float s = __uint_as_float(j & 1 ? f.s[j / 2] & 0xFFFF0000u : f.s[j / 2] << 16);
      const float z = (float)(f.z >> (8 * j) & 0xFFu);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(s, __builtin_fmaf(-z, of_x[r], sum[r]), acc[r]);
    }
  };
  int buf = 0;
  auto finish = [&](int64_t tile) {
    red[(buf * kFWaves + wave) * 64 + lane] = acc;
    acc = (f32x4){0, 0, 0, 0};
    __syncthreads();
    if (t < 256) {
      float y = 0.0f;
#pragma unroll
      for (int w = 0; w < kFWaves; ++w) y += reinterpret_cast<const float*>(red)[(buf * kFWaves + w) * 256 + t];
      // float t of a partial tile: register t % 4 of lane t / 4
      const int m = (t >> 6) * 4 + (t & 3);
      const int64_t n = tile * 16 + (t >> 2 & 15);
      if (m < M && n < N) {
        if (bias) y += bias[n];
        store1(out + m * N + n, y);
      }
    }
    buf ^= 1;  // the next tile's sums go elsewhere: its barrier stands between this one's reads and their reuse
  };
  if (nc == 0) {
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) finish(tile);
    return;
  }
  int64_t tile = blockIdx.x;
  int c = 0;
  while (tile < tiles) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (tile < tiles) {
        multiply(ring[d], c0 + c);
        if (ft < tiles) fetch(ring[d]);
        if (++c == nc) {
          finish(tile);
          c = 0;
          tile += gridDim.x;
        }
      }
    }
  }
}

int64_t few_rows(int64_t K, int dtype) {  // rows of x that fit
  const int64_t pitch = dtype == BSQ_F32 ? few_pitch<float>(K) : few_pitch<uint16_t>(K);
  const int64_t rows = (kFewLds - kFewRed) / pitch;
  return rows < kFewRows ? rows : kFewRows;
}

template <typename X, typename T, int G>
void launch_few(const X* x, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const float* bias,
                int64_t M, int64_t N, int64_t K, T* out, hipStream_t s) {
  const int64_t bytes = M * few_pitch<X>(K) + kFewRed, tiles = (N + 15) / 16;
  const bool half = bytes <= kFewLds / 2;
  const int64_t most = bsqh::device_cus() * (half ? 2 : 1);
  const dim3 grid((unsigned)(tiles < most ? tiles : most));
  if (half)
    hipLaunchKernelGGL((k_linear_int4_few<X, T, G, kFewLds / 2>), grid, dim3(kFThreads), 0, s, x, codes, scales, zeros,
                       bias, (int)M, N, (int)K, out);
  else
    hipLaunchKernelGGL((k_linear_int4_few<X, T, G, kFewLds>), grid, dim3(kFThreads), 0, s, x, codes, scales, zeros, bias,
                       (int)M, N, (int)K, out);
}

// ---------------------------------------------------------------- many rows
// The weights are unpacked to bf16 integers q - z once for all rows of
// activations (2 bytes each in the workspace, a slice of the rows of weights at
// a time), their scales turned to [group][row]; then tiles by matrix
// instructions, with the scales brought in at the end of each group: a tile has
// one set of accumulators for the group and one for the sum over groups.
//
// PL parts of the activations: 1 (bf16) or 2 (float32, split beforehand).
constexpr int kUThreads = 256;
template <typename V>
__global__ __launch_bounds__(kUThreads) void k_unpack_int4(const u32x2* __restrict__ codes,
                                                          const uint16_t* __restrict__ scales,
                                                          const uint8_t* __restrict__ zeros, int64_t units, int lanes,
                                                          int KG, int64_t pitch, V* __restrict__ w,
                                                          float* __restrict__ turned) {
  const int64_t u = (int64_t)blockIdx.x * kUThreads + threadIdx.x;
  if (u >= units) return;
  const u32x2 c = codes[u];
  const int64_t g = u / lanes;
  const float z = zeros ? (float)zeros[g] : 8.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    V v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (decltype(v[0] + v[0]))((float)(c[i] >> (4 * j) & 15u) - z);
    w[u * 2 + i] = v;
  }
  if (u % lanes == 0) turned[g % KG * pitch + g / KG] = from_bf16(scales[g]);
}

// float32 activations as two planes of fp16: a row is scaled by the power of two
// that brings its largest value to [2^14, 2^15), which is exact, and each value
// is cut into its nearest fp16 and the nearest of the rest: 22 bits, down to 2^-16
// of the row's largest; below that to 2^-39 of it. (Three bf16 planes would keep
// all 24 bits for half as many matrix instructions again; the float32 sums are
// off by more than the two bits.) A workgroup a row.
__global__ __launch_bounds__(kUThreads) void k_split_f32(const f32x4* __restrict__ x, int64_t rows, int K,
                                                        f16x8* __restrict__ planes, float* __restrict__ back) {
  __shared__ float red[kUThreads / 64];
  const int64_t row = blockIdx.x;
  const f32x4* from = x + row * (K / 4);
  float most = 0.0f;
  for (int i = threadIdx.x; i < K / 4; i += kUThreads) {
    const f32x4 v = from[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) most = fmaxf(most, fabsf(v[j]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kUThreads / 64; ++w) most = fmaxf(most, red[w]);
  // exponent of the largest, biased; a row with an infinity goes as it is (NaN and infinities stay such in fp16)
  const int e = (int)(__float_as_uint(most) >> 23);
  const int up = most < __builtin_inff() ? (141 - e < 126 ? 141 - e : 126) : 0;
  const float f = __uint_as_float((uint32_t)(127 + up) << 23);
  if (threadIdx.x == 0) back[row] = __uint_as_float((uint32_t)(127 - up) << 23);
  for (int i = threadIdx.x; i < K / 8; i += kUThreads) {
    f16x8 hi, lo;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 v = from[2 * i + h];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y = v[j] * f;
        hi[4 * h + j] = (_Float16)y;
        lo[4 * h + j] = (_Float16)(y - (float)hi[4 * h + j]);
      }
    }
    planes[row * (K / 8) + i] = lo;
    planes[(rows + row) * (K / 8) + i] = hi;
  }
}

// A step is 64 values of K: rows of 128 bytes, of which the 16-byte piece p of
// row r lies at p ^ (r / 2 % 8), so that 16 rows at one piece meet 16 different
// banks. Waves of 32 MI x 32 NI outputs, WM x WN of them; K advances through a
// ring of ST stages in LDS, filled by loads that go straight there and are
// counted here. A wave reads the next fragments while it multiplies: the barrier
// stands before the last instructions along a step, whose fragments are in
// registers by then. A group's accumulators are scaled and added to the sums
// right before the next group's first instructions write them anew.
constexpr int kStep = 64;
template <int PL>
__device__ __forceinline__ f32x16 multiply(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (PL == 1)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <typename T, int PL, int G, int WM, int WN, int MI, int NI, int ST>
__global__ __launch_bounds__(64 * WM * WN, WM * WN / 4) void k_gemm_int4(
    const uint16_t* __restrict__ a, int64_t plane, const float* __restrict__ back, const uint16_t* __restrict__ w,
    const float* __restrict__ scales, int64_t pitch, const float* __restrict__ bias, int64_t M, int N, int K,
    int64_t pitch_out, int splits, int64_t part, T* __restrict__ out) {
  constexpr int WAVES = WM * WN;
  constexpr int TM = 32 * MI * WM, TN = 32 * NI * WN;
  constexpr int GP = G < kStep ? kStep / G : 1;          // groups of a step
  constexpr int GS = G > kStep ? G / kStep : 1;          // steps of a group
  constexpr int GQ = 4 / GP;                             // instructions along a group within a step
  constexpr int SCALES = GP * TN * 4;                    // bytes of a stage
  constexpr int STAGE = (PL * TM + TN) * 128 + SCALES;
  constexpr int LA = PL * TM / 8 / WAVES, LB = TN / 8 / WAVES, LOADS = LA + LB + 1;
  constexpr int SLOTS = 4 * NI;                          // rows of matrix instructions in a step
  constexpr int FRAGS = NI + PL * MI;                    // to read for an instruction along K
  constexpr int PITCH = 32 * NI * (int)sizeof(T) + 16, OUT = 32 * PITCH;  // of a wave, 32 rows at a time
  static_assert(LA * 8 * WAVES == PL * TM && LB * 8 * WAVES == TN && TM % 8 == 0, "whole loads");
  static_assert(SCALES / 256 <= WAVES && WAVES % (SCALES / 256) == 0, "a load of scales a wave");
  static_assert(ST * STAGE <= 163840, "the LDS of a CU");
  __shared__ __attribute__((aligned(16))) uint8_t lds[ST * STAGE > WAVES * OUT ? ST * STAGE : WAVES * OUT];
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63;
  // Workgroups go round the 8 XCDs; each XCD takes a contiguous part of the tiles, columns first.
  const int ntn = (N + TN - 1) / TN;
  const int64_t ntiles = gridDim.x / splits;
  const int64_t per = ntiles / 8, extra = ntiles % 8;
  const int64_t b = blockIdx.x % ntiles;
  const int split = (int)(blockIdx.x / ntiles), xcd = (int)(b % 8);
  const int64_t tile = xcd * per + (xcd < extra ? xcd : extra) + b / 8;
  const int64_t m0 = tile / ntn * TM;
  const int n0 = (int)(tile % ntn) * TN;
  const int rows_a = M - m0 < TM ? (int)(M - m0) : TM, rows_b = N - n0 < TN ? N - n0 : TN;
  const int units = (K + GS * kStep - 1) / (GS * kStep);  // whole groups and whole steps
  const int steps = (K + kStep - 1) / kStep;
  const int st0 = (int)((int64_t)units * split / splits) * GS;
  int st1 = (int)((int64_t)units * (split + 1) / splits) * GS;
  if (st1 > steps) st1 = steps;
  // the planes of a split lie in one buffer, of 64 MiB at most
  const rsrc_words ra = descriptor(a + m0 * K, (uint32_t)(((PL - 1) * plane + (int64_t)rows_a * K) * 2));
  const rsrc_words rb = descriptor(w + (int64_t)n0 * K, (uint32_t)rows_b * K * 2);
  const int KG = K / G;
  const rsrc_words rs = descriptor(scales + n0, (uint32_t)(((int64_t)(KG - 1) * pitch + TN) * 4));
  uint32_t va[LA], vb[LB];
  {
    const int r = lane >> 3;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int row = ((wave * LA + i) * 8 + r) % TM, p = (wave * LA + i) * 8 / TM;
      va[i] = (uint32_t)(p * plane * 2) + (uint32_t)(row < rows_a ? row : rows_a - 1) * K * 2 +
              ((lane & 7) ^ (row >> 1 & 7)) * 16;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int row = (wave * LB + i) * 8 + r;
      vb[i] = (uint32_t)(row < rows_b ? row : rows_b - 1) * K * 2 + ((lane & 7) ^ (row >> 1 & 7)) * 16;
    }
  }
  const uint32_t base = lds_offset(lds);
  // Loads past the end are issued all the same (the waits count them).
  auto fetch = [&](int step, int stage, int i) {
    const bool there = step < st1;
    const uint32_t k = there ? (uint32_t)step * 128 : 0u, at = base + stage * STAGE;
    if (i < LA) {
      load_to_lds<16>(ra, buffer_at(there, true, va[i < LA ? i : 0], k), at + (wave * LA + i) * 1024);
    } else if (i < LA + LB) {
      load_to_lds<16>(rb, buffer_at(there, true, vb[i < LA || i >= LA + LB ? 0 : i - LA], k),
                      at + PL * TM * 128 + (wave * LB + i - LA) * 1024);
    } else {  // 64 scales: part c of the step's groups (several waves may fetch the same)
      const int c = wave % (SCALES / 256);
      int g = step * kStep / G + c / (TN / 64);
      if (g >= KG) g = KG - 1;
      const uint32_t vs = (uint32_t)(((int64_t)g * pitch + c % (TN / 64) * 64 + lane) * 4);
      load_to_lds<4>(rs, buffer_at(there, true, vs, 0), at + (PL * TM + TN) * 128 + c * 256);
    }
  };
  // slot k of the loads that fill one stage: the last NI rows of a step begin, the others end in the next step
  auto slot_of = [&](int step, int stage, int k) {
#pragma unroll
    for (int i = k * LOADS / SLOTS; i < (k + 1) * LOADS / SLOTS; ++i) fetch(step, stage, i);
  };
#pragma unroll
  for (int s = 0; s < ST; ++s)
#pragma unroll
    for (int k = 0; k < (s < ST - 1 ? SLOTS : NI); ++k) slot_of(st0 + s, s, k);
  wait_loads<(ST - 2) * LOADS + NI * LOADS / SLOTS>();
  lds_barrier();
  const int wm = wave / WN, wn = wave % WN;
  const int myrow = (lane & 31) * 128, mysw = lane >> 1 & 7;
  u32x4 fa[2][PL][MI], fb[2][NI];  // fragments of even and odd instructions along K
  auto read = [&](int stage, int q, int i) {
    const uint8_t* p = lds + stage * STAGE + myrow + ((2 * q + (lane >> 5)) ^ mysw) * 16;
    if (i < NI) {
      fb[q & 1][i < NI ? i : 0] = *reinterpret_cast<const u32x4*>(p + (PL * TM + (wn * NI + i) * 32) * 128);
    } else {
      const int j = i - NI < 0 ? 0 : i - NI, pl = j / MI, im = j % MI;
      fa[q & 1][pl][im] = *reinterpret_cast<const u32x4*>(p + (pl * TM + (wm * MI + im) * 32) * 128);
    }
  };
#pragma unroll
  for (int i = 0; i < FRAGS; ++i) read(0, 0, i);
  f32x16 sum[MI][NI] = {}, acc[MI][NI] = {};
  float now[GP][NI], scale[NI] = {};  // of the step's groups, of the group in the accumulators
  auto scales_of = [&](int stage) {
    const float* s = reinterpret_cast<const float*>(lds + stage * STAGE + (PL * TM + TN) * 128) + wn * 32 * NI + (lane & 31);
#pragma unroll
    for (int g = 0; g < GP; ++g)
#pragma unroll
      for (int j = 0; j < NI; ++j) now[g][j] = s[g * TN + j * 32];
  };
  auto products = [&](int q, int j, bool first) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (first) {
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[i][j][r] = __builtin_fmaf(scale[j], acc[i][j][r], sum[i][j][r]);
        acc[i][j] = multiply<PL>(fa[q & 1][0][i], fb[q & 1][j], (f32x16){});
      } else {
        acc[i][j] = multiply<PL>(fa[q & 1][0][i], fb[q & 1][j], acc[i][j]);
      }
#pragma unroll
      for (int p = 1; p < PL; ++p) acc[i][j] = multiply<PL>(fa[q & 1][p][i], fb[q & 1][j], acc[i][j]);
    }
    if (first) scale[j] = now[q / GQ][j];
  };
  const bool half = G == 32 && st1 * kStep > K;  // a last step of which there is half
  const int whole = half ? st1 - 1 : st1;
  int stage = 0;
#pragma unroll 1
  for (int step0 = st0; step0 < whole; step0 += GS) {
#pragma unroll
    for (int u = 0; u < GS; ++u) {  // the steps of a group (K is whole groups)
      const int step = step0 + u;
      const int next = stage == ST - 1 ? 0 : stage + 1, last = stage == 0 ? ST - 1 : stage - 1;
      if (u == 0) scales_of(stage);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q == 3) {
          wait_loads<(ST - 2) * LOADS>();  // the next stage has come
          lds_barrier();                   // for every wave, and this one is read
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (q == 3) slot_of(step + ST, stage, j);
          else slot_of(step + ST - 1, last, (q + 1) * NI + j);
#pragma unroll
          for (int z = j * FRAGS / NI; z < (j + 1) * FRAGS / NI; ++z) read(q == 3 ? next : stage, (q + 1) % 4, z);
          products(q, j, q % GQ == 0 && u == 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      stage = next;
    }
  }
  if (half) {
    scales_of(stage);
#pragma unroll
    for (int i = 0; i < FRAGS; ++i) read(stage, 1, i);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < NI; ++j) products(q, j, q == 0);
  }
  wait_loads<0>();
  lds_barrier();

  // outputs: lane holds column lane % 32 and rows 8 (r / 4) + 4 (lane / 32) + r % 4 of the 32 x 32 tile (i, j); they
  // leave through LDS, 32 rows of the wave at a time, as 16-byte pieces of rows
  T* to_part = out + split * part;
  uint8_t* mylds = lds + wave * OUT;
  const int nw = n0 + wn * 32 * NI;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t mw = m0 + (wm * MI + i) * 32;
    f32x4 rows[4];  // what undoes the scaling of the rows
    if constexpr (PL > 1) {
#pragma unroll
      for (int r = 0; r < 4; ++r) rows[r] = *reinterpret_cast<const f32x4*>(back + mw + 8 * r + 4 * (lane >> 5));
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int n = nw + j * 32 + (lane & 31);
      const float add = bias && n < N ? bias[n] : 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float y = __builtin_fmaf(scale[j], acc[i][j][r], sum[i][j][r]);
        if constexpr (PL > 1) y *= rows[r / 4][r % 4];
        store1(reinterpret_cast<T*>(mylds + (8 * (r / 4) + 4 * (lane >> 5) + r % 4) * PITCH) + j * 32 + (lane & 31), y + add);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave reads what its own lanes wrote
    constexpr int EP = 16 / (int)sizeof(T), OP = 32 * NI / EP;  // elements of a piece, pieces of a row
#pragma unroll
    for (int o = lane; o < 32 * OP; o += 64) {
      const int row = o / OP, pc = o % OP, n = nw + pc * EP;
      if (mw + row < M && n < N) {
        T* to = to_part + (mw + row) * pitch_out + n;
        const T* from = reinterpret_cast<const T*>(mylds + row * PITCH + pc * 16);
        if (n + EP <= N) {
          *reinterpret_cast<u32x4_a2*>(to) = *reinterpret_cast<const u32x4*>(from);
        } else {
          for (int e = 0; n + e < N; ++e) to[e] = from[e];
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// The parts of a split K, added in their order.
template <typename T>
__global__ __launch_bounds__(kUThreads) void k_join_int4(const float* __restrict__ parts, int splits, int64_t part,
                                                        int64_t M, int N, const float* __restrict__ bias,
                                                        int64_t pitch_out, T* __restrict__ out) {
  const int64_t u = (int64_t)blockIdx.x * kUThreads + threadIdx.x;
  if (u >= part) return;
  float y = 0.0f;
  for (int s = 0; s < splits; ++s) y += parts[s * part + u];
  const int64_t m = u / N;
  const int n = (int)(u - m * N);
  if (bias) y += bias[n];
  store1(out + m * pitch_out + n, y);
}

// How a call's work is laid out.
struct Plan {
  bool few;
  int64_t rows;     // few: rows of x a launch; many: rows of x split at a time
  int64_t slice;    // rows of weights unpacked at a time (of 128)
  int tile, splits; // tile: rows and columns of a workgroup's outputs, 0 64 x 64, 1 128 x 128, 2 256 x 128
  size_t w, s, x, back, parts;  // bytes of the workspace
};

constexpr int64_t kUnpacked = (int64_t)64 << 20;  // bytes of unpacked weights and of split activations at a time

Plan plan_of(int64_t M, int64_t N, int64_t K, int64_t group, int dtype) {
  Plan p = {};
  const int64_t fit = few_rows(K, dtype);
  p.few = M <= 3 * fit;
  if (p.few) {
    const int64_t launches = (M + fit - 1) / fit;
    p.rows = (M + launches - 1) / launches;
    return p;
  }
  const int64_t whole = (N + 127) / 128 * 128;
  p.slice = kUnpacked / (2 * K) / 128 * 128;
  if (whole < p.slice) p.slice = whole;
  // fewer than 2^24 workgroups of 256 work-items
  p.rows = ((int64_t)1 << 22) / (p.slice / 128) * 128;
  if (dtype == BSQ_F32 && kUnpacked / (4 * K) / 256 * 256 < p.rows) p.rows = kUnpacked / (4 * K) / 256 * 256;
  if (M < p.rows) p.rows = M;
  if (dtype == BSQ_F32) {
    p.x = (size_t)(p.rows * K * 4);
    p.back = (size_t)((p.rows + 767) / 768 * 768 * 4);  // whole tiles of 64, 128 and 192 rows
  }
  p.w = (size_t)(p.slice * K * 2);
  p.s = (size_t)(p.slice * (K / group) * 4);
  const int64_t cus = bsqh::device_cus();
  const int64_t small = ((p.rows + 127) / 128) * (p.slice / 128), big = ((p.rows + 255) / 256) * (p.slice / 128);
  p.splits = 1;
  if (small * 2 <= cus) {
    p.tile = 0;
    const int64_t tiles = ((p.rows + 63) / 64) * (p.slice / 64), most_splits = K / 256;
    int64_t sp = cus / tiles;
    if (sp > most_splits) sp = most_splits;
    if (sp > 8) sp = 8;
    p.splits = sp < 1 ? 1 : (int)sp;
  } else {
    p.tile = dtype == BSQ_F32 ? (small > cus && ((p.rows + 191) / 192) * (p.slice / 128) <= cus ? 2 : 1) : big < cus ? 1 : 2;
  }
  if (p.splits > 1) p.parts = (size_t)(p.splits * p.rows * p.slice * 4);
  return p;
}

template <typename T, int PL, int G>
void launch_tiles(const Plan& p, const uint16_t* a, int64_t plane, const float* back, const uint16_t* w, const float* sc,
                  const float* bias, int64_t M, int64_t N, int64_t K, int64_t pitch_out, int64_t part, T* out,
                  hipStream_t s) {
#define BSQ_TILE(WM, WN, MI, NI, ST)                                                                                   \
  hipLaunchKernelGGL((k_gemm_int4<T, PL, G, WM, WN, MI, NI, ST>),                                                     \
                     dim3((unsigned)(((M + 32 * MI * WM - 1) / (32 * MI * WM)) * ((N + 32 * NI * WN - 1) / (32 * NI * WN)) * \
                                     p.splits)),                                                                      \
                     dim3(64 * WM * WN), 0, s, a, plane, back, w, sc, p.slice, bias, M, (int)N, (int)K, pitch_out,    \
                     p.splits, part, out)
  if constexpr (PL == 1) {
    if (p.tile == 0) BSQ_TILE(2, 2, 1, 1, 3);
    else if (p.tile == 1) BSQ_TILE(2, 2, 2, 2, 2);
    else BSQ_TILE(4, 2, 2, 2, 3);
  } else {
    if (p.tile == 0) BSQ_TILE(2, 2, 1, 1, 3);
    else if (p.tile == 1) BSQ_TILE(2, 2, 2, 2, 3);
    else BSQ_TILE(2, 2, 3, 2, 2);
  }
#undef BSQ_TILE
}

template <typename X, typename T, int G>
int run_linear(const X* x, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const float* bias,
               int64_t M, int64_t N, int64_t K, T* out, uint8_t* ws, hipStream_t s) {
  constexpr int PL = sizeof(X) == 4 ? 2 : 1;
  const Plan p = plan_of(M, N, K, G, PL == 2 ? BSQ_F32 : BSQ_BF16);
  if (p.few) {
    for (int64_t m = 0; m < M; m += p.rows)
      launch_few<X, T, G>(x + m * K, codes, scales, zeros, bias, M - m < p.rows ? M - m : p.rows, N, K, out + m * N, s);
    return bsqh::launch_status();
  }
  typedef typename std::conditional<PL == 2, f16x8, bf16x8>::type V;
  V* w = reinterpret_cast<V*>(ws);
  float* turned = reinterpret_cast<float*>(ws + p.w);
  uint16_t* planes = reinterpret_cast<uint16_t*>(ws + p.w + p.s);
  float* back = reinterpret_cast<float*>(ws + p.w + p.s + p.x);
  float* parts = reinterpret_cast<float*>(ws + p.w + p.s + p.x + p.back);
  const int64_t KG = K / G;
  for (int64_t n0 = 0; n0 < N; n0 += p.slice) {
    const int64_t n = N - n0 < p.slice ? N - n0 : p.slice, units = n * K / 16;
    hipLaunchKernelGGL((k_unpack_int4<V>), dim3((unsigned)((units + kUThreads - 1) / kUThreads)), dim3(kUThreads), 0, s,
                       reinterpret_cast<const u32x2*>(codes + n0 * K / 2), scales + n0 * KG,
                       zeros ? zeros + n0 * KG : nullptr, units, G / 16, (int)KG, p.slice, w, turned);
    for (int64_t m0 = 0; m0 < M; m0 += p.rows) {
      const int64_t m = M - m0 < p.rows ? M - m0 : p.rows;
      const uint16_t* a = reinterpret_cast<const uint16_t*>(x + m0 * K);
      if constexpr (PL == 2) {
        if (n0 == 0 || M > p.rows)
          hipLaunchKernelGGL(k_split_f32, dim3((unsigned)m), dim3(kUThreads), 0, s,
                             reinterpret_cast<const f32x4*>(x + m0 * K), m, (int)K, reinterpret_cast<f16x8*>(planes), back);
        a = planes;
      }
      const uint16_t* wb = reinterpret_cast<const uint16_t*>(w);
      const float* add = bias ? bias + n0 : nullptr;
      T* to = out + m0 * N + n0;
      if (p.splits == 1) {
        launch_tiles<T, PL, G>(p, a, m * K, back, wb, turned, add, m, n, K, N, 0, to, s);
      } else {
        const int64_t part = m * n;
        launch_tiles<float, PL, G>(p, a, m * K, back, wb, turned, nullptr, m, n, K, n, part, parts, s);
        hipLaunchKernelGGL((k_join_int4<T>), dim3((unsigned)((part + kUThreads - 1) / kUThreads)), dim3(kUThreads), 0, s,
                           parts, p.splits, part, m, (int)n, add, N, to);
      }
    }
  }
  return bsqh::launch_status();
}

template <typename X, typename T>
int run_group(const void* x, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t group,
              const float* bias, int64_t M, int64_t N, int64_t K, void* out, void* ws, hipStream_t s) {
  const X* xx = static_cast<const X*>(x);
  T* o = static_cast<T*>(out);
  uint8_t* b = static_cast<uint8_t*>(ws);
  if (group == 32) return run_linear<X, T, 32>(xx, codes, scales, zeros, bias, M, N, K, o, b, s);
  if (group == 64) return run_linear<X, T, 64>(xx, codes, scales, zeros, bias, M, N, K, o, b, s);
  return run_linear<X, T, 128>(xx, codes, scales, zeros, bias, M, N, K, o, b, s);
}

bool is_group(int64_t g) { return g == 32 || g == 64 || g == 128; }
bool weights_ok(int64_t N, int64_t K, int64_t group) {
  return N >= 0 && N < (int64_t)1 << 31 && is_group(group) && K >= group && K <= 32768 && K % group == 0;
}
bool even(const void* p) { return ((uintptr_t)p & 1) == 0; }

}  // namespace

extern "C" int bsq_quantize_int4(const void* w, int dtype, int64_t N, int64_t K, int64_t group, int symmetric,
                                 uint8_t* codes, uint16_t* scales, uint8_t* zeros, bsq_stream_t stream) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(symmetric == 0 || symmetric == 1, BSQ_E_ENUM);
  BSQ_REQUIRE(weights_ok(N, K, group), BSQ_E_SHAPE);
  if (N == 0) return BSQ_OK;
  BSQ_REQUIRE(w && codes && scales && (zeros || symmetric), BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(w) && bsqh::aligned16(codes) && even(scales), BSQ_E_ALIGN);
  hipStream_t s = bsqh::as_stream(stream);
  if (symmetric) zeros = nullptr;
  constexpr int64_t most = bsqh::max_blocks(kQThreads) * kQThreads / 8 * 8;  // whole groups
  const int64_t units = N * K / 16;
  for (int64_t u = 0; u < units; u += most) {
    const int64_t n = units - u < most ? units - u : most;
    const dim3 grid((unsigned)((n + kQThreads - 1) / kQThreads));
    const int64_t g = u / (group / 16);
#define BSQ_Q(T, G)                                                                                               \
  hipLaunchKernelGGL((k_quant_int4<T, G>), grid, dim3(kQThreads), 0, s, static_cast<const T*>(w) + u * 16, n, symmetric, \
                     reinterpret_cast<u32x2*>(codes) + u, scales + g, zeros ? zeros + g : nullptr)
#define BSQ_QG(T)               \
  do {                          \
    if (group == 32) BSQ_Q(T, 32);      \
    else if (group == 64) BSQ_Q(T, 64); \
    else BSQ_Q(T, 128);         \
  } while (0)
    if (dtype == BSQ_F32) BSQ_QG(float);
    else BSQ_QG(uint16_t);
#undef BSQ_QG
#undef BSQ_Q
  }
  return bsqh::launch_status();
}

extern "C" int bsq_dequantize_int4(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                                   int64_t K, int64_t group, void* out, int out_dtype, bsq_stream_t stream) {
  BSQ_REQUIRE(out_dtype == BSQ_F32 || out_dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(weights_ok(N, K, group), BSQ_E_SHAPE);
  if (N == 0) return BSQ_OK;
  BSQ_REQUIRE(codes && scales && out, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(codes) && bsqh::aligned16(out) && even(scales), BSQ_E_ALIGN);
  hipStream_t s = bsqh::as_stream(stream);
  const int shift = group == 32 ? 5 : group == 64 ? 6 : 7;
  const int64_t values = N * K, E = out_dtype == BSQ_F32 ? 4 : 8, tile = kDPieces * kQThreads * E;  // of a workgroup
  const int64_t most = bsqh::max_blocks(kQThreads) * tile;  // whole groups
  for (int64_t v = 0; v < values; v += most) {
    const int64_t n = values - v < most ? values - v : most, g = v >> shift;
    const dim3 grid((unsigned)((n + tile - 1) / tile));
    if (out_dtype == BSQ_F32)
      hipLaunchKernelGGL((k_dequant_int4<float>), grid, dim3(kQThreads), 0, s, codes + v / 2, scales + g,
                         zeros ? zeros + g : nullptr, n / E, shift, static_cast<float*>(out) + v);
    else
      hipLaunchKernelGGL((k_dequant_int4<uint16_t>), grid, dim3(kQThreads), 0, s, codes + v / 2, scales + g,
                         zeros ? zeros + g : nullptr, n / E, shift, static_cast<uint16_t*>(out) + v);
  }
  return bsqh::launch_status();
}

extern "C" size_t bsq_linear_int4_workspace(int64_t M, int64_t N, int64_t K, int64_t group, int dtype) {
  if (M <= 0 || N <= 0 || M >= (int64_t)1 << 31 || !weights_ok(N, K, group)) return 0;
  const Plan p = plan_of(M, N, K, group, dtype);
  return p.w + p.s + p.x + p.back + p.parts;
}

extern "C" int bsq_linear_int4(const void* x, int dtype, const uint8_t* codes, const uint16_t* scales,
                               const uint8_t* zeros, int64_t group, const float* bias, int64_t M, int64_t N, int64_t K,
                               void* out, int out_dtype, void* ws, size_t ws_bytes, bsq_stream_t stream) {
  BSQ_REQUIRE((dtype == BSQ_F32 || dtype == BSQ_BF16) && (out_dtype == BSQ_F32 || out_dtype == BSQ_BF16), BSQ_E_DTYPE);
  BSQ_REQUIRE(M >= 0 && M < (int64_t)1 << 31 && weights_ok(N, K, group), BSQ_E_SHAPE);
  if (M == 0 || N == 0) return BSQ_OK;
  const size_t need = bsq_linear_int4_workspace(M, N, K, group, dtype);
  BSQ_REQUIRE(x && codes && scales && out && (ws || need == 0), BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(x) && bsqh::aligned16(codes) && bsqh::aligned16(ws) && even(scales) &&
                  ((uintptr_t)bias & 3) == 0 && ((uintptr_t)out & (out_dtype == BSQ_F32 ? 3 : 1)) == 0,
              BSQ_E_ALIGN);
  BSQ_REQUIRE(ws_bytes >= need, BSQ_E_WORKSPACE);
  hipStream_t s = bsqh::as_stream(stream);
  if (dtype == BSQ_BF16 && out_dtype == BSQ_BF16)
    return run_group<uint16_t, uint16_t>(x, codes, scales, zeros, group, bias, M, N, K, out, ws, s);
  if (dtype == BSQ_BF16) return run_group<uint16_t, float>(x, codes, scales, zeros, group, bias, M, N, K, out, ws, s);
  if (out_dtype == BSQ_BF16) return run_group<float, uint16_t>(x, codes, scales, zeros, group, bias, M, N, K, out, ws, s);
  return run_group<float, float>(x, codes, scales, zeros, group, bias, M, N, K, out, ws, s);
}
