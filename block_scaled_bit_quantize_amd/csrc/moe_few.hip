// A whole NVFP4 expert layer for a few tokens (decode), without dispatch.
//
//   y_t = sum_j w_tj W2_e (silu(G) * U),  (G; U) = W13_e x_t,  e = ids[t, j]
//
// The many-token chain gathers rows into 256-row tiles per expert; for a few
// tokens an expert sees one to some tens of rows, and what bounds the layer is
// reading the chosen experts' weights (0.5625 bytes a value) once. Here one
// workgroup owns 32 weight rows of one expert (for W13: 16 gate rows and their
// 16 up rows) for every token that chose it, its eight waves share the inner
// dimension, so no weight or activation is read twice by a workgroup, and the
// partial sums meet in LDS.
//
// Weights are decoded to bf16 exactly (an E2M1 value times its E4M3 scale has
// at most 6 significant bits); the activations are split into bf16 terms that
// add up to them (bf16 inputs: themselves; the float32 SwiGLU result: two,
// 2^-16 of a value; float32 inputs: three, exact), so that
// v_mfma_f32_16x16x32_bf16 multiplies them with float32 sums. The two outer
// scales and the token's weight are applied to the float32 sums.
//
// Which expert a workgroup owns comes from the ids themselves: slot s is the
// s-th smallest expert id that occurs, and grid rows past the last one exit.
// Three launches: W13 with SwiGLU, W2 into one row per (token, slot) pair, and
// the sum over a token's pairs in slot order (no atomics: the same bits every
// time).
#include "bsq_device.h"
#include "bsq_internal.h"

using namespace bsqd;

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxPairs = BSQ_MOE_FEW_MAX_PAIRS;
constexpr int kMT = 4;  // 16-pair tiles that share one decode of the weights

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Two words (16 E2M1 codes) times one E4M3 scale -> 16 bf16 in 8 words.
__device__ __forceinline__ void decode16(uint32_t w0, uint32_t w1, float s, uint32_t* out) {
  const uint32_t w[2] = {w0, w1};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f32x2 v;
    v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0);
    out[4 * i + 0] = pack_bf16(v[0] * s, v[1] * s);
    v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1);
    out[4 * i + 1] = pack_bf16(v[0] * s, v[1] * s);
    v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2);
    out[4 * i + 2] = pack_bf16(v[0] * s, v[1] * s);
    v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3);
    out[4 * i + 3] = pack_bf16(v[0] * s, v[1] * s);
  }
}

// 16 activations -> NT terms of 8 words each. bf16 rows hold them as they are.
template <int NT>
__device__ __forceinline__ void load_terms(const uint16_t* p, uint32_t (&o)[NT][8]) {
  static_assert(NT == 1, "bf16 rows are one term");
  const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *reinterpret_cast<const u32x4*>(p + 8);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[0][i] = a[i], o[0][4 + i] = b[i];
}
// float32 rows: the upper halves of the values' bits are exact bf16 terms whose
// remainders are exact too; the last term is rounded.
template <int NT>
__device__ __forceinline__ void load_terms(const float* p, uint32_t (&o)[NT][8]) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = a[j];
  }
#pragma unroll
  for (int t = 0; t < NT - 1; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = __float_as_uint(v[2 * i]) & 0xFFFF0000u, b = __float_as_uint(v[2 * i + 1]) & 0xFFFF0000u;
      o[t][i] = (a >> 16) | b;
      v[2 * i] -= __uint_as_float(a);
      v[2 * i + 1] -= __uint_as_float(b);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) o[NT - 1][i] = pack_bf16(v[2 * i], v[2 * i + 1]);
}

// The slot's expert and the pairs that chose it (ascending), or -1 when fewer
// experts occur. Every thread calls it; list and bits are LDS.
__device__ __forceinline__ int find_slot(const int32_t* __restrict__ ids, int pairs, int E, int slot, uint32_t* bits,
                                         uint16_t* list, int* count) {
  const int t = threadIdx.x, lane = t & 63;
  if (t < 32) bits[t] = 0;
  __syncthreads();
  for (int p = t; p < pairs; p += kThreads) {
    const int e = ids[p];
    if (e >= 0 && e < E) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  uint32_t word = lane < 32 ? bits[lane] : 0u;
  const int mine = __popc(word);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up(upto, o, 64);
    if (lane >= o) upto += v;
  }
  const uint64_t hit = __ballot(lane < 32 && upto - mine <= slot && slot < upto);
  if (!hit) return -1;
  const int src = __ffsll((unsigned long long)hit) - 1;
  word = (uint32_t)__shfl((int)word, src, 64);
  int skip = slot - __shfl(upto - mine, src, 64);
  for (; skip > 0; --skip) word &= word - 1;
  const int expert = src * 32 + __ffs((int)word) - 1;
  if (t < 64) {
    int n = 0;
    for (int p0 = 0; p0 < pairs; p0 += 64) {
      const bool is = p0 + lane < pairs && ids[p0 + lane] == expert;
      const uint64_t b = __ballot(is);
      if (is) list[n + __popcll(b & ((1ull << lane) - 1))] = (uint16_t)(p0 + lane);
      n += __popcll(b);
    }
    if (lane == 0) *count = n;
  }
  __syncthreads();
  return expert;
}

// One 32-row slice of one expert's product. GLU (W13): rows [f0, f0 + 16) of
// the gate half and of the up half; out[pair, f] = silu(gate) * up. Otherwise
// (W2): rows [n0, n0 + 32); out[pair, n] = weight[pair] * product.
// Row of activations of pair p: in + (GLU ? p / k : p) * K.
template <typename T, int NT, bool GLU>
__global__ __launch_bounds__(kThreads) void k_moe_part(const T* __restrict__ in, const int32_t* __restrict__ ids,
                                                      const float* __restrict__ pair_weight, int pairs, int k, int E,
                                                      int K, int rows, const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales,
                                                      const float* __restrict__ outer, float* __restrict__ out) {
  __shared__ uint32_t bits[32];
  __shared__ uint16_t list[kMaxPairs];
  __shared__ int count;
  __shared__ f32x4 part[kWaves][2][kMT][64];
  const int expert = find_slot(ids, pairs, E, (int)blockIdx.y, bits, list, &count);
  if (expert < 0) return;
  const int np = count;
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int col = lane & 15, grp = lane >> 4;
  // weight rows of this lane in the two 16-row tiles (clamped rows are computed and not stored)
  const int f0 = (int)blockIdx.x * (GLU ? 16 : 32);
  const int width = GLU ? rows / 2 : rows;  // outputs per pair
  int r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = f0 + (GLU ? 0 : 16 * i) + col;
    r[i] = (f < width ? f : width - 1) + (GLU ? i * width : 0);
  }
  const uint8_t* crow[2];
  const uint8_t* srow[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    crow[i] = codes + ((int64_t)expert * rows + r[i]) * (K / 2);
    srow[i] = scales + ((int64_t)expert * rows + r[i]) * (K / 16);
  }
  const float so = outer[expert];
  const int nblk = K / 16;                    // blocks of 16 along K
  const int steps = (nblk + 7) / 8;           // 128 values: two blocks per 16-lane group
  for (int mt0 = 0; mt0 < np; mt0 += 16 * kMT) {
    const int tiles = (np - mt0 + 15) / 16 < kMT ? (np - mt0 + 15) / 16 : kMT;
    const T* arow[kMT];
    bool have[kMT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      const int q = mt0 + 16 * m + col;
      have[m] = q < np;
      const int p = list[have[m] ? q : mt0];
      arow[m] = in + (int64_t)(GLU ? p / k : p) * K;
    }
    f32x4 acc[2][kMT] = {};
    for (int st = wave; st < steps; st += kWaves) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int blk = st * 8 + grp * 2 + b;
        const bool in_k = blk < nblk;
        uint32_t wd[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u32x2 c = {0u, 0u};
          uint32_t s8 = 0;
          if (in_k) {
            c = *reinterpret_cast<const u32x2_a4*>(crow[i] + blk * 8);
            s8 = srow[i][blk];
          }
          decode16(c[0], c[1], e4m3_val(s8), wd[i]);
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          if (m >= tiles) break;
          uint32_t a[NT][8] = {};
          if (in_k && have[m]) load_terms<NT>(arow[m] + blk * 16, a);
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bf16x8 bv = __builtin_bit_cast(
                  bf16x8, (u32x4){a[q][4 * h], a[q][4 * h + 1], a[q][4 * h + 2], a[q][4 * h + 3]});
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const bf16x8 av = __builtin_bit_cast(
                    bf16x8, (u32x4){wd[i][4 * h], wd[i][4 * h + 1], wd[i][4 * h + 2], wd[i][4 * h + 3]});
                acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv, acc[i][m], 0, 0, 0);
              }
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int m = 0; m < kMT; ++m)
        if (m < tiles) part[wave][i][m][lane] = acc[i][m];
    __syncthreads();
    // 64 threads per 16-pair tile; a lane holds 4 consecutive rows of one pair
    for (int j = t; j < tiles * 64; j += kThreads) {
      const int m = j >> 6, l = j & 63;
      const int q = mt0 + 16 * m + (l & 15);
      f32x4 s0 = part[0][0][m][l], s1 = part[0][1][m][l];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        s0 += part[w][0][m][l];
        s1 += part[w][1][m][l];
      }
      if (q >= np) continue;
      const int p = list[q];
      const int fr = f0 + 4 * (l >> 4);
      float* o = out + (int64_t)p * width;
      if constexpr (GLU) {
        f32x4 v;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float g = s0[z] * so, u = s1[z] * so;
          v[z] = g / (1.0f + expf(-g)) * u;
        }
        if (fr < width) *reinterpret_cast<f32x4*>(o + fr) = v;  // width % 16 == 0: whole or not at all
      } else {
        const float ws = pair_weight[p] * so;
        if (fr < width) *reinterpret_cast<f32x4*>(o + fr) = s0 * ws;
        if (fr + 16 < width) *reinterpret_cast<f32x4*>(o + fr + 16) = s1 * ws;
      }
    }
    __syncthreads();
  }
}

// y[t, n..n+3] = sum over the token's valid pairs, in slot order.
template <typename T>
__global__ __launch_bounds__(256) void k_moe_sum(const float* __restrict__ z, const int32_t* __restrict__ ids,
                                                 int tokens, int k, int E, int H, T* __restrict__ y) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = H / 4;
  if (id >= (int64_t)tokens * per) return;
  const int t = (int)(id / per), n = (int)(id % per) * 4;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < k; ++j) {
    const int e = ids[t * k + j];
    if (e >= 0 && e < E) s += *reinterpret_cast<const f32x4*>(z + ((int64_t)t * k + j) * H + n);
  }
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<f32x4*>(y + (int64_t)t * H + n) = s;
  } else {
    *reinterpret_cast<u32x2*>(y + (int64_t)t * H + n) = (u32x2){pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
  }
}

template <typename T, int NT, int NH>
void launch_layer(const T* x, int64_t tokens, int64_t H, int64_t F, int64_t E, int64_t k, const int32_t* ids,
                  const float* weights, const uint8_t* w13c, const uint8_t* w13s, const float* w13o,
                  const uint8_t* w2c, const uint8_t* w2s, const float* w2o, T* out, float* h, float* z,
                  hipStream_t s) {
  const int pairs = (int)(tokens * k);
  const unsigned slots = (unsigned)(pairs < E ? pairs : E);
  hipLaunchKernelGGL((k_moe_part<T, NT, true>), dim3((unsigned)((F + 15) / 16), slots), dim3(kThreads), 0, s, x, ids,
                     weights, pairs, (int)k, (int)E, (int)H, (int)(2 * F), w13c, w13s, w13o, h);
  hipLaunchKernelGGL((k_moe_part<float, NH, false>), dim3((unsigned)((H + 31) / 32), slots), dim3(kThreads), 0, s,
                     static_cast<const float*>(h), ids, weights, pairs, (int)k, (int)E, (int)F, (int)H, w2c, w2s, w2o,
                     z);
  hipLaunchKernelGGL((k_moe_sum<T>), dim3((unsigned)((tokens * (H / 4) + 255) / 256)), dim3(256), 0, s,
                     static_cast<const float*>(z), ids, (int)tokens, (int)k, (int)E, (int)H, out);
}

bool shape_ok(int64_t tokens, int64_t hidden, int64_t ffn, int64_t E, int64_t k) {
  return tokens >= 0 && hidden >= 16 && hidden % 16 == 0 && hidden <= 32768 && ffn >= 16 && ffn % 16 == 0 &&
         ffn <= 32768 && E >= 1 && E <= 1024 && k >= 1 && k <= 64 && tokens <= kMaxPairs / k;
}

}  // namespace

extern "C" size_t bsq_moe_few_nvfp4_workspace(int64_t tokens, int64_t hidden, int64_t ffn, int64_t E, int64_t k) {
  if (!shape_ok(tokens, hidden, ffn, E, k)) return 0;
  return (size_t)(tokens * k) * (size_t)(hidden + ffn) * 4;
}

extern "C" int bsq_moe_few_nvfp4(const void* x, int dtype, int64_t tokens, int64_t hidden, int64_t ffn, int64_t E,
                                 int64_t k, const int32_t* topk_ids, const float* topk_weights,
                                 const uint8_t* w13_codes, const uint8_t* w13_scales, const float* w13_outer,
                                 const uint8_t* w2_codes, const uint8_t* w2_scales, const float* w2_outer, void* out,
                                 void* ws, size_t ws_bytes, bsq_stream_t stream) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(shape_ok(tokens, hidden, ffn, E, k), BSQ_E_SHAPE);
  if (tokens == 0) return BSQ_OK;
  BSQ_REQUIRE(x && topk_ids && topk_weights && w13_codes && w13_scales && w13_outer && w2_codes && w2_scales &&
                  w2_outer && out && ws,
              BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(x) && bsqh::aligned16(w13_codes) && bsqh::aligned16(w2_codes) && bsqh::aligned16(out) &&
                  bsqh::aligned16(ws) && bsqh::aligned16(w13_scales) && bsqh::aligned16(w2_scales),
              BSQ_E_ALIGN);
  BSQ_REQUIRE((((uintptr_t)topk_ids | (uintptr_t)topk_weights | (uintptr_t)w13_outer | (uintptr_t)w2_outer) & 3) == 0,
              BSQ_E_ALIGN);
  BSQ_REQUIRE(ws_bytes >= bsq_moe_few_nvfp4_workspace(tokens, hidden, ffn, E, k), BSQ_E_WORKSPACE);
  hipStream_t s = bsqh::as_stream(stream);
  float* h = static_cast<float*>(ws);            // [pairs, ffn]
  float* z = h + tokens * k * ffn;               // [pairs, hidden]
  if (dtype == BSQ_BF16)
    launch_layer<uint16_t, 1, 2>(static_cast<const uint16_t*>(x), tokens, hidden, ffn, E, k, topk_ids, topk_weights,
                                 w13_codes, w13_scales, w13_outer, w2_codes, w2_scales, w2_outer,
                                 static_cast<uint16_t*>(out), h, z, s);
  else
    launch_layer<float, 3, 3>(static_cast<const float*>(x), tokens, hidden, ffn, E, k, topk_ids, topk_weights,
                              w13_codes, w13_scales, w13_outer, w2_codes, w2_scales, w2_outer,
                              static_cast<float*>(out), h, z, s);
  return bsqh::launch_status();
}
