// Dense products in 8-bit integers: a scale for each row of activations (a
// token) and each row of weights (an output channel).
//
//   x_q = rint(x / s),  s = max|x| / 127 per row (in float32: max|x| * f32(1/127), x * f32(1/s))
//   y[m, n] = (sum_k a_q[m, k] b_q[n, k]) s_a[m] s_b[n] + bias[n]
//
// The integer sums are exact (int32: K is limited so that they cannot
// overflow); the only roundings are those of the float32 epilogue and of the
// output type.
#include "bsq_device.h"
#include "bsq_internal.h"

using namespace bsqd;

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

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

// Four values -> four int8 codes in a word: rint(v * inv), clamped.
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = fminf(fmaxf(rintf(v[i] * inv), -127.0f), 127.0f);
    w |= ((uint32_t)(int)q & 0xFFu) << (8 * i);
  }
  return w;
}

// The row's scale: max * f32(1/127), or 1 where that would be below the normal range
// (its reciprocal could overflow); all codes of such a row are 0.
__device__ __forceinline__ float row_scale(float amax) {
  const float s = amax * (1.0f / 127.0f);
  return s >= kFltMinNormal ? s : 1.0f;
}

// TPR threads share a row and keep it in registers, up to MAXB blocks of 16
// values each: one read of x. GLU: a row of x holds 2C values, gate then up,
// and what is quantized is silu(gate) * up.
template <typename T, int TPR, int MAXB, bool GLU>
__global__ __launch_bounds__(kQThreads) void k_quant_int8(const T* __restrict__ x, int64_t rows, int64_t C,
                                                         uint32_t* __restrict__ codes, float* __restrict__ scales) {
  const int tl = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (kQThreads / TPR) + threadIdx.x / TPR;
  const bool ok = row < rows;
  const int nb = (int)(C >> 4);
  float v[MAXB][16];
  float amax = 0.0f;
#pragma unroll
  for (int b = 0; b < MAXB; ++b) {
    const int j = tl + b * TPR;
    if (ok && j < nb) {
      if constexpr (GLU) {
        float u[16];
        load16(x + row * 2 * C + j * 16, v[b]);
        load16(x + row * 2 * C + C + j * 16, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[b][i] = v[b][i] / (1.0f + expf(-v[b][i])) * u[i];
      } else {
        load16(x + row * C + j * 16, v[b]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[b][i]));
    }
  }
  if constexpr (TPR <= 64) {
    amax = group_max<TPR>(amax);
  } else {
    __shared__ float red[kQThreads / 64];
    const float wm = wave_max(amax);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = wm;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int w = 1; w < kQThreads / 64; ++w) amax = fmaxf(amax, red[w]);
  }
  const float s = row_scale(amax);
  const float inv = 1.0f / s;
  if (!ok) return;
  if (tl == 0) scales[row] = s;
#pragma unroll
  for (int b = 0; b < MAXB; ++b) {
    const int j = tl + b * TPR;
    if (j < nb)
      *reinterpret_cast<u32x4*>(codes + (row * C + j * 16) / 4) = (u32x4){
          codes4(&v[b][0], inv), codes4(&v[b][4], inv), codes4(&v[b][8], inv), codes4(&v[b][12], inv)};
  }
}

template <typename T, int TPR, bool GLU>
void launch_quant_tpr(const T* x, int64_t rows, int64_t C, uint32_t* codes, float* scales, hipStream_t s) {
  const int64_t per = (C / 16 + TPR - 1) / TPR;
  const dim3 grid((unsigned)((rows + kQThreads / TPR - 1) / (kQThreads / TPR)));
#define BSQ_Q(MB)                                                                                                \
  hipLaunchKernelGGL((k_quant_int8<T, TPR, MB, GLU>), grid, dim3(kQThreads), 0, s, x, rows, C, codes, scales)
  if (per <= 1) BSQ_Q(1);
  else if (per <= 2) BSQ_Q(2);
  else if (per <= 4) BSQ_Q(4);
  else BSQ_Q(8);
#undef BSQ_Q
}

// A wave per row while the rows fill the chip and fit its registers, else a
// workgroup per row.
template <typename T, bool GLU>
void launch_quant(const T* x, int64_t rows, int64_t C, void* codes, float* scales, hipStream_t s) {
  uint32_t* c = static_cast<uint32_t*>(codes);
  if (rows >= 2048 && C <= 64 * 16 * 8) launch_quant_tpr<T, 64, GLU>(x, rows, C, c, scales, s);
  else launch_quant_tpr<T, 256, GLU>(x, rows, C, c, scales, s);
}

int check_quant(const void* x, int dtype, int64_t rows, int64_t cols, const void* codes, const float* scales) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(rows >= 0 && rows < (int64_t)1 << 31 && cols >= 16 && cols % 16 == 0 && cols <= 32768, BSQ_E_SHAPE);
  if (rows == 0) return BSQ_OK;
  BSQ_REQUIRE(x && codes && scales, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(x) && bsqh::aligned16(codes) && ((uintptr_t)scales & 3) == 0, BSQ_E_ALIGN);
  return BSQ_OK;
}

// ---------------------------------------------------------------- epilogue
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// ---------------------------------------------------------------- few rows
// Up to 64 rows of activations: bound by reading the weights once. A workgroup
// owns 16 weight rows for all M, its eight waves share K, and the exact
// integer partial sums meet in LDS.
constexpr int kFThreads = 512;
constexpr int kFWaves = kFThreads / 64;

template <typename T, int MT>
__global__ __launch_bounds__(kFThreads) void k_gemm_int8_few(const int8_t* __restrict__ a, const float* __restrict__ sa,
                                                            const int8_t* __restrict__ b, const float* __restrict__ sb,
                                                            const float* __restrict__ bias, int M, int N, int K,
                                                            T* __restrict__ out) {
  __shared__ i32x4 part[kFWaves][MT][64];
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int col = lane & 15, grp = lane >> 4;
  const int n0 = (int)blockIdx.x * 16;
  const int8_t* brow = b + (int64_t)(n0 + col < N ? n0 + col : N - 1) * K;
  const int8_t* arow[MT];
  bool have[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    have[m] = 16 * m + col < M;
    arow[m] = a + (int64_t)(have[m] ? 16 * m + col : 0) * K;
  }
  i32x4 acc[MT] = {};
  for (int k0 = wave * 64; k0 < K; k0 += kFWaves * 64) {
    const int k = k0 + grp * 16;
    const bool in = k < K;  // K % 16 == 0: a lane's 16 values are whole or past the end
    i32x4 w = {0, 0, 0, 0};
    if (in) w = *reinterpret_cast<const i32x4*>(brow + k);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      i32x4 v = {0, 0, 0, 0};
      if (in && have[m]) v = *reinterpret_cast<const i32x4*>(arow[m] + k);
      acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, v, acc[m], 0, 0, 0);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) part[wave][m][lane] = acc[m];
  __syncthreads();
  for (int j = t; j < MT * 64; j += kFThreads) {
    const int m = j >> 6, l = j & 63;
    i32x4 s = part[0][m][l];
#pragma unroll
    for (int w = 1; w < kFWaves; ++w) s += part[w][m][l];
    const int row = 16 * m + (l & 15);
    if (row >= M) continue;
    const float fa = sa[row];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 4 * (l >> 4) + i;
      if (n < N) {
        float y = (float)s[i] * fa * sb[n];
        if (bias) y += bias[n];
        store1(out + (int64_t)row * N + n, y);
      }
    }
  }
}

// ---------------------------------------------------------------- many rows
// 128 x 128 outputs per workgroup of four waves (64 x 64 each), K in steps of
// 128 staged in LDS. 16-byte pieces of a row are placed at (piece ^ row % 8),
// so that fragment reads (32 rows at one piece) meet no bank twice.
constexpr int kTile = 128;
constexpr int kStep = 128;

template <typename T>
__global__ __launch_bounds__(256) void k_gemm_int8(const int8_t* __restrict__ a, const float* __restrict__ sa,
                                                  const int8_t* __restrict__ b, const float* __restrict__ sb,
                                                  const float* __restrict__ bias, int64_t M, int N, int K,
                                                  T* __restrict__ out) {
  __shared__ i32x4 la[kTile * 8], lb[kTile * 8];
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int ntn = (N + kTile - 1) / kTile;
  const int64_t m0 = (int64_t)(blockIdx.x / ntn) * kTile;
  const int n0 = (int)(blockIdx.x % ntn) * kTile;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int piece = t & 7, r0 = t >> 3;  // this thread's piece of rows r0, r0 + 32, ...
  const int8_t* ap[4];
  const int8_t* bp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + r0 + 32 * i;
    const int n = n0 + r0 + 32 * i;
    ap[i] = a + (m < M ? m : M - 1) * K + piece * 16;
    bp[i] = b + (int64_t)(n < N ? n : N - 1) * K + piece * 16;
  }
  i32x16 acc[2][2] = {};
  i32x4 ra[4], rb[4];
  auto fetch = [&](int k) {
    const bool in = k + piece * 16 < K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ra[i] = rb[i] = (i32x4){0, 0, 0, 0};
      if (in) {
        ra[i] = *reinterpret_cast<const i32x4*>(ap[i] + k);
        rb[i] = *reinterpret_cast<const i32x4*>(bp[i] + k);
      }
    }
  };
  fetch(0);
  for (int k = 0; k < K; k += kStep) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 32 * i;
      la[r * 8 + (piece ^ (r & 7))] = ra[i];
      lb[r * 8 + (piece ^ (r & 7))] = rb[i];
    }
    __syncthreads();
    if (k + kStep < K) fetch(k + kStep);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      i32x4 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ar = wm + 32 * i + (lane & 31), br = wn + 32 * i + (lane & 31);
        const int pc = 2 * q + (lane >> 5);
        fa[i] = la[ar * 8 + (pc ^ (ar & 7))];
        fb[i] = lb[br * 8 + (pc ^ (br & 7))];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = n0 + wn + 32 * j + (lane & 31);
    if (n >= N) continue;
    const float fb = sb[n], add = bias ? bias[n] : 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int64_t m = m0 + wm + 32 * i + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3);
        if (m < M) store1(out + m * N + n, (float)acc[i][j][q] * sa[m] * fb + add);
      }
  }
}

template <typename T>
void launch_gemm(const int8_t* a, const float* sa, const int8_t* b, const float* sb, const float* bias, int64_t M,
                 int64_t N, int64_t K, T* out, hipStream_t s) {
  if (M <= 64) {
    const dim3 grid((unsigned)((N + 15) / 16));
#define BSQ_F(MT)                                                                                                     \
  hipLaunchKernelGGL((k_gemm_int8_few<T, MT>), grid, dim3(kFThreads), 0, s, a, sa, b, sb, bias, (int)M, (int)N, (int)K, \
                     out)
    if (M <= 16) BSQ_F(1);
    else if (M <= 32) BSQ_F(2);
    else BSQ_F(4);
#undef BSQ_F
    return;
  }
  const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  hipLaunchKernelGGL((k_gemm_int8<T>), dim3((unsigned)tiles), dim3(256), 0, s, a, sa, b, sb, bias, M, (int)N, (int)K,
                     out);
}

int check_gemm(int64_t M, int64_t N, int64_t K, int out_dtype) {
  BSQ_REQUIRE(out_dtype == BSQ_F32 || out_dtype == BSQ_BF16, BSQ_E_DTYPE);
  // 128 * 128 * K stays below 2^31; fewer than 2^31 tiles
  BSQ_REQUIRE(M >= 0 && M < (int64_t)1 << 31 && N >= 0 && N < (int64_t)1 << 31 && K >= 16 && K % 16 == 0 && K < 131072,
              BSQ_E_SHAPE);
  BSQ_REQUIRE(((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile) < (int64_t)1 << 31, BSQ_E_SHAPE);
  return BSQ_OK;
}

bool out_aligned(const void* out, int out_dtype) { return ((uintptr_t)out & (out_dtype == BSQ_F32 ? 3 : 1)) == 0; }

int run_gemm(const int8_t* a, const float* sa, const int8_t* b, const float* sb, const float* bias, int64_t M,
             int64_t N, int64_t K, void* out, int out_dtype, bsq_stream_t stream) {
  hipStream_t s = bsqh::as_stream(stream);
  if (out_dtype == BSQ_BF16) launch_gemm(a, sa, b, sb, bias, M, N, K, static_cast<uint16_t*>(out), s);
  else launch_gemm(a, sa, b, sb, bias, M, N, K, static_cast<float*>(out), s);
  return bsqh::launch_status();
}

}  // namespace

extern "C" int bsq_quantize_int8(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                                 bsq_stream_t stream) {
  const int st = check_quant(x, dtype, rows, cols, codes, scales);
  if (st != BSQ_OK || rows == 0) return st;
  hipStream_t s = bsqh::as_stream(stream);
  if (dtype == BSQ_BF16) launch_quant<uint16_t, false>(static_cast<const uint16_t*>(x), rows, cols, codes, scales, s);
  else launch_quant<float, false>(static_cast<const float*>(x), rows, cols, codes, scales, s);
  return bsqh::launch_status();
}

extern "C" int bsq_swiglu_quantize_int8(const void* h13, int dtype, int64_t rows, int64_t ffn, int8_t* codes,
                                        float* scales, bsq_stream_t stream) {
  const int st = check_quant(h13, dtype, rows, ffn, codes, scales);
  if (st != BSQ_OK || rows == 0) return st;
  hipStream_t s = bsqh::as_stream(stream);
  if (dtype == BSQ_BF16) launch_quant<uint16_t, true>(static_cast<const uint16_t*>(h13), rows, ffn, codes, scales, s);
  else launch_quant<float, true>(static_cast<const float*>(h13), rows, ffn, codes, scales, s);
  return bsqh::launch_status();
}

extern "C" int bsq_gemm_int8(const int8_t* a_codes, const float* a_scales, const int8_t* b_codes,
                             const float* b_scales, const float* bias, int64_t M, int64_t N, int64_t K, void* out,
                             int out_dtype, bsq_stream_t stream) {
  const int st = check_gemm(M, N, K, out_dtype);
  if (st != BSQ_OK || M == 0 || N == 0) return st;
  BSQ_REQUIRE(a_codes && a_scales && b_codes && b_scales && out, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(a_codes) && bsqh::aligned16(b_codes) && out_aligned(out, out_dtype) &&
                  (((uintptr_t)a_scales | (uintptr_t)b_scales | (uintptr_t)bias) & 3) == 0,
              BSQ_E_ALIGN);
  return run_gemm(a_codes, a_scales, b_codes, b_scales, bias, M, N, K, out, out_dtype, stream);
}

extern "C" size_t bsq_linear_int8_workspace(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0) return 0;
  return (size_t)M * (size_t)K + ((size_t)M * 4 + 15) / 16 * 16;
}

extern "C" int bsq_linear_int8(const void* x, int dtype, const int8_t* b_codes, const float* b_scales,
                               const float* bias, int64_t M, int64_t N, int64_t K, void* out, int out_dtype, void* ws,
                               size_t ws_bytes, bsq_stream_t stream) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  int st = check_gemm(M, N, K, out_dtype);
  if (st != BSQ_OK) return st;
  BSQ_REQUIRE(K <= 32768, BSQ_E_SHAPE);
  if (M == 0 || N == 0) return BSQ_OK;
  BSQ_REQUIRE(x && b_codes && b_scales && out && ws, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(x) && bsqh::aligned16(b_codes) && bsqh::aligned16(ws) && out_aligned(out, out_dtype) &&
                  (((uintptr_t)b_scales | (uintptr_t)bias) & 3) == 0,
              BSQ_E_ALIGN);
  BSQ_REQUIRE(ws_bytes >= bsq_linear_int8_workspace(M, K), BSQ_E_WORKSPACE);
  int8_t* codes = static_cast<int8_t*>(ws);
  float* scales = reinterpret_cast<float*>(codes + M * K);  // K % 16 == 0: aligned
  st = bsq_quantize_int8(x, dtype, M, K, codes, scales, stream);
  if (st != BSQ_OK) return st;
  return run_gemm(codes, scales, b_codes, b_scales, bias, M, N, K, out, out_dtype, stream);
}
