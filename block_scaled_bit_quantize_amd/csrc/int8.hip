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
#include "bsq_lds.h"

using namespace bsqd;

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
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

// silu(g) * u by the hardware's exponential and reciprocal: within a few units
// in the last place, |g| 2^-24 more from the exponent's rounding (expf and an
// exact division made the kernel bound by the vector ALU).
__device__ __forceinline__ float swiglu(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896340736f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
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

// The larger magnitude of m >= 0 and x, NaN if one is (fmaxf would drop it; both
// are one instruction).
__device__ __forceinline__ float max_abs(float m, float x) { return __builtin_elementwise_maximum(m, fabsf(x)); }

// The row's scale: max * f32(1/127), or 1 where that would be below the normal range
// (its reciprocal could overflow); all codes of such a row are 0. A row with a
// NaN or an infinity has no codes that stand for it: its scale is NaN, and with
// it every output.
__device__ __forceinline__ float row_scale(float amax) {
  const float s = amax * (1.0f / 127.0f);
  return s < kFltMinNormal ? 1.0f : s < __builtin_inff() ? s : __builtin_nanf("");
}

// TPR threads share a row and keep it in registers, up to MAXB blocks of 16
// values each: one read of x, bound by the memory. [65536, 7168] bf16 takes
// 246 us (5.7 TB/s), [16384, 4096] 43 us; the GLU form of [16384, 2 x 1536]
// 25 us. GLU: a row of x holds 2C values, gate then up,
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
        for (int i = 0; i < 16; ++i) v[b][i] = swiglu(v[b][i], u[i]);
      } else {
        load16(x + row * C + j * 16, v[b]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = max_abs(amax, v[b][i]);
    }
  }
  static_assert(TPR == 64 || TPR == kQThreads, "a wave or a workgroup to a row");
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) amax = max_abs(amax, __shfl_xor(amax, o, 64));
  if constexpr (TPR > 64) {
    __shared__ float red[kQThreads / 64];
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int w = 1; w < kQThreads / 64; ++w) amax = max_abs(amax, red[w]);
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
  constexpr int64_t group = kQThreads / TPR, most = bsqh::max_blocks(kQThreads) * group;
  for (; rows > 0; rows -= most, x += most * C * (GLU ? 2 : 1), codes += most * C / 4, scales += most) {
    const int64_t n = rows < most ? rows : most;
    const dim3 grid((unsigned)((n + group - 1) / group));
#define BSQ_Q(MB) \
  hipLaunchKernelGGL((k_quant_int8<T, TPR, MB, GLU>), grid, dim3(kQThreads), 0, s, x, n, C, codes, scales)
    if (per <= 1) BSQ_Q(1);
    else if (per <= 2) BSQ_Q(2);
    else if (per <= 4) BSQ_Q(4);
    else BSQ_Q(8);
#undef BSQ_Q
  }
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
// Up to 64 rows of activations: bound by reading the weights once, and by how
// soon. A workgroup owns 16 weight rows for all M; its waves share K, each
// with a ring of R steps of 128 bytes in LDS of its own (no barriers), filled
// by loads that go straight there: eight lanes side by side read a whole line
// of a row (64 bytes a row took the address unit twice as long, a lane a row as
// in the matrix instruction's own layout four times). Piece p of row r lies at
// p ^ (r / 2 % 8), so that 16 rows at one piece meet 16 different banks. The
// exact integer partial sums meet in LDS. 50 x 2048 x 7168 takes 9.5 us (11.6
// with 64 bytes of a row a load; half of the CUs have no channels there, and
// every workgroup reads all activations), 64 x 8192 x 4096 15.9 us.
//
// FUSED: the activations come unquantized, few enough to lie in LDS (kFuseBytes);
// every workgroup quantizes them itself, while the first weights are on their
// way, and one launch is the whole layer. The codes are those of
// k_quant_int8: the same steps in the same order.
constexpr int kFuseBytes = 32768;
constexpr int kFuseCodes = 16384;
// Waves: as many as leave each of them a ring of three steps or more in 160 KB.
constexpr int few_waves(bool fused) { return fused ? 8 : 4; }

//
// N channels from the given ones on, in rows of `pitch` outputs.
template <typename X, typename T, int MT, bool FUSED>
__global__ __launch_bounds__(64 * few_waves(FUSED)) void k_gemm_int8_few(
    const X* __restrict__ a, const float* __restrict__ sa, const int8_t* __restrict__ b, const float* __restrict__ sb,
    const float* __restrict__ bias, int M, int N, int K, int pitch_out, T* __restrict__ out) {
  constexpr int kFWaves = few_waves(FUSED), kFThreads = 64 * kFWaves;
  constexpr int LOADS = FUSED ? 2 : 2 + 2 * MT;           // of a step: 8 rows of 128 bytes each
  constexpr int R = FUSED ? 4 : MT == 1 ? 8 : MT == 2 ? 5 : 3;
  constexpr int XLOADS = FUSED ? kFuseBytes / 1024 / kFWaves : 0;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kFWaves][R][LOADS * 1024];
  __shared__ i32x4 part[kFWaves][MT][64];
  __shared__ __attribute__((aligned(16))) uint8_t raw[FUSED ? kFuseBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t code[FUSED ? kFuseCodes + 16 * 16 + 128 : 16];
  __shared__ uint32_t rmax[16];
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63;
  const int n0 = (int)blockIdx.x * 16;
  const int rows_b = N - n0 < 16 ? N - n0 : 16;
  const int steps = (K + 127) / 128;
  const int st0 = steps * wave / kFWaves, st1 = steps * (wave + 1) / kFWaves;
  // what the epilogue will need, ahead of the stream
  constexpr int PER = (MT * 256 + kFThreads - 1) / kFThreads;
  float ea[PER], eb[PER], ec[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = t + i * kFThreads, row = j / 256 * 16 + (j >> 2 & 15), n = n0 + (j % 256 >> 6) * 4 + (j & 3);
    ea[i] = !FUSED ? sa[row < M ? row : M - 1] : 0.0f;
    eb[i] = sb[n < N ? n : N - 1];
    ec[i] = bias ? bias[n < N ? n : N - 1] : 0.0f;
  }
  const rsrc_words db = descriptor(b + (int64_t)n0 * K, (uint32_t)rows_b * K);
  const rsrc_words da = descriptor(a, FUSED ? (uint32_t)(M * K) * (uint32_t)sizeof(X) : (uint32_t)M * K);
  constexpr uint32_t kPastEnd = 0x40000000u;  // past every buffer here, once or twice
  // Rows past N or M are not fetched: what lies in their place meets outputs that are not stored.
  uint32_t vb[2], va[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int r = 8 * i + (lane >> 3);
    const uint32_t piece = (uint32_t)((lane & 7) ^ (r >> 1 & 7)) * 16;
    if (i < 2) vb[i < 2 ? i : 0] = r < rows_b ? (uint32_t)r * K + piece : kPastEnd;
    va[i] = r < M ? (uint32_t)r * K + piece : kPastEnd;
  }
  const uint32_t base = lds_offset(&ring[wave][0][0]);
  auto fetch = [&](int st, int place) {  // past the last step: issued all the same (the waits count them), past the end
    const uint32_t k = st < st1 ? (uint32_t)st * 128 : kPastEnd, at = base + place * (LOADS * 1024);
#pragma unroll
    for (int i = 0; i < 2; ++i) load_to_lds<16>(db, vb[i] + k, 0, at + i * 1024);
    if constexpr (!FUSED) {
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) load_to_lds<16>(da, va[i] + k, 0, at + (2 + i) * 1024);
    }
  };
  if constexpr (FUSED) {
    const uint32_t at = lds_offset(raw);
#pragma unroll
    for (int i = 0; i < XLOADS; ++i) {
      const int c = i * kFWaves + wave;
      load_to_lds<16>(da, c * 1024 + lane * 16, 0, at + c * 1024);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) fetch(st0 + i, i);
  const int pitch = K + 16;
  if constexpr (FUSED) {
    if (t < 16) rmax[t] = 0u;
    wait_loads<R * LOADS>();
    lds_barrier();
    const int per = K / 16, units = M * per;
    for (int u = t; u < units; u += kFThreads) {
      float v[16], mx = 0.0f;
      load16(reinterpret_cast<const X*>(raw) + u * 16, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = max_abs(mx, v[i]);
      atomicMax(&rmax[u / per], __float_as_uint(mx) & 0x7FFFFFFFu);  // by bits: a NaN's are above an infinity's
    }
    lds_barrier();
    for (int u = t; u < units; u += kFThreads) {
      const int row = u / per;
      const float inv = 1.0f / row_scale(__uint_as_float(rmax[row]));
      float v[16];
      load16(reinterpret_cast<const X*>(raw) + u * 16, v);
      *reinterpret_cast<u32x4*>(code + row * pitch + (u - row * per) * 16) =
          (u32x4){codes4(&v[0], inv), codes4(&v[4], inv), codes4(&v[8], inv), codes4(&v[12], inv)};
    }
    lds_barrier();
  }
  const int col = lane & 15, grp = lane >> 4;
  const uint8_t* crow = code + (FUSED && col < M ? col : 0) * pitch + grp * 16;  // lanes past M repeat row 0
  i32x4 acc[MT] = {};
  int place = 0;
#pragma unroll 1
  for (int st = st0; st < st1; ++st) {
    wait_loads<(R - 1) * LOADS>();
    i32x4 w[2], v[2][MT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 64 values of K each
      const uint8_t* p = &ring[wave][place][0] + col * 128 + ((4 * h + grp) ^ (col >> 1)) * 16;
      w[h] = *reinterpret_cast<const i32x4*>(p);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        v[h][m] = *reinterpret_cast<const i32x4*>(FUSED ? crow + st * 128 + h * 64 : p + (1 + m) * 2048);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the place may be filled again
    fetch(st + R, place);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (st * 128 + 128 > K && st * 128 + h * 64 + grp * 16 >= K) w[h] = (i32x4){0, 0, 0, 0};  // past the end of K
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h], v[h][m], acc[m], 0, 0, 0);
    }
    place = place == R - 1 ? 0 : place + 1;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) part[wave][m][lane] = acc[m];
  lds_barrier();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = t + i * kFThreads;
    if (j >= MT * 256) break;
    int s = 0;
#pragma unroll
    for (int w = 0; w < kFWaves; ++w) s += reinterpret_cast<const int*>(&part[w][0][0])[j];
    const int row = j / 256 * 16 + (j >> 2 & 15), n = n0 + (j % 256 >> 6) * 4 + (j & 3);
    if (row >= M || n >= N) continue;
    if constexpr (FUSED) ea[i] = row_scale(__uint_as_float(rmax[row]));
    float y = (float)s * ea[i] * eb[i];
    if (bias) y += ec[i];
    store1(out + (int64_t)row * pitch_out + n, y);
  }
}

// ---------------------------------------------------------------- many rows
// Tiles of 64 WM rows of activations by 64 WN rows of weights for a workgroup
// of four waves (32 WM x 32 WN each, v_mfma_i32_32x32x32_i8, all accumulators
// in registers). K advances in steps of KS bytes through a ring of ST stages in
// LDS, filled by loads that go straight there; the steps in flight are counted
// here, so a barrier a step is all that is waited for. A wave reads the next
// fragments while it multiplies: the barrier stands before the last
// instructions along a step, whose fragments are in registers by then, so that
// they cover the reads of the next step.
//
// 256 x 256 tiles are bound by the chip's power: the matrix instructions alone
// reach 3.4 POP/s on random codes (4.8 on zeros), and with them 62% of the
// cycles at a clock that sinks to 1.45 GHz the kernel runs at 1.9 to 2.2 POP/s
// (65536 x 2048 x 7168: 0.85 to 1.0 ms, with the loads left out 0.79). With
// short K a tile's first loads and its stores count too: 16384 x 4096 x 1536 (24
// steps) 143 us, 1.45 POP/s. Small tiles are bound by the latency of their
// loads: 128 bytes a row and step (L2 serves twice the bytes with whole lines),
// 96 KB of them in flight a CU.
//
// A stage's rows hold their 16-byte pieces in an order that depends on the row,
// so that 16 rows at one piece meet 16 different banks. Fragments past K (in a
// last step that is not whole) are set to zero on the
// weights' side; rows past M or N repeat the last one and are not stored.
//
// Weights are the matrix instruction's first operand: a lane then holds four
// neighbouring outputs of one row, which go through LDS (free by then) and
// leave as whole 16-byte pieces of rows.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// KS bytes of K a step (64 or 128), ST stages.
template <typename T, int WM, int WN, int KS, int ST>
__global__ __launch_bounds__(256, 1) void k_gemm_int8(const int8_t* __restrict__ a, const float* __restrict__ sa,
                                                     const int8_t* __restrict__ b, const float* __restrict__ sb,
                                                     const float* __restrict__ bias, int64_t M, int N, int K,
                                                     T* __restrict__ out) {
  constexpr int TM = 64 * WM, TN = 64 * WN;
  constexpr int STAGE = (TM + TN) * KS;         // bytes: rows of activations, then of weights
  constexpr int PR = KS / 16, RL = 64 / PR;     // pieces of a row, rows of a load
  constexpr int LA = TM / RL / 4, LB = TN / RL / 4;  // loads of a wave for a step
  constexpr int LOADS = LA + LB;
  constexpr int Q = KS / 32;                    // matrix instructions along a step
  constexpr int SLOTS = Q * WN;                 // rows of matrix instructions in a step
  // the output of a wave, 32 WM rows of COLS columns at a time
  constexpr int COLS = sizeof(T) == 2 ? 32 * WN : WN % 2 ? 32 : 16 * WN;
  constexpr int PITCH = COLS * (int)sizeof(T) + 16;
  constexpr int OUT = 32 * WM * PITCH;
  __shared__ __attribute__((aligned(16))) uint8_t lds[ST * STAGE > 4 * OUT ? ST * STAGE : 4 * OUT];
  __shared__ __attribute__((aligned(16))) float esa[TM], esb[TN], ebias[TN];
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63;
  // Workgroups go round the 8 XCDs; each XCD takes a contiguous part of the
  // tiles, columns first, so that the workgroups it runs at once share rows of
  // both operands in its L2.
  const int ntn = (N + TN - 1) / TN;
  const int64_t ntiles = gridDim.x;
  const int64_t per = ntiles / 8, extra = ntiles % 8;
  const int xcd = blockIdx.x % 8;
  const int64_t tile = xcd * per + (xcd < extra ? xcd : extra) + blockIdx.x / 8;
  const int64_t m0 = tile / ntn * TM;
  const int n0 = (int)(tile % ntn) * TN;
  const int rows_a = M - m0 < TM ? (int)(M - m0) : TM, rows_b = N - n0 < TN ? N - n0 : TN;
  const rsrc_words ra = descriptor(a + m0 * K, (uint32_t)rows_a * K);
  const rsrc_words rb = descriptor(b + (int64_t)n0 * K, (uint32_t)rows_b * K);
  // the tile's scales and bias, asked for before the products (loads in the
  // epilogue, each waited for, took 8 us a tile)
  const float ga = t < TM ? sa[m0 + (t < rows_a ? t : rows_a - 1)] : 0.0f;
  const float gb = t < TN ? sb[n0 + (t < rows_b ? t : rows_b - 1)] : 0.0f;
  const float gc = t < TN && bias ? bias[n0 + (t < rows_b ? t : rows_b - 1)] : 0.0f;
  // piece p of row r lies at p ^ swizzle(r), so that 16 rows at one piece meet 16 different banks
  auto swizzle = [](int r) { return r / (16 / PR) & (PR - 1); };
  uint32_t va[LA], vb[LB];
  {
    const int r = lane / PR;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int row = (wave * LA + i) * RL + r;
      va[i] = (uint32_t)(row < rows_a ? row : rows_a - 1) * K + ((lane % PR) ^ swizzle(row)) * 16;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int row = (wave * LB + i) * RL + r;
      vb[i] = (uint32_t)(row < rows_b ? row : rows_b - 1) * K + ((lane % PR) ^ swizzle(row)) * 16;
    }
  }
  const uint32_t base = lds_offset(lds);
  const int steps = (K + KS - 1) / KS;
  // Steps past the end are issued all the same (the waits count them), to empty
  // buffers. A stage's loads go out over a whole step, before the rows of matrix
  // instructions: issued together they fill the address unit's queue and the
  // wave stands behind it.
  auto fetch = [&](int step, int stage, int i) {
    if (i < LA) {
      rsrc_words d = ra;
      if (step >= steps) d[2] = 0u;
      load_to_lds<16>(d, va[i < LA ? i : 0] + step * KS, 0, base + stage * STAGE + (wave * LA + i) * 1024);
    } else {
      rsrc_words d = rb;
      if (step >= steps) d[2] = 0u;
      load_to_lds<16>(d, vb[i < LA ? 0 : i - LA] + step * KS, 0, base + stage * STAGE + TM * KS + (wave * LB + i - LA) * 1024);
    }
  };
  const int wm = wave >> 1, wn = wave & 1;
  i32x4 fa[2][WM], fb[2][WN];  // fragments of even and odd instructions along K
  // row lane % 32 of a 32-row fragment, piece 2 q + lane / 32
  const int myrow = (lane & 31) * KS, mysw = swizzle(lane & 31);
  auto read = [&](int stage, int q, int i) {
    const uint8_t* p = lds + stage * STAGE + myrow + ((2 * q + (lane >> 5)) ^ mysw) * 16 + i * 32 * KS;
    if (i < WN) fb[q & 1][i < WN ? i : 0] = *reinterpret_cast<const i32x4*>(p + (TM + wn * 32 * WN) * KS);
    if (i < WM) fa[q & 1][i < WM ? i : 0] = *reinterpret_cast<const i32x4*>(p + wm * (32 * WM) * KS);
  };
  i32x16 acc[WN][WM] = {};
  auto mask = [&](int step, int q) {
    if (step * KS + KS > K) {  // a last step that is not whole
      const bool in = step * KS + (2 * q + (lane >> 5)) * 16 < K;
#pragma unroll
      for (int i = 0; i < WN; ++i) fb[q & 1][i] = in ? fb[q & 1][i] : (i32x4){0, 0, 0, 0};
    }
  };
  constexpr int RD = (WM > WN ? WM : WN);  // fragment pairs to read for an instruction along K
  // slot k of the loads that fill one stage: the last WN rows of a step begin, the others end in the next step
  auto slot_of = [&](int step, int stage, int k) {
#pragma unroll
    for (int i = k * LOADS / SLOTS; i < (k + 1) * LOADS / SLOTS; ++i) fetch(step, stage, i);
  };
#pragma unroll
  for (int s = 0; s < ST; ++s)
#pragma unroll
    for (int k = 0; k < (s < ST - 1 ? SLOTS : WN); ++k) slot_of(s, s, k);
  wait_loads<(ST - 2) * LOADS + WN * LOADS / SLOTS>();
  lds_barrier();
#pragma unroll
  for (int i = 0; i < RD; ++i) read(0, 0, i);
  int stage = 0;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const int next = stage == ST - 1 ? 0 : stage + 1, last = stage == 0 ? ST - 1 : stage - 1;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (q == Q - 1) {
        wait_loads<(ST - 2) * LOADS>();  // the next stage has come
        lds_barrier();                   // for every wave, and this one is read
      }
      mask(step, q);
#pragma unroll
      for (int i = 0; i < WN; ++i) {
        if (q == Q - 1) slot_of(step + ST, stage, i);
        else slot_of(step + ST - 1, last, (q + 1) * WN + i);
#pragma unroll
        for (int z = i * RD / WN; z < (i + 1) * RD / WN; ++z) read(q == Q - 1 ? next : stage, (q + 1) % Q, z);
#pragma unroll
        for (int j = 0; j < WM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[q & 1][i], fa[q & 1][j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    stage = next;
  }
  wait_loads<0>();
  if (t < TM) esa[t] = ga;
  if (t < TN) esb[t] = gb, ebias[t] = gc;
  lds_barrier();

  // outputs: lane holds row lane % 32 of the 32 x 32 tile (i, j) and columns 8 (r / 4) + 4 (lane / 32) + r % 4
  uint8_t* mylds = lds + wave * OUT;
  const int64_t mw = m0 + wm * 32 * WM;
  float ma[WM];
#pragma unroll
  for (int j = 0; j < WM; ++j) ma[j] = esa[wm * 32 * WM + 32 * j + (lane & 31)];
  constexpr int HALVES = 32 * WN / COLS;
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    const int nw = n0 + wn * 32 * WN + h * COLS;
#pragma unroll
    for (int i = 0; i < COLS / 32; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int c = 32 * i + 8 * r + 4 * (lane >> 5);
        const int cn = wn * 32 * WN + h * COLS + c;
        const f32x4 s = *reinterpret_cast<const f32x4*>(esb + cn), add = *reinterpret_cast<const f32x4*>(ebias + cn);
#pragma unroll
        for (int j = 0; j < WM; ++j) {
          const i32x16& v = acc[h * (COLS / 32) + i][j];
          f32x4 y;
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            y[z] = (float)v[4 * r + z] * ma[j] * s[z];
            if (bias) y[z] += add[z];
          }
          uint8_t* at = mylds + (32 * j + (lane & 31)) * PITCH + c * (int)sizeof(T);
          if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2*>(at) = (u32x2){pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
          else *reinterpret_cast<f32x4*>(at) = y;
        }
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave reads what its own lanes wrote
    // 16-byte pieces of rows; rows of another pitch than 16 bytes take them unaligned, and the last piece of a row
    // that is not whole goes element by element
    constexpr int OP = COLS * (int)sizeof(T) / 16, EP = 16 / (int)sizeof(T);  // pieces of a row, elements of a piece
#pragma unroll 4
    for (int o = lane; o < 32 * WM * OP; o += 64) {
      const int row = o / OP, pc = o % OP;
      const int n = nw + pc * EP;
      if (mw + row < M && n < N) {
        T* to = out + (mw + row) * N + n;
        const T* from = reinterpret_cast<const T*>(mylds + row * PITCH + pc * 16);
        if (n + EP <= N) {
          *reinterpret_cast<u32x4_a2*>(to) = *reinterpret_cast<const u32x4*>(from);
        } else {
          for (int i = 0; n + i < N; ++i) to[i] = from[i];
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <typename X, typename T, int MT, bool FUSED>
void launch_few(const X* a, const float* sa, const int8_t* b, const float* sb, const float* bias, int64_t M, int64_t N,
                int64_t K, T* out, hipStream_t s) {
  constexpr int threads = 64 * few_waves(FUSED);
  constexpr int64_t most = bsqh::max_blocks(threads) * 16;
  for (int64_t n0 = 0; n0 < N; n0 += most) {
    const int64_t n = N - n0 < most ? N - n0 : most;
    hipLaunchKernelGGL((k_gemm_int8_few<X, T, MT, FUSED>), dim3((unsigned)((n + 15) / 16)), dim3(threads), 0, s, a, sa,
                       b + n0 * K, sb + n0, bias ? bias + n0 : nullptr, (int)M, (int)n, (int)K, (int)N, out + n0);
  }
}

template <typename T>
void launch_gemm(const int8_t* a, const float* sa, const int8_t* b, const float* sb, const float* bias, int64_t M,
                 int64_t N, int64_t K, T* out, hipStream_t s) {
  if (M <= 64) {
    if (M <= 16) launch_few<int8_t, T, 1, false>(a, sa, b, sb, bias, M, N, K, out, s);
    else if (M <= 32) launch_few<int8_t, T, 2, false>(a, sa, b, sb, bias, M, N, K, out, s);
    else launch_few<int8_t, T, 4, false>(a, sa, b, sb, bias, M, N, K, out, s);
    return;
  }
  const int64_t most = bsqh::max_blocks(256) / ((N + 127) / 128) * 128;  // rows that a launch of the smallest tiles takes
  if (M > most) {
    launch_gemm(a, sa, b, sb, bias, most, N, K, out, s);
    return launch_gemm(a + most * K, sa + most, b, sb, bias, M - most, N, K, out + most * N, s);
  }
  // Large tiles move fewer bytes for each product, small ones leave no CU idle.
  // Compared by the time of their rounds, in quarters of a 256 x 256 round (one
  // tile a CU): a round of one 128 x 128 tile a CU takes 1.15, of two 2.1.
  // Measured, 256 x 256 against 128 x 128: 1024 x 4096 x 4096 52 and 37 us (64
  // and 256 tiles), 2048 x 4096 x 4096 57 and 44 us, 3000 x 4096 x 4096 66 and
  // 63 us, 8192 x 1536 x 1536 34 and 35 us, 4096 x 4096 x 4096 74 and 77 us.
  // Where 128 x 128 tiles leave three CUs of four idle, 64 x 64 ones: 128 x 2048
  // x 7168 30 and 23 us, 256 x 4096 x 4096 21 and 17 us (64 tiles of 128 x 128;
  // with 128 of them, 512 x 4096 x 4096, 23 and 25 us). Where 128 x 128 tiles
  // are a few more than the CUs, 192 x 128 ones that are not: 384 x 12288 x 4096
  // 39 and 31 us, 3000 x 1536 x 4096 34 and 31 us, 1001 x 4099 x 1536 21 and 19 us.
  const int64_t cus = bsqh::device_cus();
  const int64_t big = ((M + 255) / 256) * ((N + 255) / 256), small = ((M + 127) / 128) * ((N + 127) / 128);
  const int64_t mid = ((M + 191) / 192) * ((N + 127) / 128);
  const double tb = 4.0 * (double)((big + cus - 1) / cus);
  const double ts = small <= cus ? 1.15 : 2.1 * (double)((small + 2 * cus - 1) / (2 * cus));
#define BSQ_G(WM, WN, KS, ST, TILES)                                                                                \
  hipLaunchKernelGGL((k_gemm_int8<T, WM, WN, KS, ST>), dim3((unsigned)(TILES)), dim3(256), 0, s, a, sa, b, sb, bias, M, \
                     (int)N, (int)K, out)
  if (4 * small <= cus) BSQ_G(1, 1, 128, 4, ((M + 63) / 64) * ((N + 63) / 64));
  else if (small <= cus) BSQ_G(2, 2, 128, 3, small);  // one workgroup a CU: more in flight each
  else if (mid <= cus) BSQ_G(3, 2, 128, 3, mid);
  else if (tb <= ts) BSQ_G(4, 4, 64, 4, big);
  else BSQ_G(2, 2, 128, 2, small);                    // two a CU
#undef BSQ_G
}

int check_gemm(int64_t M, int64_t N, int64_t K, int out_dtype) {
  BSQ_REQUIRE(out_dtype == BSQ_F32 || out_dtype == BSQ_BF16, BSQ_E_DTYPE);
  // 128 * 128 * K stays below 2^31; fewer than 2^31 tiles, and a launch takes those of 128 rows at least
  BSQ_REQUIRE(M >= 0 && M < (int64_t)1 << 31 && N >= 0 && N <= ((int64_t)1 << 31) - 256 && K >= 16 && K % 16 == 0 &&
                  K < 131072,
              BSQ_E_SHAPE);
  BSQ_REQUIRE(((M + 127) / 128) * ((N + 127) / 128) < (int64_t)1 << 31, BSQ_E_SHAPE);
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

// Whether the workgroups quantize the activations themselves: one launch, and no workspace.
static bool fused(int64_t M, int64_t K, int64_t bytes) {
  return M <= 16 && K <= kFuseCodes && M * K <= kFuseCodes && M * K * bytes <= kFuseBytes;
}

extern "C" size_t bsq_linear_int8_workspace(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0 || fused(M, K, 4)) return 0;
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
  const size_t need = bsq_linear_int8_workspace(M, K);
  BSQ_REQUIRE(x && b_codes && b_scales && out && (ws || need == 0), BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(x) && bsqh::aligned16(b_codes) && bsqh::aligned16(ws) && out_aligned(out, out_dtype) &&
                  (((uintptr_t)b_scales | (uintptr_t)bias) & 3) == 0,
              BSQ_E_ALIGN);
  BSQ_REQUIRE(ws_bytes >= need, BSQ_E_WORKSPACE);
  if (fused(M, K, dtype == BSQ_F32 ? 4 : 2)) {
#define BSQ_FUSED(X, T)                                                                                       \
  launch_few<X, T, 1, true>(static_cast<const X*>(x), nullptr, b_codes, b_scales, bias, M, N, K, static_cast<T*>(out), \
                            bsqh::as_stream(stream))
    if (dtype == BSQ_BF16 && out_dtype == BSQ_BF16) BSQ_FUSED(uint16_t, uint16_t);
    else if (dtype == BSQ_BF16) BSQ_FUSED(uint16_t, float);
    else if (out_dtype == BSQ_BF16) BSQ_FUSED(float, uint16_t);
    else BSQ_FUSED(float, float);
#undef BSQ_FUSED
    return bsqh::launch_status();
  }
  int8_t* codes = static_cast<int8_t*>(ws);
  float* scales = reinterpret_cast<float*>(codes + M * K);  // K % 16 == 0: aligned
  st = bsq_quantize_int8(x, dtype, M, K, codes, scales, stream);
  if (st != BSQ_OK) return st;
  return run_gemm(codes, scales, b_codes, b_scales, bias, M, N, K, out, out_dtype, stream);
}
