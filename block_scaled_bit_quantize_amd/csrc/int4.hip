// Weights in 4-bit integers with a scale, and a zero point, for each group of
// 32, 64 or 128 neighbours along K; products with unquantized activations.
//
//   w[n, k] = (q[n, k] - z[n, g]) s[n, g],  g = k / group, q and z in 0..15, z = 8 where there are no zero points
//   y[m, n] = sum_k x[m, k] w[n, k] + bias[n]
//
// The products compute with integers, which bf16 holds exactly, and bring the
// scale in once a group, in float32:
//   y[m, n] = sum_g s[n, g] sum_(k in g) (q[n, k] - z[n, g]) x[m, k]
// so that float32 sums are the only roundings before the output's for bf16
// activations. float32 ones go as two fp16 parts of their scaled row, 22 bits.
#include "bsq_int4.h"

using namespace bsqd;
using namespace bsqh;

namespace {

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
// long array of groups: K is whole groups. Bound by memory: 50021 x 4096 bf16,
// groups of 128, in 117 us, 4.4 TB/s; 2048 x 7168 float32, groups of 32, in 13.7.
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
// memory (a lane's four pieces side by side took 22 us for 2048 x 7168 float32, this
// 12.4, 5.3 TB/s; 50021 x 4096 to bf16 78 us, 6.6 TB/s).
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

// ---------------------------------------------------------------- many rows
// The weights are unpacked to 16-bit integers q - z once for all rows of
// activations (in the workspace, a slice of the rows of weights at a time), their
// scales turned to [group][row]; then tiles by matrix instructions. The
// accumulators hold the sum in units of the group's scale: before group g they
// are multiplied by s[g - 1] / s[g], at the end by the last scale, so that there
// is one set of them (a second one for the group's own sum left room for tiles of
// 256 x 128 only, which are bound by L2: 12 TB/s, 1.07 PFLOP/s).
constexpr int kUThreads = 256, kURows = 16;
// Scales too small for their row's largest are raised by a power of two, and their
// integers are that much smaller: exact, as long as the 16-bit type has the bits
// (fp16 down to 2^-24, bf16 to 2^-133). So the ratios of scales are finite, and
// none is zero: a scale of zero stands for integers of zero at the least scale.
// The sums in units of the least scale must not pass float32: bf16 x comes in any
// size, and all scales are raised to the largest's binade, so that the sums are
// below 30 sum |x|; float32 x is below 2^15, and 2^-64 leaves them below 2^100.
struct Raised {
  float scale, factor;  // of the integers
};
// top: exponent of the row's largest scale, 1/2 <= f < 1 in f 2^top.
template <typename X>
__device__ __forceinline__ int least_exponent(int top) {
  const int least = top - (sizeof(X) == 4 ? 64 : 0);
  return least > -125 ? least : -125;
}
__device__ __forceinline__ Raised raised(float s, int least) {
  if (s == 0.0f) return {__builtin_ldexpf(0.5f, least), 0.0f};
  const int up = least - __builtin_amdgcn_frexp_expf(s);  // of a NaN or an infinity 0: no output is finite
  if (up <= 0 || !(fabsf(s) < __builtin_inff())) return {s, 1.0f};
  return {__builtin_ldexpf(s, up), __builtin_ldexpf(1.0f, -up)};
}
// A wave a row of weights, 16 rows a workgroup, whose scales are turned in LDS (a
// wave's own stores of them, a line each: 4099 x 1536 in 11.6 and not 10.2 us).
// turned: [group][row] the scale of the group before over the group's, then the
// same of the scales (divisions here, once, cost the tiles nothing).
template <typename X>
__global__ __launch_bounds__(64 * kURows) void k_unpack_int4(const uint32_t* __restrict__ codes,
                                                          const uint16_t* __restrict__ scales,
                                                          const uint8_t* __restrict__ zeros, int64_t rows, int units,
                                                          int shift, int KG, int64_t pitch, u32x4* __restrict__ w,
                                                          float* __restrict__ turned) {
  __shared__ float table[2][64][kURows + 1];
  const int64_t row0 = (int64_t)blockIdx.x * kURows, row = row0 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int mine = row < rows ? KG : 0;  // groups: waves past the end have none
  float most = 0.0f;
  for (int g = lane; g < mine; g += 64) {
    const float s = fabsf(from_bf16(scales[row * KG + g]));
    most = s < __builtin_inff() ? fmaxf(most, s) : most;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
  const int least = least_exponent<X>(__builtin_amdgcn_frexp_expf(most));
  for (int g0 = 0; g0 < KG; g0 += 64) {
    const int g = g0 + lane;
    if (g < mine) {
      const float s = raised(from_bf16(scales[row * KG + g]), least).scale;
      table[0][lane][threadIdx.x >> 6] = g ? raised(from_bf16(scales[row * KG + g - 1]), least).scale / s : 0.0f;
      table[1][lane][threadIdx.x >> 6] = s;
    }
    __syncthreads();
    const int r = threadIdx.x % kURows, to = g0 + threadIdx.x / kURows;
    if (to < KG && row0 + r < rows) {
      turned[to * pitch + row0 + r] = table[0][threadIdx.x / kURows][r];
      turned[(KG + to) * pitch + row0 + r] = table[1][threadIdx.x / kURows][r];
    }
    __syncthreads();
  }
  if (row >= rows) return;
#pragma unroll 4
  for (int u = lane; u < units; u += 64) {  // eight codes
    const uint32_t c = codes[row * units + u];
    const int64_t g = row * KG + (u >> shift);
    const float z = zeros ? (float)zeros[g] : 8.0f, f = raised(from_bf16(scales[g]), least).factor;
    typename Mfma<X>::V v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = Mfma<X>::near(((float)(c >> (4 * j) & 15u) - z) * f);
    w[row * units + u] = __builtin_bit_cast(u32x4, v);
  }
}

// float32 activations as two planes of fp16, the smaller parts first, and what
// undoes the rows' scaling. A workgroup a row.
__global__ __launch_bounds__(kUThreads) void k_split_f32(const f32x4* __restrict__ x, int64_t rows, int K,
                                                        u32x4* __restrict__ planes, float* __restrict__ back) {
  __shared__ uint32_t red[kUThreads / 64];
  const int64_t row = blockIdx.x;
  const f32x4* from = x + row * (K / 4);
  uint32_t most = 0;
  for (int i = threadIdx.x; i < K / 4; i += kUThreads) {
    const u32x4 v = __builtin_bit_cast(u32x4, from[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) most = (v[j] & 0x7FFFFFFFu) > most ? v[j] & 0x7FFFFFFFu : most;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t other = (uint32_t)__shfl_xor((int)most, o, 64);
    most = other > most ? other : most;
  }
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kUThreads / 64; ++w) most = red[w] > most ? red[w] : most;
  const uint32_t e = row_factor(most);
  if (threadIdx.x == 0) back[row] = of_exponent(254u - e);
  for (int i = threadIdx.x; i < K / 8; i += kUThreads) {
    u32x4 hi, lo;
    split8(from[2 * i], from[2 * i + 1], of_exponent(e), hi, lo);
    planes[row * (K / 8) + i] = lo;
    planes[(rows + row) * (K / 8) + i] = hi;
  }
}

// A step is 64 values of K: rows of 128 bytes, of which the 16-byte piece p of
// row r lies at p ^ (r / 2 % 8), so that 16 rows at one piece meet 16 different
// banks. Waves of 32 MI x 32 NI outputs, WM x WN of them; K advances through a
// ring of ST stages in LDS, filled by loads that go straight there and are
// counted here. A wave reads the fragments of the instructions after the next
// while it multiplies (the ones right ahead came too late: 0.67 us a step of
// 128 x 128 tiles): the barrier stands before the last kAhead instructions along
// a step, whose fragments are in registers by then. 16384 x 4096 x 4096 in bf16:
// 470 to 490 us, 1.12 to 1.17 PFLOP/s (a library's bf16 product of these sizes 430
// us); 1001 x 4099 x 1536 in float32, two products each: 41 us, one round of 198
// tiles and their steps' latency.
constexpr int kStep = 64, kAhead = 2;
template <typename X, typename T, int G, int WM, int WN, int MI, int NI, int ST>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_gemm_int4(
    const uint16_t* __restrict__ a, int64_t plane, const float* __restrict__ back, const uint16_t* __restrict__ w,
    const float* __restrict__ turned, int64_t pitch, const float* __restrict__ bias, int64_t M, int N, int K,
    int64_t pitch_out, int splits, int64_t part, T* __restrict__ out) {
  constexpr int WAVES = WM * WN, PL = Mfma<X>::parts;
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
  // Workgroups go round the 8 XCDs; each XCD takes a contiguous part of the tiles, which lie in bands of kBand rows of
  // them, a band column by column: what an XCD runs at once shares rows of both operands in its L2.
  constexpr int kBand = 1024 / TM;
  const int ntn = (N + TN - 1) / TN;
  const int64_t ntiles = gridDim.x / splits;
  const int64_t per = ntiles / 8, extra = ntiles % 8;
  const int64_t b = blockIdx.x % ntiles;
  const int split = (int)(blockIdx.x / ntiles), xcd = (int)(b % 8);
  const int64_t tile = xcd * per + (xcd < extra ? xcd : extra) + b / 8;
  const int64_t band = tile / ((int64_t)kBand * ntn), in_band = tile - band * kBand * ntn;
  const int64_t left = ntiles / ntn - band * kBand;  // rows of tiles from the band on
  const int high = left < kBand ? (int)left : kBand;
  const int64_t m0 = (band * kBand + in_band % high) * TM;
  const int n0 = (int)(in_band / high) * TN;
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
  const rsrc_words rs = descriptor(turned + n0, (uint32_t)(((int64_t)(KG - 1) * pitch + TN) * 4));
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
    } else {  // 64 ratios of scales: part c of the step's groups (several waves may fetch the same)
      const int c = wave % (SCALES / 256);
      int g = step * kStep / G + c / (TN / 64);
      if (g >= KG) g = KG - 1;
      const uint32_t vs = (uint32_t)(((int64_t)g * pitch + c % (TN / 64) * 64 + lane) * 4);
      load_to_lds<4>(rs, buffer_at(there, true, vs, 0), at + (PL * TM + TN) * 128 + c * 256);
    }
  };
  // slot k of the loads that fill one stage: the last kAhead * NI rows of a step begin, the others end in the next step
  auto slot_of = [&](int step, int stage, int k) {
#pragma unroll
    for (int i = k * LOADS / SLOTS; i < (k + 1) * LOADS / SLOTS; ++i) fetch(step, stage, i);
  };
#pragma unroll
  for (int s = 0; s < ST; ++s)
#pragma unroll
    for (int k = 0; k < (s < ST - 1 ? SLOTS : kAhead * NI); ++k) slot_of(st0 + s, s, k);
  wait_loads<(ST - 2) * LOADS + kAhead * NI * LOADS / SLOTS>();
  lds_barrier();
  const int wm = wave / WN, wn = wave % WN;
  const int myrow = (lane & 31) * 128, mysw = lane >> 1 & 7;
  u32x4 fa[4][PL][MI], fb[4][NI];  // fragments of the instructions along a step, kAhead + 1 of them alive
  auto read = [&](int stage, int q, int i) {
    const uint8_t* p = lds + stage * STAGE + myrow + ((2 * q + (lane >> 5)) ^ mysw) * 16;
    if (i < NI) {
      fb[q][i < NI ? i : 0] = *reinterpret_cast<const u32x4*>(p + (PL * TM + (wn * NI + i) * 32) * 128);
    } else {
      const int j = i - NI < 0 ? 0 : i - NI, pl = j / MI, im = j % MI;
      fa[q][pl][im] = *reinterpret_cast<const u32x4*>(p + (pl * TM + (wm * MI + im) * 32) * 128);
    }
  };
#pragma unroll
  for (int q = 0; q < kAhead; ++q)
#pragma unroll
    for (int i = 0; i < FRAGS; ++i) read(0, q, i);
  f32x16 acc[MI][NI] = {};
  float ratio[GP][NI];  // of the groups that begin next
  auto ratios_of = [&](int stage) {
    const float* s = reinterpret_cast<const float*>(lds + stage * STAGE + (PL * TM + TN) * 128) + wn * 32 * NI + (lane & 31);
#pragma unroll
    for (int g = 0; g < GP; ++g)
#pragma unroll
      for (int j = 0; j < NI; ++j) ratio[g][j] = s[g * TN + j * 32];
  };
  ratios_of(0);
  auto products = [&](int q, int j, bool first) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (first) {
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] *= ratio[q / GQ][j];
      }
#pragma unroll
      for (int p = 0; p < PL; ++p) acc[i][j] = Mfma<X>::mul32(fa[q][p][i], fb[q][j], acc[i][j]);
    }
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
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q == 4 - kAhead) {
          wait_loads<(ST - 2) * LOADS>();  // the next stage has come
          lds_barrier();                   // for every wave, and this one is read
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (q >= 4 - kAhead) slot_of(step + ST, stage, (q - (4 - kAhead)) * NI + j);
          else slot_of(step + ST - 1, last, (q + kAhead) * NI + j);
          if (q == 3 && j == 0 && u == GS - 1) ratios_of(next);  // this step's are done with
#pragma unroll
          for (int z = j * FRAGS / NI; z < (j + 1) * FRAGS / NI; ++z)
            read(q >= 4 - kAhead ? next : stage, (q + kAhead) % 4, z);
          products(q, j, q % GQ == 0 && u == 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      stage = next;
    }
  }
  static_assert(kAhead == 2, "half a step is in registers");
  if (half) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < NI; ++j) products(q, j, q == 0);
  }
  wait_loads<0>();
  lds_barrier();

  // outputs: lane holds column lane % 32 and rows 8 (r / 4) + 4 (lane / 32) + r % 4 of the 32 x 32 tile (i, j); they
  // leave through LDS, 32 rows of the wave at a time, as 16-byte pieces of rows
  // in units of the last group's scale
  float scale[NI] = {};
  if (st0 < st1) {
    const int g = (st1 * kStep < K ? st1 * kStep : K) / G - 1;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int n = n0 + (wn * NI + j) * 32 + (lane & 31);  // the last tile may be wider than the scales' pitch
      if (n < N) scale[j] = turned[(int64_t)(KG + g) * pitch + n];
    }
  }
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
        float y = scale[j] * acc[i][j][r];
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
                                                        int64_t M, int64_t N, const float* __restrict__ bias,
                                                        int64_t pitch_out, T* __restrict__ out) {
  const int64_t u = (int64_t)blockIdx.x * kUThreads + threadIdx.x;
  if (u >= part) return;
  float y = 0.0f;
  for (int s = 0; s < splits; ++s) y += parts[s * part + u];
  const int64_t m = u / N, n = u - m * N;
  if (bias) y += bias[n];
  store1(out + m * pitch_out + n, y);
}

// How a call's work is laid out.
struct Plan {
  enum Way { kShare, kSlabs, kTiles } way;
  int64_t rows;      // of x a launch
  int mt;            // kSlabs: rows of 16
  int64_t slab;      // kSlabs: values of K of a workgroup
  int splits;        // slabs, or parts of K of a tile
  int64_t slice;     // rows of weights at a time (kTiles: of 128)
  int tile;          // kTiles: see launch_tiles
  size_t w, s, x, back, parts;  // bytes of the workspace
};

constexpr int64_t kUnpacked = (int64_t)128 << 20;  // bytes of unpacked weights at a time
constexpr int64_t kPlanes = (int64_t)64 << 20;    // bytes of split activations at a time
constexpr int64_t kParts = (int64_t)128 << 20;    // bytes of slabs' sums at a time
constexpr int64_t kSplits = (int64_t)96 << 20;    // bytes of the sums of a split K

Plan plan_of(int64_t M, int64_t N, int64_t K, int64_t group, int dtype) {
  Plan p = {};
  const int64_t size = dtype == BSQ_F32 ? 4 : 2, cus = bsqh::device_cus();
  p.splits = 1;
  if (M <= 16 && share_bytes(M, K, group, size) <= kFewLds) {
    p.way = Plan::kShare;
    p.rows = M;
    p.slab = K;
    return p;
  }
  // A launch of slabs takes up to 64 rows, and reads all weights; the tiles' way
  // unpacks them first. 4096 x 4096 in bf16: 64 rows 17 and 30 us, 128 rows 35 and
  // 30 us; 100003 x 4096: 128 rows 320 and 550 us, 256
  // rows 640 and 600 us. float32: 64 rows 28 and 37 us,
  // 128 rows 55 and 37 us.
  const int64_t launches = (M + 63) / 64, few = N * K < (int64_t)1 << 26 ? 1 : dtype == BSQ_F32 ? 2 : 3;
  if (launches <= few) {
    p.way = Plan::kSlabs;
    p.rows = (M + launches - 1) / launches;
    p.mt = p.rows <= 16 ? 1 : p.rows <= 32 ? 2 : 4;
    // whole loads, kSlabLds of x at most, and as many slabs as give each wave of the card a tile
    const int64_t unit = 1024 / size, most = kSlabLds / (16 * p.mt * size), tiles = (N + 15) / 16;
    int64_t want = (kFWaves * cus + tiles - 1) / tiles;
    if (want < (K + most - 1) / most) want = (K + most - 1) / most;
    p.slab = ((K + want - 1) / want + unit - 1) / unit * unit;
    p.splits = (int)((K + p.slab - 1) / p.slab);
    p.slice = N;
    if (p.splits > 1) {
      const int64_t wide = kParts / (p.splits * p.rows * 4) / 128 * 128;
      if (wide < p.slice) p.slice = wide;
      p.parts = (size_t)(p.splits * p.rows * p.slice * 4);
    }
    return p;
  }
  p.way = Plan::kTiles;
  const int64_t whole = (N + 127) / 128 * 128;
  p.slice = kUnpacked / (2 * K) / 128 * 128;
  if (whole < p.slice) p.slice = whole;
  // fewer than 2^24 workgroups of 256 work-items
  p.rows = ((int64_t)1 << 22) / (p.slice / 128) * 128;
  if (dtype == BSQ_F32 && kPlanes / (4 * K) / 256 * 256 < p.rows) p.rows = kPlanes / (4 * K) / 256 * 256;
  if (M < p.rows) p.rows = M;
  if (dtype == BSQ_F32) {
    p.x = (size_t)(p.rows * K * 4);
    p.back = (size_t)((p.rows + 767) / 768 * 768 * 4);  // whole tiles of 64, 128 and 192 rows
  }
  p.w = (size_t)(p.slice * K * 2);
  p.s = (size_t)(p.slice * (K / group) * 8);
  // The tile and the parts of K of the least time: rounds of a tile a CU, each of
  // so many us a step of 64 along K, and the parts' second launch (5 us and its
  // bytes at 4 TB/s). Measured a step: bf16 128 x 128 0.53 to 0.61, 256 x 128 0.71
  // to 0.98, 256 x 256 1.45 to 1.8 us; float32 128 x 128 0.98, 192 x 128 1.33, 128 x
  // 256 1.45 to 1.84 us. 4096 x 4096 in bf16: 256 rows 47, 38, 34 us in 1, 2, 4 parts
  // of 128 x 128; 1536 rows 80, 65, 109 us by the three tiles; 16384 rows 700, 500, 470.
  static constexpr struct {
    int m, n;
    double us;
  } kTilesOf[2][3] = {{{128, 128, 0.57}, {256, 128, 0.9}, {256, 256, 1.7}}, {{128, 128, 0.95}, {192, 128, 1.35}, {128, 256, 1.75}}};
  const int64_t steps = (K + kStep - 1) / kStep;
  double least = 1e30;
  for (int t = 0; t < 3; ++t)
    for (int64_t sp = 1; sp <= 8 && (sp == 1 || steps >= 8 * sp); sp *= 2) {
      const auto& tile = kTilesOf[dtype == BSQ_F32][t];
      const int64_t n = ((p.rows + tile.m - 1) / tile.m) * ((p.slice + tile.n - 1) / tile.n) * sp;
      if (sp > 1 && sp * p.rows * p.slice * 4 > kSplits) break;
      double us = (double)((n + cus - 1) / cus) * (double)((steps + sp - 1) / sp) * tile.us;
      if (sp > 1) us += 5.0 + (double)(sp * p.rows * p.slice) * 8.0 / 4e6;
      if (us < least) least = us, p.tile = t, p.splits = (int)sp;
    }
  if (p.splits > 1) p.parts = (size_t)(p.splits * p.rows * p.slice * 4);
  return p;
}

template <typename X, typename T, int G>
void launch_tiles(const Plan& p, const uint16_t* a, int64_t plane, const float* back, const uint16_t* w, const float* sc,
                  const float* bias, int64_t M, int64_t N, int64_t K, int64_t pitch_out, int64_t part, T* out,
                  hipStream_t s) {
#define BSQ_TILE(WM, WN, MI, NI, ST)                                                                                   \
  hipLaunchKernelGGL((k_gemm_int4<X, T, G, WM, WN, MI, NI, ST>),                                                     \
                     dim3((unsigned)(((M + 32 * MI * WM - 1) / (32 * MI * WM)) * ((N + 32 * NI * WN - 1) / (32 * NI * WN)) * \
                                     p.splits)),                                                                      \
                     dim3(64 * WM * WN), 0, s, a, plane, back, w, sc, p.slice, bias, M, (int)N, (int)K, pitch_out,    \
                     p.splits, part, out)
  if constexpr (sizeof(X) == 2) {
    if (p.tile == 0) BSQ_TILE(4, 2, 1, 2, 4);
    else if (p.tile == 1) BSQ_TILE(4, 2, 2, 2, 3);
    else BSQ_TILE(2, 4, 4, 2, 2);
  } else {
    if (p.tile == 0) BSQ_TILE(4, 2, 1, 2, 3);
    else if (p.tile == 1) BSQ_TILE(2, 4, 3, 1, 2);
    else BSQ_TILE(2, 4, 2, 2, 2);
  }
#undef BSQ_TILE
}

template <typename X, typename T, int G>
int run_linear(const X* x, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const float* bias,
               int64_t M, int64_t N, int64_t K, T* out, uint8_t* ws, hipStream_t s) {
  const Plan p = plan_of(M, N, K, G, sizeof(X) == 4 ? BSQ_F32 : BSQ_BF16);
  auto join = [&](const float* parts, int64_t m, int64_t n, const float* add, T* to) {
    const int64_t part = m * n;
    hipLaunchKernelGGL((k_join_int4<T>), dim3((unsigned)((part + kUThreads - 1) / kUThreads)), dim3(kUThreads), 0, s,
                       parts, p.splits, part, m, n, add, N, to);
  };
  if (p.way != Plan::kTiles) {
    Int4Few c = {x, sizeof(X) == 4 ? BSQ_F32 : BSQ_BF16, codes, scales, zeros, G, bias, M, N, K, p.mt, p.slab, p.splits,
                 reinterpret_cast<float*>(ws), N, out, sizeof(T) == 4};
    if (p.way == Plan::kShare) {
      int4_share(c, s);
      return launch_status();
    }
    for (int64_t n0 = 0; n0 < N; n0 += p.slice) {
      c.N = N - n0 < p.slice ? N - n0 : p.slice;
      c.codes = codes + n0 * (K / 2);
      c.scales = scales + n0 * (K / G);
      c.zeros = zeros ? zeros + n0 * (K / G) : nullptr;
      c.bias = bias ? bias + n0 : nullptr;
      for (int64_t m0 = 0; m0 < M; m0 += p.rows) {
        c.M = M - m0 < p.rows ? M - m0 : p.rows;
        c.x = x + m0 * K;
        c.out = out + m0 * N + n0;
        int4_slabs(c, s);
        if (p.splits > 1) join(c.parts, c.M, c.N, c.bias, out + m0 * N + n0);
      }
    }
    return launch_status();
  }
  u32x4* w = reinterpret_cast<u32x4*>(ws);
  float* turned = reinterpret_cast<float*>(ws + p.w);
  uint16_t* planes = reinterpret_cast<uint16_t*>(ws + p.w + p.s);
  float* back = reinterpret_cast<float*>(ws + p.w + p.s + p.x);
  float* parts = reinterpret_cast<float*>(ws + p.w + p.s + p.x + p.back);
  const int64_t KG = K / G;
  for (int64_t n0 = 0; n0 < N; n0 += p.slice) {
    const int64_t n = N - n0 < p.slice ? N - n0 : p.slice;
    hipLaunchKernelGGL((k_unpack_int4<X>), dim3((unsigned)((n + kURows - 1) / kURows)), dim3(64 * kURows), 0,
                       s, reinterpret_cast<const uint32_t*>(codes + n0 * (K / 2)), scales + n0 * KG,
                       zeros ? zeros + n0 * KG : nullptr, n, (int)(K / 8), G == 32 ? 2 : G == 64 ? 3 : 4, (int)KG, p.slice,
                       w, turned);
    for (int64_t m0 = 0; m0 < M; m0 += p.rows) {
      const int64_t m = M - m0 < p.rows ? M - m0 : p.rows;
      const uint16_t* a = reinterpret_cast<const uint16_t*>(x + m0 * K);
      if constexpr (sizeof(X) == 4) {
        if (n0 == 0 || M > p.rows)
          hipLaunchKernelGGL(k_split_f32, dim3((unsigned)m), dim3(kUThreads), 0, s,
                             reinterpret_cast<const f32x4*>(x + m0 * K), m, (int)K, reinterpret_cast<u32x4*>(planes), back);
        a = planes;
      }
      const uint16_t* wb = reinterpret_cast<const uint16_t*>(w);
      const float* add = bias ? bias + n0 : nullptr;
      T* to = out + m0 * N + n0;
      if (p.splits == 1) {
        launch_tiles<X, T, G>(p, a, m * K, back, wb, turned, add, m, n, K, N, 0, to, s);
      } else {
        launch_tiles<X, float, G>(p, a, m * K, back, wb, turned, nullptr, m, n, K, n, m * n, parts, s);
        join(parts, m, n, add, to);
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
