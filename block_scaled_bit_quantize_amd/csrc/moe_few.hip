// A whole NVFP4 expert layer for a few tokens (decode), without dispatch.
//
//   y_t = sum_j w_tj W2_e (silu(G) * U),  (G; U) = W13_e x_t,  e = ids[t, j]
//
// The many-token chain gathers rows into 256-row tiles per expert; for a few
// tokens an expert sees one to some tens of rows, and what bounds the layer is
// reading the chosen experts' weights (0.5625 bytes a value) once.
//
// Both products run as streams: one workgroup per CU takes an equal share of
// the sequence of (slot, row tile), a slot being an expert and up to 16 of the
// pairs that chose it. Its eight waves
// share the inner dimension. A wave keeps its part of the activations of an
// expert's tokens in registers and lets the weights pass by through a ring of
// three places in LDS: loads that go straight to LDS (no registers in flight,
// and 8 lanes side by side read a whole 128-byte line; with each lane reading
// its own MFMA row the address unit took one lane a cycle and was the limit).
// Up to 110 KB a CU are in flight, across tile ends too; the waves' partial
// sums meet in LDS, in two buffers, with one barrier a tile that leaves the
// loads in flight. 64 tokens, top 8 of 64 experts of 1536, hidden 4096: W13
// 96 us (453 MB, 4.7 TB/s; 8 us of them for the barrier and the stores), W2 62
// to 69 us (226 MB, 3.3 to 3.7 TB/s; 13 us of them besides the stream, and its
// six spans of K leave two of the eight waves without one), where plain reads
// reach 5.9 TB/s. One token: 16.6 and 14.6 us, of which the first bytes' way
// (ids, expert, descriptor, latency) is about 5 each.
//
// Weights are decoded to fp16 exactly (an E2M1 value times its E4M3 scale has
// at most 6 significant bits and lies in [2^-10, 2688]): a convert and a
// packed multiply, one instruction a weight. Activations are scaled by a power
// of two for each token and wave, so that the largest lies near 2^14, and
// split into fp16 terms: bf16 inputs are one term, exact down to 2^-31 of the
// largest, float32 inputs and the SwiGLU result two, 22 bits down to 2^-16 of
// the largest. What is smaller is off by half of fp16's least step, 2^-24, and
// so by 2^-39 of the largest at most.
// v_mfma_f32_16x16x32_f16 sums in float32; the powers of two are taken back
// before the waves' sums are added, the outer scales and the token's weight
// after.
//
// Which experts occur is read from the ids by every workgroup itself, so the
// layer is three launches: W13 with SwiGLU, W2 into one row per (token, slot)
// pair, and the sum over a token's pairs in slot order (no atomics: the same
// bits every time). Up to 16 pairs W2 and the sum are one (k_moe_last).
#include "bsq_device.h"
#include "bsq_internal.h"
#include "bsq_lds.h"

using namespace bsqd;

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t brsrc_t;

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxPairs = BSQ_MOE_FEW_MAX_PAIRS;
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Operands are read through buffer descriptors: a 32-bit offset per lane, the
// tile's and step's offset in a scalar register.
__device__ __forceinline__ brsrc_t buffer(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// ---------------------------------------------------------------- operands
// A step is 128 values of K: 8 blocks. Lane (c, g) = (lane % 16, lane / 16) of
// a wave holds blocks 2 g and 2 g + 1 of a step for row c: of the weights 16
// bytes of codes and two scales. Each of a step's four MFMAs takes 8 values of
// every lane; the order of K is the same for the activations.

// A step's 32 weights of a lane: four MFMA operands (kept as words: vectors of
// halves took a register for each half where control flow joins).
__device__ __forceinline__ uint32_t as_word(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ void decode(u32x4 codes, uint32_t scales, u32x4 (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s = i < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)scales, 0) : __builtin_amdgcn_cvt_f32_fp8((int)scales, 1);
    const f16x2 s2 = {(_Float16)s, (_Float16)s};
    const uint32_t c = codes[i];
    o[i] = (u32x4){as_word(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * s2),
                   as_word(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * s2),
                   as_word(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * s2),
                   as_word(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * s2)};
  }
}

// A lane's 32 activations of a step as they lie in memory, blocks b0 and
// b0 + 1, zeros unless the block is in [first, last). aoff: the lane's row in
// bytes.
template <typename T>
struct Raw {
  u32x4 v[32 * sizeof(T) / 16];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(brsrc_t act, uint32_t aoff, int b0, int first, int last) {
  constexpr int Z = (int)sizeof(T), N = 16 * Z / 16;
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t at = b0 + i >= first && b0 + i < last ? aoff + (uint32_t)(b0 + i) * (16 * Z) : kPastEnd;
#pragma unroll
    for (int q = 0; q < N; ++q)
      r.v[i * N + q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(act, at, q * 16, 0));
  }
  return r;
}
__device__ __forceinline__ float raw_get(const Raw<uint16_t>& r, int i) {
  const uint32_t w = r.v[i / 8][(i % 8) / 2];
  return i & 1 ? bf16_hi(w) : bf16_lo(w);
}
__device__ __forceinline__ float raw_get(const Raw<float>& r, int i) { return __uint_as_float(r.v[i / 4][i % 4]); }
template <typename T>
__device__ __forceinline__ float raw_max(const Raw<T>& r, float m) {
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(raw_get(r, i)));
  return m;
}
// NT fp16 terms of the activations times `scale`: rounded to nearest, the next
// term takes the (exact) remainder.
template <typename T, int NT>
__device__ __forceinline__ void split(const Raw<T>& r, float scale, u32x4 (&o)[NT][4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw_get(r, 8 * q + i) * scale;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f16x2 h = __builtin_convertvector((f32x2){v[2 * i], v[2 * i + 1]}, f16x2);
        o[t][q][i] = as_word(h);
        if (t + 1 < NT) {
          v[2 * i] -= (float)h[0];
          v[2 * i + 1] -= (float)h[1];
        }
      }
  }
}

// The power of two that brings a maximum into [2^14, 2^15), and its inverse,
// from the exponent bits; below 2^-111 and for infinities the nearest usable.
struct Scale {
  float up, down;
};
__device__ __forceinline__ Scale scale_for(float amax) {
  int e = (int)(__float_as_uint(amax) >> 23);
  e = e < 16 ? 16 : e > 254 ? 254 : e;
  return {__uint_as_float((uint32_t)(268 - e) << 23), __uint_as_float((uint32_t)(e - 14) << 23)};
}

template <int NT>
__device__ __forceinline__ f32x4 multiply(const u32x4 (&w)[4], const u32x4 (&a)[NT][4], f32x4 acc) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w[q]), __builtin_bit_cast(f16x8, a[t][q]),
                                                   acc, 0, 0, 0);
  return acc;
}

// ---------------------------------------------------------------- which experts
// The experts that occur, as slots 0 .. slots - 1: a slot is an expert and 16
// (or the last few) of the pairs that chose it, which is one pass over its
// weights. (Slots, and not experts, are what the workgroups share out: where a
// few experts take most tokens, shares of experts left the others waiting.)
// Up to 64 pairs: every wave holds all ids, a lane each, and sees an expert's
// first pair and its number of pairs by ballots (no barrier). More: the ids are
// spread over the workgroup's registers and the pairs of each expert counted
// in LDS; lane l of every wave holds the running sums of the slots of experts
// [16 l, 16 l + 16).
struct RouteLds {
  uint32_t pairs[kMaxExperts / 2];  // of two experts a word (at most kMaxPairs each)
  int count[kMaxPairs / kThreads * kWaves];
  uint16_t list[kMaxPairs];
};
struct Slot {
  int expert, part;  // pairs [16 part, 16 part + 16) of the expert's
};
struct Route {
  static constexpr int C = kMaxPairs / kThreads;
  static constexpr int G = kMaxExperts / 64;  // experts of a lane
  int id[C];
  bool few;
  uint64_t first;  // few: the first pair of each expert
  int upto;        // else: slots of this lane's experts and of all before
  int slots;

  __device__ __forceinline__ static int slots_of(uint32_t n) { return (int)((n + 15) / 16); }
  __device__ __forceinline__ static int pairs_of(const RouteLds& lds, int e) {
    return (int)(lds.pairs[e >> 1] >> (16 * (e & 1)) & 0xFFFFu);
  }

  __device__ __forceinline__ void init(const int32_t* __restrict__ ids, int pairs, int E, RouteLds& lds) {
    const int t = threadIdx.x, lane = t & 63;
    slots = 0;
    first = 0;
    upto = 0;
    few = pairs <= 64;
    if (few) {
      const int v = ids[lane < pairs ? lane : 0];
      id[0] = lane < pairs && v < E ? v : -1;
      if (pairs <= 16) {  // no loop over experts, whose turns each wait for the one before
        bool again = id[0] < 0;
#pragma unroll
        for (int p = 0; p < 15; ++p) again |= lane > p && id[0] == __builtin_amdgcn_readlane(id[0], p);
        first = __ballot(!again);
        slots = __popcll(first);
        return;
      }
      for (uint64_t rem = __ballot(id[0] >= 0); rem;) {
        const int p = __ffsll((unsigned long long)rem) - 1;
        const uint64_t m = __ballot(id[0] == __builtin_amdgcn_readlane(id[0], p));
        first |= 1ull << p;
        slots += slots_of(__popcll(m));
        rem &= ~m;
      }
      return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int p = t + c * kThreads;
      id[c] = -1;
      if (c * kThreads < pairs) {
        const int v = ids[p < pairs ? p : 0];
        id[c] = p < pairs && v < E ? v : -1;
      }
    }
    static_assert(kMaxExperts / 2 == kThreads, "a word each");
    lds.pairs[t] = 0;
    lds_barrier();
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (id[c] >= 0) atomicAdd(&lds.pairs[id[c] >> 1], 1u << (16 * (id[c] & 1)));
    lds_barrier();
#pragma unroll
    for (int w = 0; w < G / 2; ++w) {
      const uint32_t n = lds.pairs[lane * (G / 2) + w];
      upto += slots_of(n & 0xFFFFu) + slots_of(n >> 16);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    slots = __builtin_amdgcn_readlane(upto, 63);
  }

  // A slot below `slots`, counted out by the scalar unit.
  __device__ __forceinline__ Slot slot(int s, const RouteLds& lds) const {
    if (few) {
      uint64_t rem = first;
      for (;; rem &= rem - 1) {
        const int e = __builtin_amdgcn_readlane(id[0], __ffsll((unsigned long long)rem) - 1);
        const int n = slots_of(__popcll(__ballot(id[0] == e)));
        if (s < n) return {e, s};
        s -= n;
      }
    }
    const int src = __ffsll((unsigned long long)__ballot(s < upto)) - 1;
    if (src > 0) s -= __builtin_amdgcn_readlane(upto, src - 1);
    int e = src * G;
#pragma unroll 1
    for (;; ++e) {
      const int n = slots_of(uniform(pairs_of(lds, e)));
      if (s < n) return {e, s};
      s -= n;
    }
  }

  // Writes the pairs of an expert into lds.list, ascending, and returns how
  // many they are. Every wave calls it, after its last use of the list before.
  __device__ __forceinline__ int list_pairs(int expert, int pairs, RouteLds& lds) const {
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    if (few) {
      const uint64_t m = __ballot(id[0] == expert);
      if (wave == 0 && id[0] == expert) lds.list[__popcll(m & ((1ull << lane) - 1))] = (uint16_t)lane;
      lds_barrier();
      return __popcll(m);
    }
    uint64_t mask[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      mask[c] = __ballot(id[c] == expert);
      if (lane == 0) lds.count[c * kWaves + wave] = __popcll(mask[c]);
    }
    lds_barrier();
    const int counts = lds.count[lane & (C * kWaves - 1)];
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c * kThreads < pairs) {
        int mine = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          if (w == wave) mine = n;
          n += __builtin_amdgcn_readlane(counts, c * kWaves + w);
        }
        if (id[c] == expert) lds.list[mine + __popcll(mask[c] & ((1ull << lane) - 1))] = (uint16_t)(t + c * kThreads);
      }
    }
    lds_barrier();
    return n;
  }
};

// ---------------------------------------------------------------- the stream
struct Product {
  const void* in;         // activations: row of pair p is p / share
  const int32_t* ids;
  int pairs, k, E, K;
  int width;              // outputs of a pair
  int share;              // k for W13, 1 for W2
  const uint8_t* codes;
  const uint8_t* scales;
  const float* outer;
  float* out;             // [pairs, width]
  int span0, spans;       // k_moe_stream: the part of K, in spans of 256 values
};

// The end of a tile: the waves' partial sums of 16 x 16 outputs meet in LDS and
// are stored. GLU (W13): the tiles are gate rows, then their up rows, and the
// result is silu(gate) * up. Otherwise (W2) RT * 16 rows. One barrier, which
// leaves loads in flight, and no load of its own, whose wait would be one for
// all that are in flight (the pairs' weights are left to the last sum); the
// caller alternates between two buffers.
template <bool GLU, int RT>
__device__ __forceinline__ void finish(const Product& a, float (&part)[kWaves][RT][256], const f32x4 (&acc)[RT],
                                       float down, int tile, int mt0, int np, float so, const uint16_t* list) {
  constexpr int OUT = GLU ? RT * 8 : RT * 16, PER = OUT * 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < RT; ++i) *reinterpret_cast<f32x4*>(&part[wave][i][lane * 4]) = acc[i] * down;
  lds_barrier();
  int o0 = threadIdx.x;
  asm volatile("" : "+v"(o0));  // its addresses are formed here, not kept in registers over the stream
  // float j of a 16 x 16 tile is row 4 (j / 64) + j % 4 of pair j / 4 % 16
  for (int o = o0; o < PER; o += kThreads) {
    const int i = o / 256, j = o % 256;
    const int q = mt0 + (j >> 2 & 15);
    const int f = tile * OUT + 16 * i + 4 * (j >> 6) + (j & 3);
    float v = part[0][i][j];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += part[w][i][j];
    if constexpr (GLU) {
      float up = part[0][i + RT / 2][j];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) up += part[w][i + RT / 2][j];
      const float g = v * so;
      v = g / (1.0f + expf(-g)) * (up * so);
    }
    if (q < np && f < a.width) {
      if constexpr (!GLU) v *= so;
      a.out[(int64_t)list[q] * a.width + f] = v;
    }
  }
}

// Rows of one block (K = 16), which k_moe_stream's loads do not take: weights
// and activations straight to registers, read again for every tile.
template <typename T, int NT, bool GLU, int RT>
__global__ __launch_bounds__(kThreads, 2) void k_moe_any(Product a) {
  constexpr int OUT = GLU ? RT * 8 : RT * 16;  // outputs of a tile
  __shared__ RouteLds lds;
  __shared__ float part[2][kWaves][RT][256];
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63;
  const int col = lane & 15, grp = lane >> 4;
  Route route;
  route.init(a.ids, a.pairs, a.E, lds);
  const int tiles = (a.width + OUT - 1) / OUT;
  const int64_t units = (int64_t)route.slots * tiles;
  int u = uniform((int)(units * blockIdx.x / gridDim.x));
  const int u1 = uniform((int)(units * (blockIdx.x + 1) / gridDim.x));
  const int nblk = a.K / 16;
  const int steps = (nblk + 7) / 8;
  const int st0 = steps * wave / kWaves, st1 = steps * (wave + 1) / kWaves;
  const int rows = GLU ? 2 * a.width : a.width;
  const brsrc_t act = buffer(a.in, (int64_t)(a.pairs / a.share) * a.K * (int)sizeof(T));
  int buf = 0;
  while (u < u1) {
    const int at = u / tiles, tile0 = u - at * tiles;
    const int tile1 = tile0 + (u1 - u) < tiles ? tile0 + (u1 - u) : tiles;
    u += tile1 - tile0;
    const Slot slot = route.slot(at, lds);
    const int expert = uniform(slot.expert), mt0 = uniform(slot.part) * 16;
    const int np = uniform(route.list_pairs(expert, a.pairs, lds));
    const int64_t wrow = (int64_t)expert * rows;
    const brsrc_t codes = buffer(a.codes + wrow * (a.K / 2), (int64_t)rows * (a.K / 2));
    const brsrc_t scales = buffer(a.scales + wrow * nblk, (int64_t)rows * nblk);
    const float so = a.outer[expert];
    {
      const int mine = lds.list[mt0 + col < np ? mt0 + col : mt0];
      const uint32_t aoff = (uint32_t)(mine / a.share * a.K) * (uint32_t)sizeof(T);
      auto raw_at = [&](int st) {
        const int b = st * 8 + grp * 2;
        return load_raw<T>(act, aoff, b, b, nblk);
      };
      float mx = 0.0f;
      for (int st = st0; st < st1; ++st) mx = raw_max(raw_at(st), mx);
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const Scale sc = scale_for(mx);
#pragma unroll 1
      for (int tile = tile0; tile < tile1; ++tile) {
        f32x4 acc[RT] = {};
#pragma unroll 1
        for (int st = st0; st < st1; ++st) {
          u32x4 x[NT][4];
          split<T, NT>(raw_at(st), sc.up, x);
          const int b = st * 8 + grp * 2;
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const int f = tile * OUT + 16 * (GLU ? i % (RT / 2) : i) + col;
            const uint32_t r = (uint32_t)((f < a.width ? f : a.width - 1) + (GLU && i >= RT / 2 ? a.width : 0)) * nblk + b;
            u32x4 c;
            uint32_t s8 = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool in = b + h < nblk;
              const u32x2 w = __builtin_bit_cast(
                  u32x2, __builtin_amdgcn_raw_buffer_load_b64(codes, in ? (r + h) * 8 : kPastEnd, 0, 0));
              c[2 * h] = w[0];
              c[2 * h + 1] = w[1];
              s8 |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(scales, in ? r + h : kPastEnd, 0, 0) << (8 * h);
            }
            u32x4 d[4];
            decode(c, s8, d);
            acc[i] = multiply<NT>(d, x, acc[i]);
          }
        }
        finish<GLU, RT>(a, part[buf], acc, sc.down, tile, mt0, np, so, lds.list);
        buf ^= 1;
      }
    }
    lds_barrier();  // the list is rewritten next
  }
}

// One place of a wave's ring: a span (256 values of K, 16 blocks) of 32 weight
// rows. Codes as four loads of 8 rows of 128 bytes, the eight 16-byte pieces of
// row c in the order piece ^ (c / 2 % 8), so that 16 rows at one piece meet 16
// different banks. Scales as one load of 16 bytes a row, or, where rows of
// scales are not aligned, five aligned words a row.
struct Place {
  u32x4 codes[4][64];
  uint32_t scales[256];
};

// S: spans of a wave. EVEN: K % 256 == 0. A tile is two 16-row tiles (W13: 16
// gate rows and their up rows; W2: 32 rows), 16 pairs one pass over them.
template <typename T, int NT, bool GLU, int S, bool EVEN>
__global__ __launch_bounds__(kThreads, 2) void k_moe_stream(Product a) {
  constexpr int R = 3;                        // places of the ring
  constexpr int LOADS = EVEN ? 5 : 7;         // of a span
  constexpr int OUT = GLU ? 16 : 32;          // outputs of a tile
  __shared__ RouteLds lds;
  __shared__ float part[2][kWaves][2][256];
  __shared__ Place ring[R][kWaves];
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63;
  const int col = lane & 15, grp = lane >> 4;
  Route route;
  route.init(a.ids, a.pairs, a.E, lds);
  const int tiles = (a.width + OUT - 1) / OUT;
  const int64_t units = (int64_t)route.slots * tiles;
  int u = uniform((int)(units * blockIdx.x / gridDim.x));
  const int u1 = uniform((int)(units * (blockIdx.x + 1) / gridDim.x));
  const int nblk = a.K / 16;
  const int pitch = nblk * 8;  // bytes of a row's codes
  const int sp0 = a.span0 + a.spans * wave / kWaves, cnt = a.span0 + a.spans * (wave + 1) / kWaves - sp0;
  const int rows = GLU ? 2 * a.width : a.width;
  const int up = GLU ? a.width : 16;  // from a row of the first 16-row tile to the second's
  const brsrc_t act = buffer(a.in, (int64_t)(a.pairs / a.share) * a.K * (int)sizeof(T));
  // In a last span that is not whole, pieces past the end move back to the
  // row's last two blocks; the activations are zero where another lane has one.
  auto block_of = [&](int span, int piece) {
    const int b = span * 16 + piece * 2;
    return EVEN || b < nblk - 2 ? b : nblk - 2;
  };
  // this lane's share of the loads: codes, rows 8 b + lane / 8 of the tile's 32
  uint32_t coff[4], piece[2];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int c = (b & 1) * 8 + (lane >> 3);
    piece[b & 1] = (lane & 7) ^ (c >> 1 & 7);
    coff[b] = (uint32_t)(c + (b >> 1) * up) * pitch + (EVEN ? piece[b & 1] * 16 : 0);
  }
  // its own 16-byte piece of rows col and 16 + col at piece grp, and the same at piece 4 + grp
  const int mine0 = (col >> 3) * 64 + (col & 7) * 8 + (grp ^ (col >> 1 & 7)), mine1 = mine0 ^ 4;
  int buf = 0;
  while (u < u1) {
    const int at = u / tiles, tile0 = u - at * tiles;
    const int tile1 = tile0 + (u1 - u) < tiles ? tile0 + (u1 - u) : tiles;
    u += tile1 - tile0;
    const Slot slot = route.slot(at, lds);
    const int expert = uniform(slot.expert), mt0 = uniform(slot.part) * 16;
    const int64_t wrow = (int64_t)expert * rows;
    const rsrc_words codes = descriptor(a.codes + wrow * pitch, (uint32_t)rows * pitch);
    const uint8_t* sbase = a.scales + wrow * nblk;
    const uint32_t phase = EVEN ? 0u : (uint32_t)((uintptr_t)sbase & 15u);  // aligned words from an aligned base
    const rsrc_words scales = descriptor(sbase - phase, (phase + (uint32_t)rows * nblk + 3u) & ~3u);
    const float so = a.outer[expert];

    // the loads of span s of this wave for a tile, into one place of the ring; past the last tile, and for a span that
    // this wave has not, they are issued all the same (the waits count them) but past the buffers' ends
    auto fetch = [&](int tile, int s, int place) {
      const bool some = tile < tile1 && s < cnt;
      const bool both = GLU || tile * 32 + 16 < a.width;
      const int span = sp0 + s;
      const uint32_t at = lds_offset(&ring[place][wave]);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t v = EVEN ? coff[b] : coff[b] + (uint32_t)block_of(span, piece[b & 1]) * 8;
        load_to_lds<16>(codes, buffer_at(some, both || b < 2, v, (uint32_t)(tile * OUT) * pitch + (EVEN ? span * 128 : 0)),
                        at + b * 1024);
      }
      if constexpr (EVEN) {
        const int r = (lane & 15) + (lane >> 4 & 1) * up;
        load_to_lds<16>(scales, buffer_at(some, lane < 32 && (both || lane < 16), (uint32_t)r * nblk,
                                          (uint32_t)(tile * OUT) * nblk + span * 16), at + 4096);
      } else {
        const int w0 = block_of(span, 0);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const int i = j * 64 + lane, rr = i / 5;
          const uint32_t r = tile * OUT + (rr & 15) + (rr >> 4) * up;
          load_to_lds<4>(scales, buffer_at(some, i < 160 && (both || rr < 16), ((phase + r * nblk + w0) & ~3u) + i % 5 * 4, 0),
                         at + 4096 + j * 256);
        }
      }
    };

    // the ring starts before the activations are looked for
    wait_loads<0>();  // what was in flight to its places before
#pragma unroll
    for (int i = 0; i < R; ++i) fetch(tile0 + i / S, i % S, i);
    const int np = uniform(route.list_pairs(expert, a.pairs, lds));

    {
      // lanes past the last pair repeat one and are not stored
      const int pair = lds.list[mt0 + col < np ? mt0 + col : mt0];
      const uint32_t aoff = (uint32_t)(pair / a.share * a.K) * (uint32_t)sizeof(T);
      u32x4 x[S][2][NT][4];
      Scale sc;
      {
        // G spans at a time; where that is not all, they are read once for the maximum and once to be split
        constexpr int G = S > 2 ? S / 2 : S;
        Raw<T> raw[G][2];
        auto read = [&](int g) {
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int p = 0; p < 2; ++p)
              raw[s][p] = load_raw<T>(act, aoff, block_of(sp0 + g + s, 4 * p + grp),
                                      g + s < cnt ? (sp0 + g + s) * 16 + 2 * (4 * p + grp) : nblk, nblk);
          __builtin_amdgcn_sched_barrier(0);
        };
        float mx = 0.0f;
#pragma unroll
        for (int g = 0; g < S; g += G) {
          read(g);
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              mx = raw_max(raw[s][p], mx);
              __builtin_amdgcn_sched_barrier(0);
            }
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        sc = scale_for(mx);
#pragma unroll
        for (int g = 0; g < S; g += G) {
          if (G < S) read(g);
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              split<T, NT>(raw[s][p], sc.up, x[g + s][p]);
              __builtin_amdgcn_sched_barrier(0);
            }
        }
      }
      int place = 0;
#pragma unroll 1
      for (int tile = tile0; tile < tile1; ++tile) {
        f32x4 acc[2] = {};
#pragma unroll
        for (int s = 0; s < S; ++s) {
          wait_loads<(R - 1) * LOADS>();
          if (s < cnt) {
            const Place& pl = ring[place][wave];
            u32x4 c[2][2];
            uint32_t s8[2][2];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                c[p][i] = (&pl.codes[0][0])[i * 128 + (p ? mine1 : mine0)];
                if constexpr (EVEN) {
                  s8[p][i] = reinterpret_cast<const uint16_t*>(pl.scales)[(i * 16 + col) * 8 + 4 * p + grp];
                } else {
                  const int w0 = block_of(sp0 + s, 0);
                  const uint32_t r = tile * OUT + col + i * up;
                  const uint8_t* q = reinterpret_cast<const uint8_t*>(pl.scales) + (i * 16 + col) * 20 +
                                     ((phase + r * nblk + w0) & 3u) + (block_of(sp0 + s, 4 * p + grp) - w0);
                  s8[p][i] = (uint32_t)q[0] | (uint32_t)q[1] << 8;
                }
              }
            wait_lds();  // the place may be filled again
            fetch(tile + (s + R) / S, (s + R) % S, place);
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                u32x4 d[4];
                decode(c[p][i], s8[p][i], d);
                acc[i] = multiply<NT>(d, x[s][p], acc[i]);
              }
          } else {
            fetch(tile + (s + R) / S, (s + R) % S, place);
          }
          place = place == R - 1 ? 0 : place + 1;
          __builtin_amdgcn_sched_barrier(0);
        }
        finish<GLU, 2>(a, part[buf], acc, sc.down, tile, mt0, np, so, lds.list);
        buf ^= 1;
      }
    }
    lds_barrier();  // the list is rewritten next
  }
}

// ---------------------------------------------------------------- few pairs
// W2 and the weighted sum in one launch where all pairs fit the 16 columns of a
// matrix instruction (one token with its 8 experts, two with theirs): every
// pair's activations lie in a column, each expert's weights are multiplied by
// all of them, and a column keeps the sums of its own expert. A workgroup owns
// 16 outputs of every token and streams those rows of all experts that occur,
// so a token's experts meet in it, in slot order, and nothing is left to another
// launch. A wave has one or two spans of K, its activations stay in registers;
// where K has fewer spans than there are waves, groups of waves take the
// experts in turn. One token of 4096 x 1536, top 8: 14.6 us against 14 for W2 and 4
// for the sum; 10 of them are latency (28 MB take 5).
struct SmallPlace {  // a span of 16 weight rows; as Place
  u32x4 codes[2][64];
  uint32_t scales[128];
};

template <typename T, int S, bool EVEN>
__global__ __launch_bounds__(kThreads, 2) void k_moe_last(Product a, const float* __restrict__ weights,
                                                         T* __restrict__ y) {
  constexpr int NT = 2, R = 6;
  constexpr int LOADS = EVEN ? 3 : 4;  // of a span
  __shared__ RouteLds lds;
  __shared__ float part[2][kWaves][256];
  __shared__ float val[256], wlds[16];
  __shared__ SmallPlace ring[R][kWaves];
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63;
  const int col = lane & 15, grp = lane >> 4;
  const int tiles = a.width / 16;
  const int tile0 = uniform((int)((int64_t)tiles * blockIdx.x / gridDim.x));
  const int tile1 = uniform((int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x));
  if (tile0 == tile1) return;
  const int nblk = a.K / 16;
  const int pitch = nblk * 8;
  const int spans = (nblk + 15) / 16;
  const int nw = spans < kWaves ? spans : kWaves, groups = kWaves / nw;
  const int gi = uniform(wave / nw), wi = wave - gi * nw;
  const int sp0 = uniform(spans * wi / nw), cnt = uniform(spans * (wi + 1) / nw) - sp0;
  auto block_of = [&](int span, int piece) {
    const int b = span * 16 + piece * 2;
    return EVEN || b < nblk - 2 ? b : nblk - 2;
  };
  // the activations, which wait for no id
  Raw<float> raw[S][2];
  {
    const brsrc_t act = buffer(a.in, (int64_t)a.pairs * a.K * 4);
    const uint32_t aoff = (uint32_t)((col < a.pairs ? col : 0) * a.K) * 4u;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        raw[s][p] = load_raw<float>(act, aoff, block_of(sp0 + s, 4 * p + grp),
                                    s < cnt ? (sp0 + s) * 16 + 2 * (4 * p + grp) : nblk, nblk);
    __builtin_amdgcn_sched_barrier(0);
  }
  Route route;
  route.init(a.ids, a.pairs, a.E, lds);
  // the bits of `first` that this wave's group takes, from one to the next
  auto skip = [](uint64_t m, int n) {
    for (int i = 0; i < n; ++i) m &= m - 1;  // (0 stays 0)
    return m;
  };
  const uint64_t start = gi < groups ? skip(route.first, gi) : 0;
  auto expert_of = [&](uint64_t rem) { return __builtin_amdgcn_readlane(route.id[0], __ffsll((unsigned long long)rem) - 1); };
  uint32_t coff[2], piece[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int c = b * 8 + (lane >> 3);
    piece[b] = (lane & 7) ^ (c >> 1 & 7);
    coff[b] = (uint32_t)c * pitch + (EVEN ? piece[b] * 16 : 0);
  }
  const int mine0 = (col >> 3) * 64 + (col & 7) * 8 + (grp ^ (col >> 1 & 7)), mine1 = mine0 ^ 4;

  // where the weights of this lane's pair begin (scalar products for every span took longer than the span)
  const uint64_t e64 = (uint64_t)(route.id[0] < 0 ? 0 : route.id[0]);
  const uint64_t cbase = (uint64_t)a.codes + e64 * (uint64_t)((uint32_t)a.width * pitch);
  const uint64_t sbase = (uint64_t)a.scales + e64 * (uint64_t)((uint32_t)a.width * nblk);
  const uint32_t clo = (uint32_t)cbase, chi = (uint32_t)(cbase >> 32) & 0xFFFFu;
  const uint32_t slo = (uint32_t)sbase, shi = (uint32_t)(sbase >> 32) & 0xFFFFu;
  // the next span to be asked for
  uint64_t nrem = start;
  int ntile = tile0, ns = 0;
  auto fetch = [&](int place) {  // past the last tile: issued all the same (the waits count them), past the end
    const bool some = ntile < tile1;
    const int src = __ffsll((unsigned long long)nrem) - 1, span = sp0 + ns;
    const uint32_t row0 = (uint32_t)ntile * 16;
    const rsrc_words codes = {(uint32_t)__builtin_amdgcn_readlane((int)clo, src),
                              (uint32_t)__builtin_amdgcn_readlane((int)chi, src), (uint32_t)a.width * pitch, 0x00020000u};
    const uint32_t slow = (uint32_t)__builtin_amdgcn_readlane((int)slo, src), phase = EVEN ? 0u : slow & 3u;
    const rsrc_words scales = {slow - phase, (uint32_t)__builtin_amdgcn_readlane((int)shi, src),
                               (phase + (uint32_t)a.width * nblk + 3u) & ~3u, 0x00020000u};
    const uint32_t at = lds_offset(&ring[place][wave]);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t v = EVEN ? coff[b] : coff[b] + (uint32_t)block_of(span, piece[b]) * 8;
      load_to_lds<16>(codes, buffer_at(some, true, v, row0 * pitch + (EVEN ? span * 128 : 0)), at + b * 1024);
    }
    if constexpr (EVEN) {
      load_to_lds<4>(scales, buffer_at(some, true, (uint32_t)(lane >> 2) * nblk + (lane & 3) * 4, row0 * nblk + span * 16),
                     at + 2048);
    } else {
      const int w0 = block_of(span, 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = j * 64 + lane;
        load_to_lds<4>(scales, buffer_at(some, i < 80, ((phase + (row0 + i / 5) * nblk + w0) & ~3u) + i % 5 * 4, 0),
                       at + 2048 + j * 256);
      }
    }
    if (++ns == cnt) {
      ns = 0;
      nrem = skip(nrem, groups);
      if (!nrem) nrem = start, ++ntile;
    }
  };
  if (start) {
#pragma unroll
    for (int i = 0; i < R; ++i) fetch(i);
  }

  // this lane's column, and this thread's output in the tile: row 4 (t / 64) + t % 4 of pair t / 4 % 16
  const int mine = __shfl(route.id[0], col, 64);  // -1 past the last pair
  const int tp = t >> 2 & 15, te = __shfl(route.id[0], tp, 64);
  float so = te >= 0 ? a.outer[te] : 0.0f;
  if (t < 16) wlds[t] = route.id[0] >= 0 ? weights[t] : 0.0f;
  u32x4 x[S][2][NT][4];
  Scale sc;
  {
    float mx = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int p = 0; p < 2; ++p) mx = raw_max(raw[s][p], mx);
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    sc = scale_for(mx);
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int p = 0; p < 2; ++p) split<float, NT>(raw[s][p], sc.up, x[s][p]);
  }
  asm volatile("" : "+v"(so));  // waited for here, not in the stream

  int place = 0, buf = 0;
#pragma unroll 1
  for (int tile = tile0; tile < tile1; ++tile) {
    f32x4 total = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (uint64_t rem = start; rem; rem = skip(rem, groups)) {
      const int expert = expert_of(rem);
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (s < cnt) {
          wait_loads<(R - 1) * LOADS>();
          const SmallPlace& pl = ring[place][wave];
          u32x4 c[2];
          uint32_t s8[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            c[p] = (&pl.codes[0][0])[p ? mine1 : mine0];
            if constexpr (EVEN) {
              s8[p] = reinterpret_cast<const uint16_t*>(pl.scales)[col * 8 + 4 * p + grp];
            } else {
              const int w0 = block_of(sp0 + s, 0);
              const uint32_t at = (uint32_t)(uintptr_t)(a.scales + ((int64_t)expert * a.width + tile * 16 + col) * nblk + w0);
              const uint8_t* q = reinterpret_cast<const uint8_t*>(pl.scales) + col * 20 + (at & 3u) +
                                 (block_of(sp0 + s, 4 * p + grp) - w0);
              s8[p] = (uint32_t)q[0] | (uint32_t)q[1] << 8;
            }
          }
          wait_lds();  // the place may be filled again
          fetch(place);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            u32x4 d[4];
            decode(c[p], s8[p], d);
            acc = multiply<NT>(d, x[s][p], acc);
          }
          place = place == R - 1 ? 0 : place + 1;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) total[i] = mine == expert ? acc[i] : total[i];
    }
    *reinterpret_cast<f32x4*>(&part[buf][wave][lane * 4]) = total * sc.down;
    lds_barrier();
    if (wave < 4) {
      float v = part[buf][0][t];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += part[buf][w][t];
      val[t] = v * so;
      wait_lds();  // the pairs of a row lie in one wave
      if (tp < a.pairs && tp % a.k == 0) {
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j) sum += wlds[tp + j] * val[t + 4 * j];
        const int64_t o = (int64_t)(tp / a.k) * a.width + tile * 16 + (t >> 6) * 4 + (t & 3);
        if constexpr (sizeof(T) == 4) y[o] = sum;
        else y[o] = (T)(pack_bf16(sum, 0.0f) & 0xFFFFu);
      }
    }
    buf ^= 1;
  }
}

// h[p, f] = silu(gate) * up from the parts' sums [parts, pairs, 2 F] of W13.
// (Rows of pairs without an expert hold anything, and are read by nobody.)
__global__ __launch_bounds__(256) void k_moe_act(const float* __restrict__ raw, int64_t pairs, int F, int parts,
                                                 float* __restrict__ h) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= pairs * F) return;
  const float* at = raw + id / F * 2 * F + id % F;
  float g = 0.0f, u = 0.0f;
  for (int c = 0; c < parts; ++c) g += at[c * pairs * 2 * F], u += at[c * pairs * 2 * F + F];
  h[id] = g / (1.0f + expf(-g)) * u;
}

// y[t, n..n+3] = weighted sum over the token's valid pairs, in slot order, of
// the parts' sums [parts, tokens k, H].
template <typename T>
__global__ __launch_bounds__(256) void k_moe_sum(const float* __restrict__ z, const int32_t* __restrict__ ids,
                                                 const float* __restrict__ weights, int tokens, int k, int E, int H,
                                                 int parts, T* __restrict__ y) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = H / 4;
  if (id >= (int64_t)tokens * per) return;
  const int t = (int)(id / per), n = (int)(id % per) * 4;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* zt = z + (int64_t)t * k * H + n;
  for (int j0 = 0; j0 < k; j0 += 8) {  // eight rows' loads at once; an invalid pair's row holds anything
    f32x4 v[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int q = j0 + j < k ? j0 + j : k - 1;
      const int e = ids[t * k + q];
      w[j] = weights[t * k + q];
      v[j] = *reinterpret_cast<const f32x4*>(zt + (int64_t)q * H);
      for (int c = 1; c < parts; ++c)
        v[j] += *reinterpret_cast<const f32x4*>(zt + ((int64_t)c * tokens * k + q) * H);
      if (j0 + j >= k || e < 0 || e >= E) v[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, w[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s += w[j] * v[j];
  }
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<f32x4*>(y + (int64_t)t * H + n) = s;
  } else {
    *reinterpret_cast<u32x2*>(y + (int64_t)t * H + n) = (u32x2){pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
  }
}

// Registers hold up to 128 words of activations: 32 for each span of a wave
// (eight waves to K) and term. Longer K goes in parts, each a product of its
// own, whose sums meet in k_moe_act and k_moe_sum (16 tokens, 2 of 4 experts of
// 10240 x 10240: 210 us, where reading the activations again for every tile
// took 465; 2 of 8 experts of 4096 x 14336 195 and 289 us).
int parts_of(int64_t K, int NT) { return (int)(((K + 255) / 256 * NT + 31) / 32); }

template <typename T, int NT, bool GLU, int S>
void launch_stream(const Product& a, hipStream_t s) {
  const dim3 grid((unsigned)bsqh::device_cus()), block(kThreads);
  if (a.K % 256 == 0) hipLaunchKernelGGL((k_moe_stream<T, NT, GLU, S, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_moe_stream<T, NT, GLU, S, false>), grid, block, 0, s, a);
}
template <typename T, int NT, bool GLU>
void launch_product(Product a, hipStream_t s) {
  a.span0 = 0;
  a.spans = (a.K + 255) / 256;
  if (a.K < 32)
    hipLaunchKernelGGL((k_moe_any<T, NT, GLU, 2>), dim3((unsigned)bsqh::device_cus()), dim3(kThreads), 0, s, a);
  else if (a.spans * NT <= 16) launch_stream<T, NT, GLU, 2 / NT>(a, s);
  else launch_stream<T, NT, GLU, 4 / NT>(a, s);
}
// The part sums [parts, pairs, width], from a.out on.
template <typename T, int NT>
void launch_parts(Product a, int parts, hipStream_t s) {
  const int spans = (a.K + 255) / 256;
  for (int c = 0; c < parts; ++c) {
    a.span0 = (int)((int64_t)spans * c / parts);
    a.spans = (int)((int64_t)spans * (c + 1) / parts) - a.span0;
    launch_stream<T, NT, false, 4 / NT>(a, s);
    a.out += (int64_t)a.pairs * a.width;
  }
}

// W2 and the sum: one launch for up to 16 pairs with K in registers (two spans
// a wave). Whole layers this way and with the sum apart: one token of 4096 x 1536,
// top 8, 31 and 34 us, two 49 and 52 us; two of 7168 x 2048 90 and 92 us.
template <typename T>
bool launch_last(const Product& a, const float* weights, T* y, hipStream_t s) {
  const int spans = (a.K / 16 + 15) / 16;
  if (a.pairs > 16 || a.K < 32 || spans > 2 * kWaves) return false;
  const int tiles = a.width / 16, cus = bsqh::device_cus();
  const dim3 grid((unsigned)(tiles < cus ? tiles : cus)), block(kThreads);
  if (a.K % 256 == 0) {
    if (spans <= kWaves) hipLaunchKernelGGL((k_moe_last<T, 1, true>), grid, block, 0, s, a, weights, y);
    else hipLaunchKernelGGL((k_moe_last<T, 2, true>), grid, block, 0, s, a, weights, y);
  } else {
    if (spans <= kWaves) hipLaunchKernelGGL((k_moe_last<T, 1, false>), grid, block, 0, s, a, weights, y);
    else hipLaunchKernelGGL((k_moe_last<T, 2, false>), grid, block, 0, s, a, weights, y);
  }
  return true;
}

template <typename T, int NT>
void launch_layer(const T* x, int64_t tokens, int64_t H, int64_t F, int64_t E, int64_t k, const int32_t* ids,
                  const float* weights, const uint8_t* w13c, const uint8_t* w13s, const float* w13o,
                  const uint8_t* w2c, const uint8_t* w2s, const float* w2o, T* out, float* ws, hipStream_t s) {
  const int pairs = (int)(tokens * k);
  const int n13 = parts_of(H, NT), n2 = parts_of(F, 2);
  float* h = ws;                          // [pairs, F]
  float* z = h + tokens * k * F;          // [n2, pairs, H]
  float* raw = z + n2 * tokens * k * H;   // [n13, pairs, 2 F] where n13 > 1
  const int w = (int)F, w2 = 2 * (int)F;
  if (n13 == 1) {
    launch_product<T, NT, true>({x, ids, pairs, (int)k, (int)E, (int)H, w, (int)k, w13c, w13s, w13o, h, 0, 0}, s);
  } else {
    launch_parts<T, NT>({x, ids, pairs, (int)k, (int)E, (int)H, w2, (int)k, w13c, w13s, w13o, raw, 0, 0}, n13, s);
    hipLaunchKernelGGL(k_moe_act, dim3((unsigned)((tokens * k * F + 255) / 256)), dim3(256), 0, s,
                       static_cast<const float*>(raw), tokens * k, (int)F, n13, h);
  }
  const Product down{h, ids, pairs, (int)k, (int)E, (int)F, (int)H, 1, w2c, w2s, w2o, z, 0, 0};
  if (launch_last<T>(down, weights, out, s)) return;
  if (n2 == 1) launch_product<float, 2, false>(down, s);
  else launch_parts<float, 2>(down, n2, s);
  hipLaunchKernelGGL((k_moe_sum<T>), dim3((unsigned)((tokens * (H / 4) + 255) / 256)), dim3(256), 0, s,
                     static_cast<const float*>(z), ids, weights, (int)tokens, (int)k, (int)E, (int)H, n2, out);
}

bool shape_ok(int64_t tokens, int64_t hidden, int64_t ffn, int64_t E, int64_t k) {
  return tokens >= 0 && hidden >= 16 && hidden % 16 == 0 && hidden <= 32768 && ffn >= 16 && ffn % 16 == 0 &&
         ffn <= 32768 && E >= 1 && E <= kMaxExperts && k >= 1 && k <= 64 && tokens <= kMaxPairs / k;
}

}  // namespace

extern "C" size_t bsq_moe_few_nvfp4_workspace(int64_t tokens, int64_t hidden, int64_t ffn, int64_t E, int64_t k) {
  if (!shape_ok(tokens, hidden, ffn, E, k)) return 0;
  const int n13 = parts_of(hidden, 2), n2 = parts_of(ffn, 2);  // of float32 x; of bfloat16 n13 may be less
  return (size_t)(tokens * k) * (size_t)(ffn + n2 * hidden + (n13 > 1 ? n13 * 2 * ffn : 0)) * 4;
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
  float* sums = static_cast<float*>(ws);
  if (dtype == BSQ_BF16)
    launch_layer<uint16_t, 1>(static_cast<const uint16_t*>(x), tokens, hidden, ffn, E, k, topk_ids, topk_weights,
                              w13_codes, w13_scales, w13_outer, w2_codes, w2_scales, w2_outer,
                              static_cast<uint16_t*>(out), sums, s);
  else
    launch_layer<float, 2>(static_cast<const float*>(x), tokens, hidden, ffn, E, k, topk_ids, topk_weights, w13_codes,
                           w13_scales, w13_outer, w2_codes, w2_scales, w2_outer, static_cast<float*>(out), sums, s);
  return bsqh::launch_status();
}
