// Log probability of a given token, entropy and the largest alternatives of
// rows of logits, and the gradient of the first two.
//
// Row x, m its maximum, z_i = x_i - m, S = sum e^z_i, p_i = e^z_i / S:
//   log p_t = z_t - log S
//   H = -sum p_i log p_i = log S - (sum z_i e^z_i) / S
// Gradient of g log p_t + h H:
//   d_i = g ([i = t] - p_i) - h p_i (log p_i + H)
//
// One pass over the logits with a running maximum: sums relative to m become
// sums relative to m' > m by s' = s f, u' = (u + (m - m') s) f, f = e^(m - m').
// Bound by memory for many rows (4096 x 131072 bf16: 220 to 250 us, 4.3 to 4.9
// TB/s; the gradient, which reads and writes, 350 to 360, 6 TB/s); few rows are cut
// into parts for as many workgroups, whose sums meet in a second launch (one row of
// 100003 float32, top 20: 3.8 and 11.7 us, 64 of 131072 bf16, top 5: 10.4 and 8.4).
//
// Alternatives: the pass also leaves the maximum of every block of 64
// neighbours. Ordered by value, then by lower index, the k best elements lie
// in the k best blocks (each block ahead of an element's own holds an element
// ahead of it), and the same holds for any groups of blocks or elements. So the
// second launch ranks groups, keeps the best ones' members, and so on to blocks,
// then in the same way to elements, each rank by counting the larger ones.
#include <math.h>

#include "bsq_device.h"
#include "bsq_internal.h"
#include "bsq_rows.h"

using namespace bsqd;

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kBlock = 64;      // elements of a block
constexpr int kMaxTop = 64;
constexpr int kMaxParts = 256;  // of a row
constexpr float kInf = __builtin_inff();
constexpr float kFar = -200.0f;  // e^kFar is 0 in float32

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// Key of a logit: unsigned order = float order, both zeros alike, 0 = masked.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -kInf)) return 0u;  // -inf or NaN
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
// Larger: a larger value, or the same at a lower index. 0: masked.
__device__ __forceinline__ u64 ranked(uint32_t key, uint32_t index) {
  return key ? (u64)key << 32 | (uint32_t)~index : 0ull;
}

// e^z for z <= 0: z is rounded once more by the factor, 1.5 |z| 2^-24 and the
// instruction's unit in the last place; terms that count have a small |z|.
__device__ __forceinline__ float exp_fast(float z) { return __builtin_amdgcn_exp2f(z * 1.44269504088896340736f); }

// A row in 16-byte pieces at aligned addresses: the first and the last may
// hold elements of the neighbours.
template <typename T>
struct Row {
  static constexpr int E = 16 / (int)sizeof(T);  // elements of a piece
  const T* base;  // of piece 0
  int lead, V;    // elements before the row in piece 0; the row's
  __device__ __forceinline__ Row(const T* x, int64_t row, int v) : V(v) {
    const T* at = x + row * v;
    lead = (int)(((uintptr_t)at & 15) / sizeof(T));
    base = at - lead;
  }
  __device__ __forceinline__ int pieces() const { return (lead + V + E - 1) / E; }
  __device__ __forceinline__ bool whole(int p) const { return p * E >= lead && (p + 1) * E <= lead + V; }
  // elements of piece p, `other` where they are not the row's
  __device__ __forceinline__ void load(int p, float (&v)[E], float other) const {
    if (whole(p)) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(base + p * E);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
        else v[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int at = p * E + i;
        v[i] = at >= lead && at < lead + V ? load1(base + at) : other;
      }
    }
  }
};

struct Sums {
  float m, s, u;  // maximum, sum e^(x - m), sum (x - m) e^(x - m)
  __device__ __forceinline__ void raise(float to) {  // to >= m
    if (to > m) {
      const float d = __builtin_elementwise_maximum(m - to, kFar), f = exp_fast(d);
      u = (u + d * s) * f;
      s *= f;
      m = to;
    }
  }
};
// Lane exchanges within a wave's 16-lane rows, then across them.
template <typename Op>
__device__ __forceinline__ float wave_all(float v, Op op) {
  v = op(v, dpp<0xB1>(v));   // lane ^ 1
  v = op(v, dpp<0x4E>(v));   // lane ^ 2
  v = op(v, dpp<0x141>(v));  // 7 - lane of 8: halves of equal quads
  v = op(v, dpp<0x140>(v));  // 15 - lane of 16
  v = op(v, __shfl_xor(v, 16, 64));
  return op(v, __shfl_xor(v, 32, 64));
}
// Sums of a workgroup of `waves` waves, in every thread.
__device__ __forceinline__ Sums joined(Sums a, Sums* lds, int waves) {
  a.raise(wave_all(a.m, [](float p, float q) { return fmaxf(p, q); }));
  a.s = wave_all(a.s, [](float p, float q) { return p + q; });
  a.u = wave_all(a.u, [](float p, float q) { return p + q; });
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
  __syncthreads();
  float m = -kInf;
  for (int w = 0; w < waves; ++w) m = fmaxf(m, lds[w].m);
  Sums t = {m, 0.0f, 0.0f};
  for (int w = 0; w < waves; ++w) {
    Sums o = lds[w];
    o.raise(m);
    t.s += o.s;
    t.u += o.u;
  }
  return t;
}

struct Out {
  float *logprobs, *entropy, *stats, *top_logprobs;
  int32_t* top_ids;
};

// What a row's sums give; one thread. stats: m and log S (0 and 0 for a row without an unmasked logit).
template <typename T>
__device__ __forceinline__ void finish(const T* __restrict__ x, const int64_t* __restrict__ targets, int64_t row, int V,
                                       const Sums& a, const Out& o) {
  const bool none = !(a.m > -kInf) && a.s == 0.0f;
  const float m = none ? 0.0f : a.m, log_s = none ? 0.0f : logf(a.s);
  o.stats[2 * row] = m;
  o.stats[2 * row + 1] = log_s;
  o.entropy[row] = none ? 0.0f : log_s - a.u / a.s;
  const int64_t t = targets[row];
  o.logprobs[row] = t >= 0 && t < V ? load1(x + row * V + t) - m - log_s : 0.0f;
}

// Part `part` of a row's pieces. TOP: blocks' maxima are left, too.
template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void k_token_stats(const T* __restrict__ x, const int64_t* __restrict__ targets,
                                                         int64_t row0, int V, int parts, int per, Sums* __restrict__ sums,
                                                         uint32_t* __restrict__ maxima, int blocks, Out out) {
  constexpr int E = Row<T>::E, LB = kBlock / E;  // lanes of a block
  constexpr int U = 4;                           // pieces of a thread on their way
  __shared__ Sums lds[kWaves];
  const int64_t row = row0 + blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  const Row<T> r(x, row, V);
  const int pieces = r.pieces();
  const int first = part * per, last = first + per < pieces ? first + per : pieces;
  Sums a = {-kInf, 0.0f, 0.0f};
  for (int p0 = first; p0 < last; p0 += U * kThreads) {
    float v[U][E];
    float most = -kInf;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int p = p0 + i * kThreads + (int)threadIdx.x;
      if (p < last) {
        r.load(p, v[i], -kInf);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = -kInf;
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float big = v[i][0];
#pragma unroll
      for (int e = 1; e < E; ++e) big = fmaxf(big, v[i][e]);
      most = fmaxf(most, big);
      if constexpr (TOP) {
        big = fmaxf(big, dpp<0xB1>(big));
        big = fmaxf(big, dpp<0x4E>(big));
        big = fmaxf(big, dpp<0x141>(big));
        if constexpr (LB == 16) big = fmaxf(big, dpp<0x140>(big));
        const int p = p0 + i * kThreads + (int)threadIdx.x;
        if (p < last && p % LB == 0) maxima[row * blocks + p / LB] = key_of(big);
      }
    }
    a.raise(fmaxf(a.m, most));
    const float m = a.m > -kInf ? a.m : 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float z = __builtin_elementwise_maximum(v[i][e] - m, kFar);  // NaN stays
        const float f = exp_fast(z);
        a.s += f;
        a.u = __builtin_fmaf(z, f, a.u);
      }
  }
  a = joined(a, lds, kWaves);
  if (threadIdx.x == 0) {
    if (sums) sums[row * parts + part] = a;
    else finish(x, targets, row, V, a, out);
  }
}

// The alternatives' kernel: 1024 threads a row, eight to a key. A ranking of n
// keys is n^2 comparisons, so that lists of more than 128 are narrowed by groups
// first (rankings of up to 512 made it 13 us for one row of 100003, top 20).
constexpr int kJThreads = 1024, kJWaves = kJThreads / 64;
constexpr int kMost = 128;          // keys that are ranked at a time
constexpr int kLarge = 1 << 20, kSmall = 1 << 18;  // vocabularies
constexpr int blocks_of(int V) { return V / kBlock + 1; }  // at most: the row may begin within a block
// groups of a row's blocks, so that the best ones' blocks fit the list
constexpr int first_of(int V) { return V > kSmall ? 512 : kMost; }

using bsqd::dpp;
template <int CTRL>
__device__ __forceinline__ u64 dpp(u64 v) {
  return (u64)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xF, 0xF, false) << 32 |
         (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xF, 0xF, false);
}

// keys[0, n) are distinct but for zeros. Each key's rank is the number of larger
// ones, of which its eight threads count an eighth each; `take` gets (index,
// rank) of those that are not zero and among the `top` first, in each of them.
template <typename Take>
__device__ __forceinline__ void ranks(const u64* keys, int n, int top, Take take) {
  const int t = threadIdx.x;
  for (int i = t >> 3; i < n; i += kJThreads / 8) {
    const u64 mine = keys[i];
    int rank = 0;
#pragma unroll 8
    for (int j = t & 7; j < n; j += 8) rank += keys[j] > mine;
    rank += __builtin_amdgcn_update_dpp(0, rank, 0xB1, 0xF, 0xF, false);
    rank += __builtin_amdgcn_update_dpp(0, rank, 0x4E, 0xF, 0xF, false);
    rank += __builtin_amdgcn_update_dpp(0, rank, 0x141, 0xF, 0xF, false);
    if (mine && rank < top) take(i, rank);
  }
}
// The `top` largest of keys[0, n) to best[], largest first, 0 where none is left.
__device__ __forceinline__ void best_of(const u64* keys, int n, int top, u64* best) {
  const int t = threadIdx.x;
  if (t < top) best[t] = 0ull;
  __syncthreads();
  ranks(keys, n, top, [&](int i, int rank) {
    if ((t & 7) == 0) best[rank] = keys[i];
  });
  __syncthreads();
}
// Groups of `size` of n items, key(i) distinct but for zeros: the items of the
// best `top` groups to out[0, top * size).
template <typename Key>
__device__ __forceinline__ void narrow(Key key, int n, int size, int top, u64* most, u64* out) {
  const int t = threadIdx.x, groups = (n + size - 1) / size;
  for (int g = t >> 3; g < groups; g += kJThreads / 8) {
    u64 m = 0;
    for (int i = g * size + (t & 7); i < (g + 1) * size && i < n; i += 8) {
      const u64 k = key(i);
      m = k > m ? k : m;
    }
    u64 o = dpp<0xB1>(m);
    m = o > m ? o : m;
    o = dpp<0x4E>(m);
    m = o > m ? o : m;
    o = dpp<0x141>(m);
    m = o > m ? o : m;
    if ((t & 7) == 0) most[g] = m;
  }
  for (int i = t; i < top * size; i += kJThreads) out[i] = 0ull;
  __syncthreads();
  ranks(most, groups, top, [&](int g, int rank) {
    for (int i = t & 7; i < size; i += 8)
      if (g * size + i < n) out[rank * size + i] = key(g * size + i);
  });
  __syncthreads();
}
// The same of a list, until few enough are left: list[0, n) and `other` are overwritten.
__device__ __forceinline__ void best_of_list(u64* list, u64* other, int n, int top, u64* most, u64* best) {
  while (n > kMost) {  // ends: 64 ceil(n / 128) < n
    const int size = (n + kMost - 1) / kMost;
    const u64* from = list;
    narrow([&](int i) { return from[i]; }, n, size, top, most, other);
    n = top * size;
    u64* was = list;
    list = other;
    other = was;
  }
  best_of(list, n, top, best);
}

// A workgroup a row: the parts' sums, then the alternatives. MAXV: the largest
// vocabulary.
template <typename T, int MAXV>
__global__ __launch_bounds__(kJThreads) void k_token_join(const T* __restrict__ x, const int64_t* __restrict__ targets,
                                                         int64_t row0, int V, int parts, const Sums* __restrict__ sums,
                                                         const uint32_t* __restrict__ maxima, int pitch, int top,
                                                         Out out) {
  constexpr int E = Row<T>::E, PB = kBlock / E;  // elements of a piece, pieces of a block
  constexpr int kBlocks = blocks_of(MAXV);
  constexpr int kFirst = first_of(MAXV);
  constexpr int kList = kMaxTop * ((kBlocks + kFirst - 1) / kFirst);  // blocks of the best groups
  constexpr int kElements = kMaxTop * kBlock;                        // of the best blocks
  constexpr int kOther = kMaxTop * ((kList + kMost - 1) / kMost);    // what a list narrows to
  static_assert(kMaxTop * ((kElements + kMost - 1) / kMost) <= kList, "the elements of the best groups fit the list");
  __shared__ Sums lds[kJWaves];
  __shared__ union {
    uint32_t maxima[kBlocks];
    u64 element[kElements];
  } a_;
  __shared__ u64 list[kList], other[kOther], most[kFirst], best[kMaxTop];
  const int t = threadIdx.x;
  const int64_t row = row0 + blockIdx.x;
  const Row<T> r(x, row, V);
  const int blocks = (r.pieces() + PB - 1) / PB;
  Sums a = {-kInf, 0.0f, 0.0f};
  if (t < parts) a = sums[row * parts + t];
  if (top) {
    const uint32_t* mx = maxima + row * pitch;
    for (int b = t; b < blocks; b += kJThreads) a_.maxima[b] = mx[b];
  }
  a = joined(a, lds, kJWaves);  // its barrier is the maxima's, too
  if (t == 0) finish(x, targets, row, V, a, out);
  if (top == 0) return;
  const int size = (blocks + kFirst - 1) / kFirst;
  narrow([&](int b) { return ranked(a_.maxima[b], (uint32_t)b); }, blocks, size, top, most, list);
  best_of_list(list, other, top * size, top, most, best);
  // the elements of the best blocks
  for (int i = t; i < top * PB; i += kJThreads) {
    const u64 g = best[i / PB];
    const int p = (int)(uint32_t)~(uint32_t)g * PB + i % PB;
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = -kInf;
    if (g) r.load(p, v, -kInf);
#pragma unroll
    for (int e = 0; e < E; ++e) a_.element[i * E + e] = ranked(key_of(v[e]), (uint32_t)(p * E + e));
  }
  __syncthreads();
  const int of = (top * kBlock + kMost - 1) / kMost;
  narrow([&](int i) { return a_.element[i]; }, top * kBlock, of, top, most, list);
  best_of_list(list, other, top * of, top, most, best);
  if (t < top) {
    const bool none = !(a.m > -kInf) && a.s == 0.0f;
    const u64 k = best[t];
    const float m = none ? 0.0f : a.m, log_s = none ? 0.0f : logf(a.s);
    out.top_logprobs[row * top + t] = k ? of_key((uint32_t)(k >> 32)) - m - log_s : -kInf;
    out.top_ids[row * top + t] = k ? (int)(uint32_t)~(uint32_t)k - r.lead : -1;
  }
}

// Segments of a row; each thread U pieces.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_token_grad(const float* __restrict__ dlogprobs,
                                                        const float* __restrict__ dentropy, const T* __restrict__ x,
                                                        const int64_t* __restrict__ targets,
                                                        const float* __restrict__ stats,
                                                        const float* __restrict__ entropy, int64_t row0, int V,
                                                        int segments, T* __restrict__ dlogits) {
  constexpr int E = Row<T>::E, U = 4;
  const int64_t row = row0 + blockIdx.x / segments;
  const int seg = (int)(blockIdx.x % segments);
  const Row<T> r(x, row, V), d(dlogits, row, V);
  const int pieces = r.pieces();
  const int64_t t = targets[row];
  const bool aim = t >= 0 && t < V;
  const float g = aim && dlogprobs ? dlogprobs[row] : 0.0f, h = dentropy ? dentropy[row] : 0.0f;
  const float m = stats[2 * row], log_s = stats[2 * row + 1], c = g + h * entropy[row];
  const int target = aim ? (int)t + r.lead : -1;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int p = (seg * U + i) * kThreads + (int)threadIdx.x;
    if (p >= pieces) break;
    float v[E], o[E];
    r.load(p, v, -kInf);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float lp = __builtin_elementwise_maximum(v[e] - m - log_s, kFar);
      o[e] = -exp_fast(lp) * __builtin_fmaf(h, lp, c);
    }
    if (target / E == p && target >= 0) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (target % E == e && v[e] > -kInf) o[e] += g;
    }
    T* to = const_cast<T*>(d.base) + p * E;
    if (r.whole(p)) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
          w[e] = __float_as_uint(o[e]);
        } else {
          w[e] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)o[2 * e]) |
                 (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)o[2 * e + 1]) << 16;
        }
      }
      *reinterpret_cast<u32x4*>(to) = w;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (p * E + e >= r.lead && p * E + e < r.lead + V) store1(to + e, o[e]);
    }
  }
}

// Parts of a row: as many as give a thousand workgroups, of 512 pieces at least.
struct Cut {
  int parts, per, blocks;  // pieces of a part; blocks of a row
  size_t sums, maxima;     // bytes of the workspace
};
Cut cut_of(int64_t T, int64_t V, int64_t top, int64_t size) {
  const int64_t E = 16 / size, pieces = (V + 2 * (E - 1)) / E;  // at most: the lead differs from row to row
  int64_t parts = (1024 + T - 1) / T, most = (pieces + 511) / 512;
  if (parts > most) parts = most;
  if (parts > kMaxParts) parts = kMaxParts;
  const int64_t LB = kBlock / E;
  Cut c;
  c.per = (int)(((pieces + parts - 1) / parts + LB - 1) / LB * LB);
  c.parts = (int)parts;
  c.blocks = (int)((pieces + LB - 1) / LB);
  const bool join = c.parts > 1 || top > 0;
  c.sums = join ? ((size_t)T * parts * sizeof(Sums) + 15) / 16 * 16 : 0;
  c.maxima = top > 0 ? (size_t)T * c.blocks * 4 : 0;
  return c;
}

template <typename T>
int run_logprobs(const void* logits, const int64_t* targets, int64_t tokens, int64_t V, int64_t top, const Out& out,
                 uint8_t* ws, hipStream_t s) {
  const T* x = static_cast<const T*>(logits);
  const Cut c = cut_of(tokens, V, top, sizeof(T));
  Sums* sums = c.sums ? reinterpret_cast<Sums*>(ws) : nullptr;
  uint32_t* maxima = reinterpret_cast<uint32_t*>(ws + c.sums);
  const int64_t most = bsqh::max_blocks(kJThreads) / c.parts;
  for (int64_t r = 0; r < tokens; r += most) {
    const int64_t n = tokens - r < most ? tokens - r : most;
    if (top > 0)
      hipLaunchKernelGGL((k_token_stats<T, true>), dim3((unsigned)(n * c.parts)), dim3(kThreads), 0, s, x, targets, r,
                         (int)V, c.parts, c.per, sums, maxima, c.blocks, out);
    else
      hipLaunchKernelGGL((k_token_stats<T, false>), dim3((unsigned)(n * c.parts)), dim3(kThreads), 0, s, x, targets, r,
                         (int)V, c.parts, c.per, sums, maxima, c.blocks, out);
    if (sums && V <= kSmall)
      hipLaunchKernelGGL((k_token_join<T, kSmall>), dim3((unsigned)n), dim3(kJThreads), 0, s, x, targets, r, (int)V,
                         c.parts, sums, maxima, c.blocks, (int)top, out);
    else if (sums)
      hipLaunchKernelGGL((k_token_join<T, kLarge>), dim3((unsigned)n), dim3(kJThreads), 0, s, x, targets, r, (int)V,
                         c.parts, sums, maxima, c.blocks, (int)top, out);
  }
  return bsqh::launch_status();
}

template <typename T>
int run_backward(const float* dlogprobs, const float* dentropy, const void* logits, const int64_t* targets,
                 const float* stats, const float* entropy, int64_t tokens, int64_t V, void* dlogits, hipStream_t s) {
  const int64_t E = 16 / (int64_t)sizeof(T), pieces = (V + 2 * (E - 1)) / E;
  const int64_t segments = (pieces + 4 * kThreads - 1) / (4 * kThreads), most = bsqh::max_blocks(kThreads) / segments;
  for (int64_t r = 0; r < tokens; r += most) {
    const int64_t n = tokens - r < most ? tokens - r : most;
    hipLaunchKernelGGL((k_token_grad<T>), dim3((unsigned)(n * segments)), dim3(kThreads), 0, s, dlogprobs, dentropy,
                       static_cast<const T*>(logits), targets, stats, entropy, r, (int)V, (int)segments,
                       static_cast<T*>(dlogits));
  }
  return bsqh::launch_status();
}

bool shape_ok(int64_t tokens, int64_t V) {
  return tokens >= 0 && tokens < (int64_t)1 << 31 && V >= 1 && V <= kLarge;
}

}  // namespace

extern "C" size_t bsq_token_logprobs_workspace(int64_t tokens, int64_t V, int64_t top, int dtype) {
  if (tokens <= 0 || !shape_ok(tokens, V) || top < 0 || top > kMaxTop) return 0;
  const Cut c = cut_of(tokens, V, top, dtype == BSQ_F32 ? 4 : 2);
  return c.sums + c.maxima;
}

extern "C" int bsq_token_logprobs(const void* logits, int dtype, const int64_t* targets, int64_t tokens, int64_t V,
                                  int64_t top, float* logprobs, float* entropy, float* stats, float* top_logprobs,
                                  int32_t* top_ids, void* ws, size_t ws_bytes, bsq_stream_t stream) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(shape_ok(tokens, V) && top >= 0 && top <= kMaxTop && top <= V, BSQ_E_SHAPE);
  if (tokens == 0) return BSQ_OK;
  const size_t need = bsq_token_logprobs_workspace(tokens, V, top, dtype);
  BSQ_REQUIRE(logits && targets && logprobs && entropy && stats && (ws || need == 0) &&
                  (top == 0 || (top_logprobs && top_ids)),
              BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(logits) && bsqh::aligned16(ws) && ((uintptr_t)targets & 7) == 0 &&
                  (((uintptr_t)logprobs | (uintptr_t)entropy | (uintptr_t)stats) & 3) == 0 &&
                  (top == 0 || (((uintptr_t)top_logprobs | (uintptr_t)top_ids) & 3) == 0),
              BSQ_E_ALIGN);
  BSQ_REQUIRE(ws_bytes >= need, BSQ_E_WORKSPACE);
  const Out out = {logprobs, entropy, stats, top_logprobs, top_ids};
  uint8_t* b = static_cast<uint8_t*>(ws);
  hipStream_t s = bsqh::as_stream(stream);
  if (dtype == BSQ_F32) return run_logprobs<float>(logits, targets, tokens, V, top, out, b, s);
  return run_logprobs<uint16_t>(logits, targets, tokens, V, top, out, b, s);
}

extern "C" int bsq_token_logprobs_backward(const float* dlogprobs, const float* dentropy, const void* logits, int dtype,
                                           const int64_t* targets, const float* stats, const float* entropy,
                                           int64_t tokens, int64_t V, void* dlogits, bsq_stream_t stream) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(shape_ok(tokens, V), BSQ_E_SHAPE);
  if (tokens == 0) return BSQ_OK;
  BSQ_REQUIRE((dlogprobs || dentropy) && logits && targets && stats && entropy && dlogits, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(logits) && bsqh::aligned16(dlogits) && ((uintptr_t)targets & 7) == 0 &&
                  (((uintptr_t)dlogprobs | (uintptr_t)dentropy | (uintptr_t)stats | (uintptr_t)entropy) & 3) == 0,
              BSQ_E_ALIGN);
  hipStream_t s = bsqh::as_stream(stream);
  if (dtype == BSQ_F32)
    return run_backward<float>(dlogprobs, dentropy, logits, targets, stats, entropy, tokens, V, dlogits, s);
  return run_backward<uint16_t>(dlogprobs, dentropy, logits, targets, stats, entropy, tokens, V, dlogits, s);
}
