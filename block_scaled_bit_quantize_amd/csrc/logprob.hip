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
// Bound by memory for many rows; few rows are cut into parts for as many
// workgroups, whose sums meet in a second launch.
//
// Alternatives: the pass also leaves the maximum of every block of 64
// neighbours. Ordered by value, then by lower index, the k best elements lie
// in the k best blocks (each block ahead of an element's own holds an element
// ahead of it), and the same holds for groups of blocks. So the second launch
// ranks groups, blocks of the best groups, eighths of the best blocks and their
// elements, each rank by counting the larger ones among a few hundred.
#include <math.h>

#include "bsq_device.h"
#include "bsq_internal.h"

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

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
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
  __device__ __forceinline__ void add(Sums o) {
    const float to = fmaxf(m, o.m);
    raise(to);
    o.raise(to);
    s += o.s;
    u += o.u;
  }
};
__device__ __forceinline__ Sums shuffled(const Sums& a, int o) {
  return {__shfl_xor(a.m, o, 64), __shfl_xor(a.s, o, 64), __shfl_xor(a.u, o, 64)};
}
// Sums of a workgroup, in every thread.
__device__ __forceinline__ Sums joined(Sums a, Sums* lds) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) a.add(shuffled(a, o));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
  __syncthreads();
  a = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) a.add(lds[w]);
  return a;
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
#pragma unroll
        for (int o = 1; o < LB; o *= 2) big = fmaxf(big, __shfl_xor(big, o, 64));
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
  a = joined(a, lds);
  if (threadIdx.x == 0) {
    if (sums) sums[row * parts + part] = a;
    else finish(x, targets, row, V, a, out);
  }
}

// How many of keys[0, n) are larger than each of the thread's.
template <int N>
__device__ __forceinline__ void rank_of(const u64* keys, int n, const u64 (&mine)[N], int (&rank)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) rank[i] = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const u64 k = keys[j];
#pragma unroll
    for (int i = 0; i < N; ++i) rank[i] += k > mine[i];
  }
}

// keys[0, n) (distinct but for zeros, n <= 512): the `top` largest to best[], largest first, 0 where none is left.
__device__ __forceinline__ void best_of(const u64* keys, int n, int top, u64* best) {
  const int t = threadIdx.x;
  u64 mine[2];
  int rank[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) mine[i] = t + i * kThreads < n ? keys[t + i * kThreads] : 0ull;
  if (t < kMaxTop) best[t] = 0ull;
  __syncthreads();
  rank_of<2>(keys, n, mine, rank);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (mine[i] && rank[i] < top) best[rank[i]] = mine[i];
  __syncthreads();
}

// A workgroup a row: the parts' sums, then the alternatives.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_token_join(const T* __restrict__ x, const int64_t* __restrict__ targets,
                                                        int64_t row0, int V, int parts, const Sums* __restrict__ sums,
                                                        const uint32_t* __restrict__ maxima, int pitch, int top,
                                                        Out out) {
  constexpr int E = Row<T>::E;
  __shared__ Sums lds[kWaves];
  __shared__ u64 keys[kMaxTop * 33], best[kMaxTop];
  const int t = threadIdx.x;
  const int64_t row = row0 + blockIdx.x;
  Sums a = {-kInf, 0.0f, 0.0f};
  if (t < parts) a = sums[row * parts + t];
  a = joined(a, lds);
  if (t == 0) finish(x, targets, row, V, a, out);
  if (top == 0) return;
  const uint32_t* mx = maxima + row * pitch;
  const Row<T> r(x, row, V);
  const int blocks = (r.pieces() + kBlock / E - 1) / (kBlock / E);
  // groups of `size` blocks; with up to 64 groups kept, `keys` holds their blocks
  const int groups = blocks > 16 * kThreads ? 2 * kThreads : kThreads, size = (blocks + groups - 1) / groups;
  for (int g = t; g < groups; g += kThreads) {
    u64 big = 0;
    for (int b = g * size; b < (g + 1) * size && b < blocks; ++b) {
      const u64 k = ranked(mx[b], (uint32_t)b);
      big = k > big ? k : big;
    }
    keys[g] = big;
  }
  __syncthreads();
  best_of(keys, groups, top, best);
  // the blocks of the best groups; more than 512 are grouped once more
  int n = top * size;
  for (int i = t; i < n; i += kThreads) {
    const u64 g = best[i / size];
    const int b = (int)((uint32_t)~(uint32_t)g) / size * size + i % size;
    keys[i] = g && b < blocks ? ranked(mx[b], (uint32_t)b) : 0ull;
  }
  __syncthreads();
  if (n > 512) {
    const int per = (n + kThreads - 1) / kThreads;  // 9 at most: 64 groups of 33 blocks
    u64 mine[9];
    u64 most = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      mine[i] = i < per && t * per + i < n ? keys[t * per + i] : 0ull;
      most = mine[i] > most ? mine[i] : most;
    }
    __syncthreads();
    keys[t] = most;
    __syncthreads();
    const u64 one[1] = {most};
    int rank[1];
    rank_of<1>(keys, kThreads, one, rank);
    __syncthreads();
    n = top * per;
    for (int i = t; i < n; i += kThreads) keys[i] = 0ull;
    __syncthreads();
    if (most && rank[0] < top) {
#pragma unroll
      for (int i = 0; i < 9; ++i)
        if (i < per) keys[rank[0] * per + i] = mine[i];
    }
    __syncthreads();
  }
  if (n > 512) {  // up to 64 groups of 9: in two parts, whose best meet
    u64* half = keys + 1024;
    best_of(keys, 512, top, half);
    best_of(keys + 512, n - 512, top, half + kMaxTop);
    best_of(half, 2 * kMaxTop, top, best);
  } else {
    best_of(keys, n, top, best);
  }
  // eighths of the best blocks, then the elements of the best eighths
  constexpr int EI = kBlock / 8, PE = EI / E;  // elements and pieces of an eighth
  n = top * 8;
  __syncthreads();
  for (int i = t; i < n; i += kThreads) {
    const u64 g = best[i / 8];
    u64 k = 0;
    if (g) {
      const int p0 = (int)(uint32_t)~(uint32_t)g * (kBlock / E) + i % 8 * PE;
      for (int q = 0; q < PE; ++q) {
        float v[E];
        r.load(p0 + q, v, -kInf);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const u64 o = ranked(key_of(v[e]), (uint32_t)((p0 + q) * E + e));
          k = o > k ? o : k;
        }
      }
    }
    keys[i] = k;
  }
  __syncthreads();
  best_of(keys, n, top, best);
  for (int i = t; i < n; i += kThreads) {
    const u64 g = best[i / 8];
    u64 k = 0;
    if (g) {
      const int at = (int)((uint32_t)~(uint32_t)g) / EI * EI + i % 8;
      if (at >= r.lead && at < r.lead + V) k = ranked(key_of(load1(r.base + at)), (uint32_t)at);
    }
    keys[i] = k;
  }
  static_assert(EI == 8, "an eighth's elements");
  __syncthreads();
  best_of(keys, n, top, best);
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
  const int64_t most = bsqh::max_blocks(kThreads) / c.parts;
  for (int64_t r = 0; r < tokens; r += most) {
    const int64_t n = tokens - r < most ? tokens - r : most;
    if (top > 0)
      hipLaunchKernelGGL((k_token_stats<T, true>), dim3((unsigned)(n * c.parts)), dim3(kThreads), 0, s, x, targets, r,
                         (int)V, c.parts, c.per, sums, maxima, c.blocks, out);
    else
      hipLaunchKernelGGL((k_token_stats<T, false>), dim3((unsigned)(n * c.parts)), dim3(kThreads), 0, s, x, targets, r,
                         (int)V, c.parts, c.per, sums, maxima, c.blocks, out);
    if (sums)
      hipLaunchKernelGGL((k_token_join<T>), dim3((unsigned)n), dim3(kThreads), 0, s, x, targets, r, (int)V, c.parts,
                         sums, maxima, c.blocks, (int)top, out);
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
  return tokens >= 0 && tokens < (int64_t)1 << 31 && V >= 1 && V <= (int64_t)1 << 20;
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
