// Top-k expert selection over router logits, and its gradient.
//
// For a token with logits l_0 .. l_(E-1) the k largest are selected (ties to
// the lowest index; -inf and NaN are masked) and weighted by a softmax over
// the selected ones, or over all unmasked ones:
//   w_j = e^(l_j - m) / sum e^(l_i - m),  m the row's maximum.
// Gradient of sum_j g_j w_j with the selection held fixed:
//   over the selected:  dl_j = w_j (g_j - sum_s w_s g_s), 0 elsewhere;
//   over all:           dl_i = p_i ([i selected] g_i - sum_s w_s g_s).
//
// Bound by memory for many tokens (each logit read once, k pairs written) and
// by the launch for few. 16 lanes share a row up to 256 experts (four rows a
// wave; the row-wide maximum is then four DPP rotations inside a 16-lane row,
// no LDS), 64 lanes above that. A lane keeps its logits in registers as
// unsigned keys in the order of the floats. float32: each of the k rounds takes
// the row's largest key, then the lowest index that holds it. bf16: key and
// index share a word (a larger word is a larger logit or the same at a lower
// index), so a lane sorts its words once and a round is one row-wide maximum
// of the lanes' first words, whose owner moves on to its next. 65536 tokens, 128
// experts, top 8: 13.5 us in bf16, bound by the vector ALU (20 us by the
// float32 rounds); the whole call 16 us in float32, whose bytes take 6.
#include "bsq_device.h"
#include "bsq_internal.h"
#include "bsq_rows.h"

using namespace bsqd;

namespace {

constexpr int kThreads = 256;

// Key of a logit: unsigned order = float order, both zeros alike, 0 = masked.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -__builtin_inff())) return 0u;  // -inf or NaN
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// e^x by the hardware's base-2 exponential: x is rounded once more, so the
// result is off by 1.5 |x| 2^-24 and the instruction's unit in the last place.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// A bf16 logit's key above the complement of its index; 0 = masked.
__device__ __forceinline__ uint32_t word_of(float x, int index) {
  const uint32_t k = key_of(x) >> 16;  // exact: the lower half of a bf16's bits is 0 (or all ones, complemented)
  return k ? k << 16 | (uint32_t)(0xFFFF - index) : 0u;
}
__device__ __forceinline__ float of_word(uint32_t w) {
  const uint32_t k = w >> 16;
  return __uint_as_float((k & 0x8000u ? k ^ 0x8000u : ~k) << 16);
}
// Batcher's odd-even merge sort, largest first.
template <int V>
__device__ __forceinline__ void sort_words(uint32_t (&w)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (p * 2) == (i + j + k) / (p * 2)) {
            const uint32_t a = w[i + j], b = w[i + j + k];
            w[i + j] = a > b ? a : b;
            w[i + j + k] = a > b ? b : a;
          }
}

// KR: registers that hold a row's k results, lane j % L holding result j.
template <typename T, int L, int V, bool WHOLE, int KR>
__global__ __launch_bounds__(kThreads) void k_moe_gate(const T* __restrict__ logits, int64_t tokens, int E, int k,
                                                      int renorm, float* __restrict__ weights,
                                                      int32_t* __restrict__ ids) {
  const int sub = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool ok = t < tokens;  // lanes past the end run along on masked rows
  float x[V];
  load_logits<T, V, WHOLE>(logits + (ok ? t : 0) * E, sub * V, E, ok, x);
  float rv[KR];  // the selected logits, -inf where none was left
  int ri[KR];
#pragma unroll
  for (int q = 0; q < KR; ++q) rv[q] = -__builtin_inff(), ri[q] = -1;
  float m = 0.0f, total = 0.0f;
  if constexpr (sizeof(T) == 2) {
    uint32_t w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = word_of(x[i], sub * V + i);
    sort_words<V>(w);
    uint32_t best = row_max<L>(w[0]);
    if (best) m = of_word(best);
    for (int j = 0; j < k; ++j) {
      if (j) best = row_max<L>(w[0]);
      const bool own = w[0] == best;  // words are distinct while any is left
      const uint32_t move = own ? 0xFFFFFFFFu : 0u;  // by bits: as a choice of elements it became one of indexes
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) w[i] = __builtin_amdgcn_bitop3_b32(move, w[i + 1], w[i], 0xCA);
      w[V - 1] &= ~move;
#pragma unroll
      for (int q = 0; q < KR; ++q)
        if (j == q * L + sub && best) {
          rv[q] = of_word(best);
          ri[q] = 0xFFFF - (int)(best & 0xFFFFu);
        }
    }
  } else {
    uint32_t key[V];
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = key_of(x[i]);
      best = best > key[i] ? best : key[i];
    }
    best = row_max<L>(best);
    if (best) m = of_key(best);
    for (int j = 0; j < k; ++j) {
      if (j) {
        best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = best > key[i] ? best : key[i];
        best = row_max<L>(best);
      }
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)(sub * V + i) : at;
      at = row_min<L>(at);
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = at == (uint32_t)(sub * V + i) ? 0u : key[i];
#pragma unroll
      for (int q = 0; q < KR; ++q)
        if (j == q * L + sub && best) {
          rv[q] = of_key(best);
          ri[q] = (int)at;
        }
    }
  }
  if (!renorm) {
#pragma unroll
    for (int i = 0; i < V; ++i) total += x[i] > -__builtin_inff() ? exp_fast(x[i] - m) : 0.0f;  // NaN is masked too
  }
  float e[KR];
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    e[q] = ri[q] >= 0 ? exp_fast(rv[q] - m) : 0.0f;
    if (renorm) total += e[q];
  }
  total = row_sum<L>(total);
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    const int j = q * L + sub;
    if (ok && j < k) {
      weights[t * k + j] = e[q] * inv;
      ids[t * k + j] = ri[q];
    }
  }
}

// The row's k incoming gradients are spread over its E experts in LDS (zeros,
// then one write per selected expert); each lane then reads its own V. The
// lanes of a row belong to one wave, whose LDS operations stay in order.
template <typename T, int L, int V, bool WHOLE, int KR, bool RENORM>
__global__ __launch_bounds__(kThreads) void k_moe_gate_backward(const float* __restrict__ dweights,
                                                               const float* __restrict__ weights,
                                                               const int32_t* __restrict__ ids,
                                                               const T* __restrict__ logits, int64_t tokens, int E,
                                                               int k, T* __restrict__ dlogits) {
  __shared__ float spread[kThreads / L][L * V];
  const int sub = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool ok = t < tokens;
  float* mine = spread[threadIdx.x / L];
  float w[KR], g[KR];
  int id[KR];
  float inner = 0.0f;
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    const int j = q * L + sub;
    const bool in = ok && j < k;
    id[q] = in ? ids[t * k + j] : -1;
    if (id[q] >= E) id[q] = -1;
    w[q] = id[q] >= 0 ? weights[t * k + j] : 0.0f;
    g[q] = id[q] >= 0 ? dweights[t * k + j] : 0.0f;
    inner += w[q] * g[q];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) mine[sub * V + i] = 0.0f;
  inner = row_sum<L>(inner);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int q = 0; q < KR; ++q)
    if (id[q] >= 0) mine[id[q]] = RENORM ? w[q] * (g[q] - inner) : g[q];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = mine[sub * V + i];
  if constexpr (!RENORM) {
    float x[V];
    load_logits<T, V, WHOLE>(logits + (ok ? t : 0) * E, sub * V, E, ok, x);
    uint32_t best = 0, key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = key_of(x[i]);
      best = best > key[i] ? best : key[i];
    }
    best = row_max<L>(best);
    const float m = best ? of_key(best) : 0.0f;
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = key[i] ? exp_fast(x[i] - m) : 0.0f;
      total += x[i];
    }
    total = row_sum<L>(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = x[i] * inv * (d[i] - inner);
  }
  if (ok) store_grads<T, V, WHOLE>(dlogits + t * E, sub * V, E, d);
}

template <typename T, int L, int V, bool WHOLE>
void launch_gate_k(const T* logits, int64_t tokens, int E, int k, int renorm, float* weights, int32_t* ids,
                   hipStream_t s) {
  constexpr int64_t per = kThreads / L, most = bsqh::max_blocks(kThreads) * per;
  for (; tokens > 0; tokens -= most, logits += most * E, weights += most * k, ids += most * k) {
    const int64_t n = tokens < most ? tokens : most;
    const unsigned grid = (unsigned)((n + per - 1) / per);
    if (k <= L)
      hipLaunchKernelGGL((k_moe_gate<T, L, V, WHOLE, 1>), dim3(grid), dim3(kThreads), 0, s, logits, n, E, k, renorm,
                         weights, ids);
    else
      hipLaunchKernelGGL((k_moe_gate<T, L, V, WHOLE, 64 / L>), dim3(grid), dim3(kThreads), 0, s, logits, n, E, k,
                         renorm, weights, ids);
  }
}

template <typename T, int L, int V, bool WHOLE, int KR>
void launch_back_k(const float* dw, const float* w, const int32_t* ids, const T* logits, int64_t tokens, int E, int k,
                   int renorm, T* dlogits, hipStream_t s) {
  constexpr int64_t per = kThreads / L, most = bsqh::max_blocks(kThreads) * per;
  for (; tokens > 0; tokens -= most, dw += most * k, w += most * k, ids += most * k, dlogits += most * E) {
    const int64_t n = tokens < most ? tokens : most;
    const unsigned grid = (unsigned)((n + per - 1) / per);
    if (renorm)
      hipLaunchKernelGGL((k_moe_gate_backward<T, L, V, WHOLE, KR, true>), dim3(grid), dim3(kThreads), 0, s, dw, w, ids,
                         logits, n, E, k, dlogits);
    else
      hipLaunchKernelGGL((k_moe_gate_backward<T, L, V, WHOLE, KR, false>), dim3(grid), dim3(kThreads), 0, s, dw, w, ids,
                         logits, n, E, k, dlogits);
    if (logits) logits += most * E;  // not given where the weights are renormalized
  }
}
template <typename T, int L, int V, bool WHOLE>
void launch_back(const float* dw, const float* w, const int32_t* ids, const T* logits, int64_t tokens, int E, int k,
                 int renorm, T* dlogits, hipStream_t s) {
  if (k <= L) launch_back_k<T, L, V, WHOLE, 1>(dw, w, ids, logits, tokens, E, k, renorm, dlogits, s);
  else launch_back_k<T, L, V, WHOLE, 64 / L>(dw, w, ids, logits, tokens, E, k, renorm, dlogits, s);
}

bool shape_ok(int64_t tokens, int64_t E, int64_t k) {
  return tokens >= 0 && tokens < (int64_t)1 << 31 && E >= 1 && E <= 1024 && k >= 1 && k <= 64 && k <= E;
}

}  // namespace

extern "C" int bsq_moe_gate(const void* logits, int dtype, int64_t tokens, int64_t E, int64_t k, int renormalize,
                            float* weights, int32_t* topk_ids, bsq_stream_t stream) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(renormalize == 0 || renormalize == 1, BSQ_E_ENUM);
  BSQ_REQUIRE(shape_ok(tokens, E, k), BSQ_E_SHAPE);
  if (tokens == 0) return BSQ_OK;
  BSQ_REQUIRE(logits && weights && topk_ids, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(logits) && ((uintptr_t)weights & 3) == 0 && ((uintptr_t)topk_ids & 3) == 0, BSQ_E_ALIGN);
  hipStream_t s = bsqh::as_stream(stream);
  if (dtype == BSQ_F32) {
    BSQ_GATE_SHAPES(launch_gate_k, float, static_cast<const float*>(logits), tokens, (int)E, (int)k, renormalize,
                    weights, topk_ids, s);
  } else {
    BSQ_GATE_SHAPES(launch_gate_k, uint16_t, static_cast<const uint16_t*>(logits), tokens, (int)E, (int)k,
                    renormalize, weights, topk_ids, s);
  }
  return bsqh::launch_status();
}

extern "C" int bsq_moe_gate_backward(const float* dweights, const float* weights, const int32_t* topk_ids,
                                     const void* logits, int dtype, int64_t tokens, int64_t E, int64_t k,
                                     int renormalize, void* dlogits, bsq_stream_t stream) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE(renormalize == 0 || renormalize == 1, BSQ_E_ENUM);
  BSQ_REQUIRE(shape_ok(tokens, E, k), BSQ_E_SHAPE);
  if (tokens == 0) return BSQ_OK;
  BSQ_REQUIRE(dweights && weights && topk_ids && dlogits && (logits || renormalize), BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(logits) && bsqh::aligned16(dlogits) && ((uintptr_t)weights & 3) == 0 &&
                  ((uintptr_t)dweights & 3) == 0 && ((uintptr_t)topk_ids & 3) == 0,
              BSQ_E_ALIGN);
  hipStream_t s = bsqh::as_stream(stream);
  if (dtype == BSQ_F32) {
    BSQ_GATE_SHAPES(launch_back, float, dweights, weights, topk_ids, static_cast<const float*>(logits), tokens,
                    (int)E, (int)k, renormalize, static_cast<float*>(dlogits), s);
  } else {
    BSQ_GATE_SHAPES(launch_back, uint16_t, dweights, weights, topk_ids, static_cast<const uint16_t*>(logits), tokens,
                    (int)E, (int)k, renormalize, static_cast<uint16_t*>(dlogits), s);
  }
  return bsqh::launch_status();
}
