// Rows of router logits: several lanes of a wave share a row (gfx950).
#pragma once
#include "bsq_device.h"

namespace bsqd {

// Rotation of v by N lanes inside each row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}

// All-reduce over the L lanes (16 or 64) that share a row. Every lane gets the
// same bits: each step combines the same two partial results in all lanes that
// hold them, and the operations commute.
template <int L, typename Op>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, Op op) {
  v = op(v, ror16<8>(v));
  v = op(v, ror16<4>(v));
  v = op(v, ror16<2>(v));
  v = op(v, ror16<1>(v));
  if constexpr (L == 64) {
    v = op(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    v = op(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return row_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  return row_reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  return __uint_as_float(row_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// Lane exchange by the control word CTRL within 16 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// The V logits of a lane: experts [e0, e0 + V). WHOLE: the row has exactly
// L * V experts, so the lane's values are whole and aligned to their size.
template <typename T, int V, bool WHOLE>
__device__ __forceinline__ void load_logits(const T* __restrict__ row, int e0, int E, bool ok, float (&x)[V]) {
  if constexpr (WHOLE && V * sizeof(T) >= 4) {
    constexpr int W = V * sizeof(T) / 4;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
    if (ok) __builtin_memcpy(w, __builtin_assume_aligned(row + e0, W * 4 > 16 ? 16 : W * 4), W * 4);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
      else x[i] = (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = ok && e0 + i < E ? load1(row + e0 + i) : -__builtin_inff();
  }
}

template <typename T, int V, bool WHOLE>
__device__ __forceinline__ void store_grads(T* __restrict__ row, int e0, int E, const float (&d)[V]) {
  uint32_t w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) w[i] = __float_as_uint(d[i]);
  if constexpr (sizeof(T) == 4) {
    if constexpr (WHOLE) {
      __builtin_memcpy(__builtin_assume_aligned(row + e0, V * 4 > 16 ? 16 : V * 4), w, V * 4);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < E) row[e0 + i] = (T)d[i];
    }
  } else {
    uint16_t h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = __builtin_bit_cast(uint16_t, (__bf16)d[i]);
    if constexpr (WHOLE) {
      __builtin_memcpy(__builtin_assume_aligned(row + e0, V * 2 > 16 ? 16 : V * 2), h, V * 2);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < E) row[e0 + i] = h[i];
    }
  }
}

}  // namespace bsqd

// L lanes of V experts each: 16 lanes to a row up to 256 experts, 64 above.
// Rows of exactly 64, 128 or 256 experts take whole-vector loads and stores
// (their rows are then aligned, since the base pointers are).
#define BSQ_GATE_SHAPES(FN, T, ...)                                    \
  if (E == 64) FN<T, 16, 4, true>(__VA_ARGS__);                        \
  else if (E == 128) FN<T, 16, 8, true>(__VA_ARGS__);                  \
  else if (E == 256) FN<T, 16, 16, true>(__VA_ARGS__);                 \
  else if (E <= 32) FN<T, 16, 2, false>(__VA_ARGS__);                  \
  else if (E < 64) FN<T, 16, 4, false>(__VA_ARGS__);                   \
  else if (E < 128) FN<T, 16, 8, false>(__VA_ARGS__);                  \
  else if (E < 256) FN<T, 16, 16, false>(__VA_ARGS__);                 \
  else FN<T, 64, 16, false>(__VA_ARGS__)
