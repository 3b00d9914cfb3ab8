// Expert selection by scores, a balancing bias and groups of experts, and the
// gradient of its weights.
//
// A token's logits l_i give scores s_i: sigmoid(l_i), or the softmax over the
// unmasked ones. The keys c_i = s_i + b_i (bias b, which the weights do not
// see) choose: a group of experts is worth the sum of its one or two largest
// keys, the best group_k groups stay, and of their experts the k with the
// largest keys are selected. Ties go to the lowest index at both steps. The
// order is that of keys evaluated in float64. Weights:
//   w_j = scale s_j, or scale s_j / sum of the selected scores (renormalized).
// Gradient of sum g_j w_j, the selection held fixed, with h = sum g_j w_j:
//   sigmoid:  dl_j = w_j (g_j - [renormalized] h / scale) (1 - s_j), 0 where not selected
//   softmax:  renormalized  dl_j = w_j (g_j - h / scale), 0 where not selected
//             else          dl_i = s_i (scale [i selected] g_i - h)
//
// How the order can be that of float64 keys at the speed of float32: keys are
// made in float32 with a bound on their error, the selection is made by them,
// and the groups at the cut, the selected keys next to each other, and the least
// of them with all that are not selected are then looked at (all: a bound goes
// with the score, so a key that a bias takes back from a large score may reach
// past one that is ahead of it). Where two are nearer than their bounds and are not
// keys of equal logits and biases (a true tie), the row is ambiguous (1 row in about
// 500 of random logits). Where all that may be selected has a place in its lanes,
// those are put in order by float64 keys; else, and where it is groups that are
// near or tie, its wave selects from the start in float64 with all 64 lanes (with
// that for all ambiguous rows 38.6 us in place of 32: 65536 tokens, 128 experts,
// bf16; for rows of equal logits in 8 groups, all of which go there, 201 us).
//
// 8 lanes share a row up to 128 experts, 16 up to 256 and 64 above; a lane holds
// V neighbouring experts in registers. Bound by vector instructions: k rounds
// of a search of V keys and an exchange over L lanes (65536 x 128, top 8 of 4 of 8
// groups: 28 us among others of its kind, 30 to 33 in a trace, for bytes of 4; 16381
// x 60, top 6 of 3 of 5: 14.8; one token 5.2).
#include <math.h>

#include "bsq_device.h"
#include "bsq_internal.h"
#include "bsq_rows.h"

using namespace bsqd;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxGroups = 64;
// A value that has been taken out of the selection: below every key, and a
// number whatever its low word holds.
constexpr uint32_t kGone = 0xFFEFFFFFu;
constexpr float kInf = __builtin_inff();
constexpr float kBig = __FLT_MAX__ * (1.0f - 0x1p-20f);  // below an infinite key, and below a sum past float32

struct Choice {
  int E, k, groups, size, group_k, group_top;  // groups 1: no restriction
  int lanes;                                   // lanes that share a group, 0: through LDS
  int over_size;                               // e / size = e * over_size >> 20, for e < 1024 and size <= 512
  bool softmax, renorm;
  float scale;
};

// e^x for x <= 0: the product's rounding is carried along, so that what is left
// is the exponential instruction's error and a rounding (2^-22 relative).
__device__ __forceinline__ float exp_neg(float x) {
  x = fmaxf(x, -256.0f);
  const float t = x * 1.44269504088896340736f;
  const float r = __builtin_fmaf(x, 1.44269504088896340736f, -t) + x * 1.92596299112661746887e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * 0.693147180559945309417f, e);
}
__device__ __forceinline__ float sigmoid32(float x) {
  const float e = exp_neg(-fabsf(x));
  return (x >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e);
}

// Error bound of a float32 key c = s + b: the sigmoid is off by less than
// 2^-21 s (in 2^-24: the exponential 3, the sum and the product 1 each, the
// reciprocal 2; over all floats 4.3 were measured);
// a softmax score by less than 2^-16 s (its sum by 2^-19, |l - m| 2^-24 from the
// difference, up to 64 of it: beyond, s is below 2^-92 and the last term covers it);
// the sum with the bias by 2^-24 |c|, and the bound's own sum or difference with c
// by as much. Exponentials that flush to zero are below 2^-110.
__device__ __forceinline__ float key_bound(float s, float c, bool softmax) {
  return s * (softmax ? 0x1p-16f : 0x1p-21f) + fabsf(c) * 0x1.8p-23f + 0x1p-90f;
}

// Key above its index in one float64: a larger number is a larger key, or the
// same key at a lower index. The key's low 29 bits are free.
__device__ __forceinline__ double with_index(float c, int index) {
  if (!(c > -kInf)) return __hiloint2double((int)kGone, 0);
  c = fminf(fmaxf(c + 0.0f, -__FLT_MAX__), __FLT_MAX__);
  const uint64_t b = __double_as_longlong((double)c);
  return __longlong_as_double((long long)(b | (uint32_t)(c < 0.0f ? index : 1023 - index)));
}
__device__ __forceinline__ bool is_gone(double d) { return (uint32_t)__double2hiint(d) == kGone; }
__device__ __forceinline__ int index_of(double d) {
  const int low = __double2loint(d) & 1023;
  return __double2hiint(d) < 0 ? low : 1023 - low;
}

using bsqd::dpp;
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, false),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, false));
}
// Lane exchanges: ^1, ^2, ^3 within 4 lanes, 7 - lane within 8 (^7), 15 - lane within 16 (^15), rotations within 16.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor3 = 0x1B, kXor7 = 0x141, kXor15 = 0x140;
constexpr int ror(int n) { return 0x120 + n; }

// All-reduce over the L lanes (8, 16 or 64) that share a row; each step combines
// the same two results in all lanes that hold them.
template <int L, typename V, typename Op>
__device__ __forceinline__ V over_row(V v, Op op) {
  v = op(v, dpp<kXor1>(v));
  v = op(v, dpp<kXor2>(v));
  v = op(v, dpp<kXor7>(v));
  if constexpr (L > 8) v = op(v, dpp<kXor15>(v));
  if constexpr (L > 16) {
    v = op(v, __shfl_xor(v, 16, 64));
    v = op(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ double row_max64(double v) {
  return over_row<L>(v, [](double a, double b) { return fmax(a, b); });
}
template <int L>
__device__ __forceinline__ float row_maxf(float v) {
  return over_row<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float row_addf(float v) {
  return over_row<L>(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// A group's best keys and largest score, over `lanes` aligned lanes of 16.
struct Top {
  float a, b, s;  // largest key, second, largest score
};
template <int CTRL>
__device__ __forceinline__ void merge(Top& t) {
  const float a = dpp<CTRL>(t.a), b = dpp<CTRL>(t.b);
  t.b = fmaxf(fminf(t.a, a), fmaxf(t.b, b));
  t.a = fmaxf(t.a, a);
  t.s = fmaxf(t.s, dpp<CTRL>(t.s));
}
// [low, high] that holds the group's worth.
__device__ __forceinline__ void worth(const Top& t, int group_top, bool softmax, float& low, float& high) {
  if (!(t.a > -kInf)) {
    low = high = -kInf;
    return;
  }
  const bool two = group_top == 2 && t.b > -kInf;
  const float w = two ? t.a + t.b : t.a;
  if (!(fabsf(w) <= kBig)) {  // an infinite bias, or a sum past float32
    low = w > 0.0f ? kBig : -kInf;
    high = w > 0.0f ? kInf : -kBig;
    return;
  }
  float tol = key_bound(t.s, t.a, softmax);
  if (two) tol += key_bound(t.s, t.b, softmax) + fabsf(w) * 0x1p-23f;
  low = w - tol;
  high = w + tol;
}

// What a wave needs of LDS: the rows' float32 keys, then what they are at most, by
// lanes (in registers, 124 in place of 98, 65536 x 128 took 31 us and not 29), or
// one row's keys in float64; a word for each of their groups (or the groups' worth
// in float64), the groups kept.
template <int L, int V>
struct WaveLds {
  union {
    float key[64 / L][L * V];
    float high[V][64];
    double key64[L * V];
  };
  union {
    float bound[64 / L][kMaxGroups][2];
    double worth64[kMaxGroups];
  };
  uint32_t keep[kMaxGroups];
  int pick[128];
};

// The key of a logit that is not masked, in float64.
__device__ __noinline__ double key64(double x, float bias, bool softmax, double m, double total) {
  return (softmax ? exp(x - m) / total : 1.0 / (1.0 + exp(-x))) + (double)bias;
}

// One row in float64 by all lanes of a wave: the selected indexes go to lds.pick (-1: none left).
template <typename T, int L, int V>
__device__ __noinline__ void select64(const T* __restrict__ row, const float* __restrict__ bias, const Choice c,
                                      WaveLds<L, V>& lds) {
  const int lane = threadIdx.x & 63;
  double total = 1.0, m = 0.0;
  if (c.softmax) {
    float top = -kInf;
    for (int e = lane; e < c.E; e += 64) {
      const float x = load1(row + e);
      if (x > top) top = x;
    }
    top = row_maxf<64>(top);
    m = top > -kInf ? (double)top : 0.0;
    total = 0.0;
    for (int e = lane; e < c.E; e += 64) {
      const float x = load1(row + e);
      if (x > -kInf) total += exp((double)x - m);
    }
    for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
  }
  for (int e = lane; e < c.E; e += 64) {
    const double x = load1(row + e), key = key64(x, bias ? bias[e] : 0.0f, c.softmax, m, total);
    lds.key64[e] = x > -(double)kInf && key > -(double)kInf ? key : -(double)kInf;
  }
  wave_fence();
  if (c.groups > 1) {
    double w = -(double)kInf;
    if (lane < c.groups) {
      double a = -(double)kInf, b = a;
      for (int e = lane * c.size; e < (lane + 1) * c.size; ++e) {
        const double v = lds.key64[e];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
      w = c.group_top == 2 && b > -(double)kInf ? a + b : a;
      lds.worth64[lane] = w;
    }
    wave_fence();
    if (lane < c.groups) {
      int rank = 0;
      for (int g = 0; g < c.groups; ++g) {
        const double o = lds.worth64[g];
        rank += o > w || (o == w && g < lane);
      }
      lds.keep[lane] = rank < c.group_k;
    }
    wave_fence();
    for (int e = lane; e < c.E; e += 64)
      if (!lds.keep[e / c.size]) lds.key64[e] = -(double)kInf;
    wave_fence();
  }
  for (int j = 0; j < c.k; ++j) {
    double best = -(double)kInf;
    int at = 0x7FFFFFFF;
    for (int e = lane; e < c.E; e += 64) {
      const double v = lds.key64[e];
      if (v > best) best = v, at = e;
    }
    for (int o = 32; o > 0; o >>= 1) {
      const double v = __shfl_xor(best, o, 64);
      const int i = __shfl_xor(at, o, 64);
      if (v > best || (v == best && i < at)) best = v, at = i;
    }
    const bool any = best > -(double)kInf;
    if (lane == 0) lds.pick[j] = any ? at : -1;
    if (any && (at & 63) == lane) lds.key64[at] = -(double)kInf;
    wave_fence();
  }
}

// KR: registers that hold a row's results, lane j % L holding result j; more than
// k of them, for those that may be selected in place of others.
template <typename T, int L, int V, bool WHOLE, int KR>
__global__ __launch_bounds__(kThreads) void k_group_gate(const T* __restrict__ logits, const float* __restrict__ bias,
                                                        int64_t tokens, Choice c, float* __restrict__ weights,
                                                        int32_t* __restrict__ ids) {
  __shared__ WaveLds<L, V> shared[kWaves];
  WaveLds<L, V>& lds = shared[threadIdx.x >> 6];
  const int lane = threadIdx.x & 63, sub = lane % L, mine = lane / L;  // row of the wave
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool ok = t < tokens;  // lanes past the end run along on masked rows
  const T* row = logits + (ok ? t : 0) * c.E;
  const int e0 = sub * V;
  float x[V], b[V], s[V];
  load_logits<T, V, WHOLE>(row, e0, c.E, ok, x);
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = 0.0f;
  if (bias) {
    if constexpr (WHOLE) {
      __builtin_memcpy(b, bias + e0, sizeof(b));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = e0 + i < c.E ? bias[e0 + i] : 0.0f;
    }
  }
  float m = 0.0f, inv = 1.0f;
  if (c.softmax) {
    float top = -kInf, total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);  // drops NaN
    top = row_maxf<L>(top);
    m = top > -kInf ? top : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = x[i] > -kInf ? exp_neg(x[i] - m) : 0.0f;
      total += s[i];
    }
    total = row_addf<L>(total);
    inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sigmoid32(x[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {  // the key
    const float v = s[i] + b[i];
    b[i] = x[i] > -kInf && v > -kInf ? v : -kInf;  // no NaN, of a logit or a bias
  }
  bool unsure = false;
  if (c.groups > 1) {
    Top g = {-kInf, -kInf, 0.0f};
    if (c.lanes) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        g.b = fmaxf(g.b, fminf(g.a, b[i]));
        g.a = fmaxf(g.a, b[i]);
        g.s = fmaxf(g.s, s[i]);
      }
      if (c.lanes > 1) merge<kXor1>(g);
      if (c.lanes > 2) merge<kXor2>(g);
      if (c.lanes > 4) merge<kXor7>(g);
      float low, high;
      worth(g, c.group_top, c.softmax, low, high);
      int over = 0, near = 0;  // groups that are surely better, that may be
      auto meet = [&](float other_low, float other_high) {
        over += other_low > high;
        near += other_high >= low;
      };
      if constexpr (L == 8) {  // lane ^ n for all n, of which other groups' are multiples of c.lanes
        const float l7 = dpp<kXor7>(low), h7 = dpp<kXor7>(high);
        if (c.lanes < 2) {
          meet(dpp<kXor1>(low), dpp<kXor1>(high));
          meet(dpp<kXor3>(low), dpp<kXor3>(high));
          meet(dpp<kXor2>(l7), dpp<kXor2>(h7));
          meet(l7, h7);
        }
        if (c.lanes < 4) {
          meet(dpp<kXor2>(low), dpp<kXor2>(high));
          meet(dpp<kXor1>(l7), dpp<kXor1>(h7));
        }
        meet(dpp<kXor3>(l7), dpp<kXor3>(h7));
      } else {
#define BSQ_TURN(N) \
  if (((N) & (c.lanes - 1)) == 0) meet(dpp<ror(N)>(low), dpp<ror(N)>(high));
        BSQ_TURN(1) BSQ_TURN(2) BSQ_TURN(3) BSQ_TURN(4) BSQ_TURN(5) BSQ_TURN(6) BSQ_TURN(7) BSQ_TURN(8)
        BSQ_TURN(9) BSQ_TURN(10) BSQ_TURN(11) BSQ_TURN(12) BSQ_TURN(13) BSQ_TURN(14) BSQ_TURN(15)
#undef BSQ_TURN
      }
      const bool keep = near < c.group_k;
      unsure = high > -kInf && !keep && over < c.group_k;
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = keep ? b[i] : -kInf;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) lds.key[mine][e0 + i] = b[i];
      // the largest score stands for all: the bound is wider than it need be
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) most = fmaxf(most, s[i]);
      most = row_maxf<L>(most);
      wave_fence();
      for (int q = sub; q < c.groups; q += L) {
        Top o = {-kInf, -kInf, most};
#pragma unroll 4
        for (int e = q * c.size; e < (q + 1) * c.size; ++e) {
          const float v = lds.key[mine][e];
          o.b = fmaxf(o.b, fminf(o.a, v));
          o.a = fmaxf(o.a, v);
        }
        float low, high;
        worth(o, c.group_top, c.softmax, low, high);
        lds.bound[mine][q][0] = low;
        lds.bound[mine][q][1] = high;
      }
      wave_fence();
      uint64_t kept = 0;  // of the groups that this lane looks at
      for (int q = sub; q < c.groups; q += L) {
        const float low = lds.bound[mine][q][0], high = lds.bound[mine][q][1];
        int over = 0, near = 0;
        for (int p = 0; p < c.groups; ++p) {
          over += p != q && lds.bound[mine][p][0] > high;
          near += p != q && lds.bound[mine][p][1] >= low;
        }
        const bool keep = near < c.group_k;
        unsure |= high > -kInf && !keep && over < c.group_k;
        kept |= (uint64_t)keep << q;
      }
#pragma unroll
      for (int o = 1; o < L; o *= 2) kept |= __shfl_xor((unsigned long long)kept, o, 64);
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = e0 + i < c.E && (kept >> ((e0 + i) * c.over_size >> 20) & 1) ? b[i] : -kInf;
    }
  }
  double key[V];
  wave_fence();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = with_index(b[i], e0 + i);
    lds.high[i][lane] = b[i] + key_bound(s[i], b[i], c.softmax);
  }
  auto next = [&]() {  // the row's largest key, which is taken out
    double best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = fmax(best, key[i]);
    best = row_max64<L>(best);
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = key[i] == best ? __hiloint2double((int)kGone, __double2loint(key[i])) : key[i];
    return best;
  };
  auto left = [&]() {  // the most that a key not taken out may be, of this lane's
    float most = -kInf;
#pragma unroll
    for (int i = 0; i < V; ++i) most = fmaxf(most, is_gone(key[i]) ? -kInf : lds.high[i][lane]);
    return most;
  };
  int ri[KR];
#pragma unroll
  for (int q = 0; q < KR; ++q) ri[q] = -1;
  double last = 0.0;
  for (int j = 0; j < c.k; ++j) {
    last = next();
#pragma unroll
    for (int q = 0; q < KR; ++q)
      if (j == q * L + sub && !is_gone(last)) ri[q] = index_of(last);
  }
  // the selected ones' logits, biases, scores and keys
  float rx[KR], rb[KR], rs[KR], rc[KR], tol[KR];
  auto look = [&](int i, float& lx, float& lb, float& ls, float& lc, float& lt) {
    lx = load1(row + i);
    lb = bias ? bias[i] : 0.0f;
    ls = c.softmax ? exp_neg(lx - m) * inv : sigmoid32(lx);
    lc = ls + lb;
    lt = key_bound(ls, lc, c.softmax);
  };
#pragma unroll
  for (int q = 0; q < KR; ++q) look(ri[q] >= 0 ? ri[q] : 0, rx[q], rb[q], rs[q], rc[q], tol[q]);
  // the selected each against the one after it, and all others against the least of them
  const int first = mine * L;  // the row's first lane
  const uint64_t of_row = (L == 64 ? ~0ull : (1ull << (L & 63)) - 1) << first;
  bool close = false;          // two selected that follow each other are nearer than the bounds
  float low = kInf;            // what the selected keys are at least
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    const int from = first + (sub + 1) % L;
    int ni = __shfl(ri[q], from, 64);
    float nx = __shfl(rx[q], from, 64), nb = __shfl(rb[q], from, 64), nc = __shfl(rc[q], from, 64);
    float nt = __shfl(tol[q], from, 64);
    if constexpr (KR > 1) {
      const int q1 = q + 1 < KR ? q + 1 : q;
      const int li = __shfl(ri[q1], first, 64);
      const float lx = __shfl(rx[q1], first, 64), lb = __shfl(rb[q1], first, 64), lc = __shfl(rc[q1], first, 64);
      const float lt = __shfl(tol[q1], first, 64);
      if (sub == L - 1) ni = li, nx = lx, nb = lb, nc = lc, nt = lt;
    }
    const int j = q * L + sub;
    if (j < c.k - 1 && ri[q] >= 0 && ni >= 0)
      close |= !(nx == rx[q] && nb == rb[q]) && !(rc[q] - nc > tol[q] + nt);
    if (j < c.k && ri[q] >= 0) low = fminf(low, rc[q] == kInf ? kBig : rc[q] - tol[q]);
  }
  low = over_row<L>(low, [](float p, float q) { return fminf(p, q); });
  bool open = row_maxf<L>(left()) >= low;  // it is open what is selected
  if (__any(open && ok)) {  // of the others, those of the same inputs are behind the last selected by their index
    uint32_t equal = 0;  // this lane's of the same float32 key
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t low_bits = (uint32_t)(__double2loint(key[i]) ^ __double2loint(last));
      equal |= (uint32_t)(__double2hiint(key[i]) == __double2hiint(last) && low_bits < 1u << 29) << i;
    }
    if (__any(open && ok && equal)) {
      const int at = first + (c.k - 1) % L;
      float lx = 0, lb = 0, rest = -kInf;
#pragma unroll
      for (int q = 0; q < KR; ++q)
        if (q == (c.k - 1) / L) lx = __shfl(rx[q], at, 64), lb = __shfl(rb[q], at, 64);
      bool tie = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        bool same = open && (equal >> i & 1);
        if (same) same = load1(row + e0 + i) == lx && (bias ? bias[e0 + i] : 0.0f) == lb;
        tie |= same;
        rest = fmaxf(rest, same || is_gone(key[i]) ? -kInf : lds.high[i][lane]);
      }
      open = row_maxf<L>(rest) >= low;
      tie = (__ballot(tie) & of_row) != 0;
      unsure |= tie && close;  // one of the same may belong before a selected one
    }
  }
  if (KR <= 2 && __any((close || open) && ok)) {
    // Where it is open what is selected, the free places of a row take the keys that follow: all that may be
    // selected are then there, unless one that is left may still reach the least of the selected. What is there is
    // put in order by float64 keys.
    constexpr int C = L * KR;
    const bool more = __any(open && ok);
    for (int j = c.k; more && j < C; ++j) {
      const double best = next();
#pragma unroll
      for (int q = 0; q < KR; ++q)
        if (j == q * L + sub && !is_gone(best)) ri[q] = index_of(best);
    }
    const bool sort = (__ballot(close || open) & of_row) != 0;
    unsure |= row_maxf<L>(left()) >= low && open;
    double total = 1.0;
    if (c.softmax) {
      total = 0.0;
#pragma unroll 1
      for (int e = e0; e < e0 + V && e < c.E; ++e) {
        const float l = load1(row + e);
        if (l > -kInf) total += exp((double)l - (double)m);
      }
      total = over_row<L>(total, [](double p, double q) { return p + q; });
    }
    double kd[KR];
#pragma unroll
    for (int q = 0; q < KR; ++q) {
      float ls, lc, lt;
      kd[q] = -(double)kInf;
      if (ri[q] >= 0) {
        look(ri[q], rx[q], rb[q], ls, lc, lt);
        // NaN where a softmax row holds +inf: above the empty places, so that ranks are distinct there too
        kd[q] = fmax(key64(rx[q], rb[q], c.softmax, m, total), -__DBL_MAX__);
      }
    }
    int rank[KR];
#pragma unroll
    for (int q = 0; q < KR; ++q) rank[q] = 0;
#pragma unroll
    for (int z = 0; z < KR; ++z)
#pragma unroll 8
      for (int l = 0; l < L; ++l) {
        const double od = __shfl(kd[z], first + l, 64);
        const int oi = __shfl(ri[z], first + l, 64);
#pragma unroll
        for (int q = 0; q < KR; ++q) rank[q] += od > kd[q] || (od == kd[q] && oi < ri[q]);
      }
#pragma unroll
    for (int q = 0; q < KR; ++q)
      if (ri[q] >= 0) lds.pick[mine * C + rank[q]] = ri[q];
    wave_fence();
    if (sort) {
#pragma unroll
      for (int q = 0; q < KR; ++q) {
        const int j = q * L + sub;
        if (j < c.k && ri[q] >= 0) {
          ri[q] = lds.pick[mine * C + j];
          rx[q] = load1(row + ri[q]);
        }
      }
    }
    wave_fence();
  } else {
    unsure |= close || open;
  }
  // rows that float32 cannot settle, one after the other
  uint64_t again = __ballot(unsure && ok);
  while (again) {
    const int r = __builtin_ctzll(again) / L;
    again &= L == 64 ? 0ull : ~(((1ull << (L & 63)) - 1) << (r * L));
    const int64_t tr = (int64_t)blockIdx.x * (kThreads / L) + (threadIdx.x >> 6) * (64 / L) + r;
    wave_fence();
    select64<T, L, V>(logits + tr * c.E, bias, c, lds);
    if (mine == r) {
#pragma unroll
      for (int q = 0; q < KR; ++q) {
        const int j = q * L + sub;
        if (j < c.k) {
          ri[q] = lds.pick[j];
          rx[q] = load1(row + (ri[q] >= 0 ? ri[q] : 0));
        }
      }
    }
    wave_fence();
  }
  // Weights. Sigmoids over e^a, a the largest min(l, 0): their ratios hold for logits of any size.
  float e[KR], total = 0.0f, a = -kInf;
  if (!c.softmax && c.renorm) {
#pragma unroll
    for (int q = 0; q < KR; ++q)
      if (q * L + sub < c.k && ri[q] >= 0) a = fmaxf(a, fminf(rx[q], 0.0f));
    a = row_maxf<L>(a);
  } else {
    a = 0.0f;
  }
  if (c.softmax && c.renorm) {  // the softmax over the selected
    a = -kInf;
#pragma unroll
    for (int q = 0; q < KR; ++q)
      if (q * L + sub < c.k && ri[q] >= 0) a = fmaxf(a, rx[q]);
    a = row_maxf<L>(a);
    m = a;
  }
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    const bool in = q * L + sub < c.k && ri[q] >= 0;
    if (c.softmax) e[q] = in ? exp_neg(rx[q] - m) : 0.0f;
    else e[q] = in ? exp_neg(fminf(rx[q], 0.0f) - a) / (1.0f + exp_neg(-fabsf(rx[q]))) : 0.0f;
    total += e[q];
  }
  total = row_addf<L>(total);
  const float f = c.renorm ? (total > 0.0f ? c.scale / total : 0.0f) : c.softmax ? c.scale * inv : c.scale;
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    const int j = q * L + sub;
    if (ok && j < c.k) {
      weights[t * c.k + j] = e[q] * f;
      ids[t * c.k + j] = ri[q];
    }
  }
}

// The row's incoming gradients are spread over its E experts in LDS (zeros,
// then one write per selected expert); each lane then reads its own V. Bound by
// memory: 65536 x 128, top 8, bf16 7.2 us, of which 23 MB at a copy's rate are 4.8.
template <typename T, int L, int V, bool WHOLE, int KR>
__global__ __launch_bounds__(kThreads) void k_group_gate_backward(const float* __restrict__ dweights,
                                                                 const float* __restrict__ weights,
                                                                 const int32_t* __restrict__ ids,
                                                                 const T* __restrict__ logits, int64_t tokens,
                                                                 Choice c, T* __restrict__ dlogits) {
  __shared__ float spread[kThreads / L][L * V];
  const int sub = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool ok = t < tokens, all = c.softmax && !c.renorm;
  float* mine = spread[threadIdx.x / L];
  const T* row = logits + (ok ? t : 0) * c.E;
  float w[KR], g[KR], x[V];
  int id[KR];
  float inner = 0.0f;
  if (all) load_logits<T, V, WHOLE>(row, sub * V, c.E, ok, x);
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    const int j = q * L + sub;
    const bool in = ok && j < c.k;
    id[q] = in ? ids[t * c.k + j] : -1;
    if (id[q] >= c.E) id[q] = -1;
    w[q] = id[q] >= 0 ? weights[t * c.k + j] : 0.0f;
    g[q] = id[q] >= 0 ? dweights[t * c.k + j] : 0.0f;
    inner += w[q] * g[q];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) mine[sub * V + i] = 0.0f;
  inner = row_addf<L>(inner);
  wave_fence();
  const float mean = c.renorm ? inner / c.scale : 0.0f;
#pragma unroll
  for (int q = 0; q < KR; ++q)
    if (id[q] >= 0) {
      float d = w[q] * (g[q] - mean);
      if (all) {
        d = c.scale * g[q];
      } else if (!c.softmax) {
        const float l = load1(row + id[q]), n = exp_neg(-fabsf(l));
        d *= (l >= 0.0f ? n : 1.0f) / (1.0f + n);  // 1 - sigmoid(l)
      }
      mine[id[q]] = d;
    }
  wave_fence();
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = mine[sub * V + i];
  if (all) {
    float top = -kInf, total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);  // drops NaN
    top = row_maxf<L>(top);
    const float m = top > -kInf ? top : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = x[i] > -kInf ? exp_neg(x[i] - m) : 0.0f;
      total += x[i];
    }
    total = row_addf<L>(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = x[i] * inv * (d[i] - inner);
  }
  if (ok) store_grads<T, V, WHOLE>(dlogits + t * c.E, sub * V, c.E, d);
}

template <typename T, int L, int V, bool WHOLE>
void launch_gate(const T* logits, const float* bias, int64_t tokens, Choice c, float* weights, int32_t* ids,
                 hipStream_t s) {
  constexpr int64_t per = kThreads / L, most = bsqh::max_blocks(kThreads) * per;
  // groups that whole lanes hold, a power of two of them: exchanged between lanes, else through LDS
  c.lanes = 0;
  if (L <= 16 && c.E == L * V && c.size % V == 0 && ((c.size / V) & (c.size / V - 1)) == 0) c.lanes = c.size / V;
  for (; tokens > 0; tokens -= most, logits += most * c.E, weights += most * c.k, ids += most * c.k) {
    const int64_t n = tokens < most ? tokens : most;
    const unsigned grid = (unsigned)((n + per - 1) / per);
#define BSQ_K(KR) \
  hipLaunchKernelGGL((k_group_gate<T, L, V, WHOLE, KR>), dim3(grid), dim3(kThreads), 0, s, logits, bias, n, c, weights, ids)
    if (c.k < L) {
      BSQ_K(1);
      continue;
    }
    if constexpr (L < 16) {
      if (c.k < 16) {
        BSQ_K(16 / L);
        continue;
      }
    }
    BSQ_K(64 / L + 1);
#undef BSQ_K
  }
}

template <typename T, int L, int V, bool WHOLE>
void launch_back(const float* dw, const float* w, const int32_t* ids, const T* logits, int64_t tokens, Choice c,
                 T* dlogits, hipStream_t s) {
  constexpr int64_t per = kThreads / L, most = bsqh::max_blocks(kThreads) * per;
  for (; tokens > 0;
       tokens -= most, dw += most * c.k, w += most * c.k, ids += most * c.k, logits += most * c.E, dlogits += most * c.E) {
    const int64_t n = tokens < most ? tokens : most;
    const unsigned grid = (unsigned)((n + per - 1) / per);
    if (c.k <= L)
      hipLaunchKernelGGL((k_group_gate_backward<T, L, V, WHOLE, 1>), dim3(grid), dim3(kThreads), 0, s, dw, w, ids,
                         logits, n, c, dlogits);
    else
      hipLaunchKernelGGL((k_group_gate_backward<T, L, V, WHOLE, 64 / L>), dim3(grid), dim3(kThreads), 0, s, dw, w, ids,
                         logits, n, c, dlogits);
  }
}

// L lanes of V experts each. A selection's round costs a search of V keys in a
// lane, for 64 / L rows at once, and an exchange over L lanes: 8 lanes of 16
// experts took 38.6 us where 16 lanes of 8 took 41 (65536 tokens, 128 experts).
#define BSQ_GROUP_SHAPES(FN, T, ...)                  \
  if (E == 64) FN<T, 8, 8, true>(__VA_ARGS__);        \
  else if (E == 128) FN<T, 8, 16, true>(__VA_ARGS__); \
  else if (E == 256) FN<T, 16, 16, true>(__VA_ARGS__); \
  else if (E <= 32) FN<T, 8, 4, false>(__VA_ARGS__);  \
  else if (E < 64) FN<T, 8, 8, false>(__VA_ARGS__);   \
  else if (E < 128) FN<T, 8, 16, false>(__VA_ARGS__); \
  else if (E < 256) FN<T, 16, 16, false>(__VA_ARGS__); \
  else FN<T, 64, 16, false>(__VA_ARGS__)

int check(int dtype, int64_t tokens, int64_t E, int64_t k, int score, int renormalize, float scale) {
  BSQ_REQUIRE(dtype == BSQ_F32 || dtype == BSQ_BF16, BSQ_E_DTYPE);
  BSQ_REQUIRE((score == BSQ_SCORE_SIGMOID || score == BSQ_SCORE_SOFTMAX) && (renormalize == 0 || renormalize == 1),
              BSQ_E_ENUM);
  BSQ_REQUIRE(scale >= 0x1p-64f && scale <= 0x1p64f, BSQ_E_ENUM);  // NaN fails too
  BSQ_REQUIRE(tokens >= 0 && tokens < (int64_t)1 << 31 && E >= 1 && E <= 1024 && k >= 1 && k <= 64 && k <= E,
              BSQ_E_SHAPE);
  return BSQ_OK;
}

}  // namespace

extern "C" int bsq_moe_gate_grouped(const void* logits, int dtype, const float* bias, int64_t tokens, int64_t E,
                                    int64_t k, int64_t groups, int64_t group_k, int group_top, int score,
                                    int renormalize, float scale, float* weights, int32_t* topk_ids,
                                    bsq_stream_t stream) {
  const int st = check(dtype, tokens, E, k, score, renormalize, scale);
  if (st != BSQ_OK) return st;
  BSQ_REQUIRE(group_top == 1 || group_top == 2, BSQ_E_ENUM);
  BSQ_REQUIRE(groups >= 1 && groups <= kMaxGroups && E % groups == 0 && group_k >= 1 && group_k <= groups &&
                  k <= group_k * (E / groups),
              BSQ_E_SHAPE);
  if (tokens == 0) return BSQ_OK;
  BSQ_REQUIRE(logits && weights && topk_ids, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(logits) && (((uintptr_t)weights | (uintptr_t)topk_ids | (uintptr_t)bias) & 3) == 0,
              BSQ_E_ALIGN);
  hipStream_t s = bsqh::as_stream(stream);
  // all groups kept: no choice of groups
  const Choice c = {(int)E, (int)k, group_k == groups ? 1 : (int)groups, (int)(E / groups), (int)group_k, group_top, 0,
                    (int)(((1 << 20) + E / groups - 1) / (E / groups)),
                    score == BSQ_SCORE_SOFTMAX, renormalize == 1, scale};
  if (dtype == BSQ_F32) {
    BSQ_GROUP_SHAPES(launch_gate, float, static_cast<const float*>(logits), bias, tokens, c, weights, topk_ids, s);
  } else {
    BSQ_GROUP_SHAPES(launch_gate, uint16_t, static_cast<const uint16_t*>(logits), bias, tokens, c, weights, topk_ids, s);
  }
  return bsqh::launch_status();
}

extern "C" int bsq_moe_gate_grouped_backward(const float* dweights, const float* weights, const int32_t* topk_ids,
                                             const void* logits, int dtype, int64_t tokens, int64_t E, int64_t k,
                                             int score, int renormalize, float scale, void* dlogits,
                                             bsq_stream_t stream) {
  const int st = check(dtype, tokens, E, k, score, renormalize, scale);
  if (st != BSQ_OK || tokens == 0) return st;
  BSQ_REQUIRE(dweights && weights && topk_ids && dlogits && logits, BSQ_E_NULL);
  BSQ_REQUIRE(bsqh::aligned16(logits) && bsqh::aligned16(dlogits) &&
                  (((uintptr_t)weights | (uintptr_t)dweights | (uintptr_t)topk_ids) & 3) == 0,
              BSQ_E_ALIGN);
  hipStream_t s = bsqh::as_stream(stream);
  const Choice c = {(int)E, (int)k, 1, (int)E, 1, 1, 0, 0, score == BSQ_SCORE_SOFTMAX, renormalize == 1, scale};
  if (dtype == BSQ_F32) {
    BSQ_GATE_SHAPES(launch_back, float, dweights, weights, topk_ids, static_cast<const float*>(logits), tokens, c,
                    static_cast<float*>(dlogits), s);
  } else {
    BSQ_GATE_SHAPES(launch_back, uint16_t, dweights, weights, topk_ids, static_cast<const uint16_t*>(logits), tokens, c,
                    static_cast<uint16_t*>(dlogits), s);
  }
  return bsqh::launch_status();
}
