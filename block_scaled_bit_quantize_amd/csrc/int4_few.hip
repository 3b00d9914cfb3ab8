// Products of up to 64 rows of activations a launch with weights in 4-bit groups.
//
// Up to 64 rows of activations, which stay in LDS: bound by reading the weights
// once. Weights go from memory to registers: a wave keeps kDeep chunks of 16 rows
// by 256 codes on their way, across tiles of 16 rows. (With chunks of 128 the loads
// of scales and zero points, a row a lane, kept the address unit as busy as those
// of the codes: 72 us for 100003 x 4096 and one row. As it is 5 rows take 43 us,
// 4.9 TB/s; 4096 x 4096 and one row 6.8 us, its latency from launch to first weights,
// 16 tiles' rounds and the joined sums.)
//   SHARE: up to 16 rows of x, whole in LDS. The eight waves of a workgroup share
//   K, and their partial sums meet in LDS; a workgroup takes tile after tile.
//   else: more rows, or longer ones. A workgroup has a slab of K of them in LDS,
//   and each wave tiles of its own; the slabs' sums meet in a second launch.
//
// Lane l holds row l % 16's codes [32 p, 32 p + 32) of each half of a chunk, p =
// l / 16, as one 16-byte load. Matrix instruction i of a half multiplies one word
// of each lane: 32 codes. Groups of 128 take them as they lie; for shorter groups
// lanes exchange words first, so that the 32 codes are of one group.
//
// Zero points: sum (q - z) x = sum q x - z sum x; the second sums are made once
// for all tiles, by the same instruction with ones.
#include "bsq_int4.h"

using namespace bsqd;
using namespace bsqh;

namespace {

template <int G>
__device__ __forceinline__ void regroup(u32x4& w) {
  if constexpr (G == 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[2], w[3], false, false);
    w = (u32x4){a[0], b[0], a[1], b[1]};
  } else if constexpr (G == 32) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = (u32x4){c[0], c[1], d[0], d[1]};
  }
}
// Where in the chunk the eight codes begin that lane group p holds in word i after regroup().
template <int G>
__device__ __forceinline__ int place_of(int p, int i) {
  if constexpr (G == 128) return p * 32 + i * 8;
  else if constexpr (G == 64) return (i >> 1) * 64 + (p & 1) * 32 + (p >> 1) * 8 + (i & 1) * 16;
  else return i * 32 + p * 8;
}

// Of a lane's row: a chunk's codes, and the scales and zero points of its groups,
// the first lowest. Each is what one load gives: anything done to it on the way
// would wait for it, and for all loads before it.
template <int G>
struct Chunk {
  static constexpr int groups = kChunk / G;
  u32x4 w[2];
  uint32_t s[groups / 2], z[groups > 4 ? groups / 4 : 1];
};

// KIND: K of whole chunks with zero points, without, or neither. BYTES of LDS: half of a CU's where that does, for
// two workgroups a CU. slab: values of K of a workgroup. Outputs, or (parts given) a slab's sums, [slab][M][N].
template <typename X, int G, int MT, bool SHARE, int KIND, int BYTES>
__global__ __launch_bounds__(kFThreads) void k_linear_int4_few(const X* __restrict__ x, const uint8_t* __restrict__ codes,
                                                              const uint16_t* __restrict__ scales,
                                                              const uint8_t* __restrict__ zeros,
                                                              const float* __restrict__ bias, int M, int64_t N, int K,
                                                              int slab, float* __restrict__ parts, int64_t pitch_out,
                                                              void* __restrict__ out, int out_f32) {
  constexpr bool RAGGED = KIND == kRagged;
  const bool ZEROS = KIND == kZeros || (RAGGED && zeros);
  constexpr int P = Mfma<X>::parts, GP = 128 / G, GC = 2 * GP;  // groups of half a chunk, of a chunk
  __shared__ __attribute__((aligned(16))) uint8_t lds[BYTES];
  __shared__ uint32_t rmax[P > 1 ? 16 * MT : 1];
  f32x4* red = reinterpret_cast<f32x4*>(lds);  // SHARE: [2][waves][64]
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63, col = lane & 15, p = lane >> 4;
  const int k0 = SHARE ? 0 : (int)blockIdx.y * slab, k_end = K - k0 < slab ? K : k0 + slab;  // this workgroup's K
  const int chunks = (k_end - k0 + kChunk - 1) / kChunk, pitch = (int)few_pitch(slab, sizeof(X));
  f32x4* table = reinterpret_cast<f32x4*>(lds + (SHARE ? kFewRed : 0));
  uint8_t* xs = lds + (SHARE ? kFewRed : 0) + few_table(slab, G, MT);
  {
    const rsrc_words d = descriptor(x, (uint32_t)M * K * (uint32_t)sizeof(X));
    const uint32_t base = lds_offset(xs), from = (uint32_t)k0 * sizeof(X), to = (uint32_t)k_end * sizeof(X);
    const int row_loads = pitch / 1024;
    for (int i = wave; i < M * row_loads; i += kFWaves) {
      const int r = i / row_loads, c = i - r * row_loads;
      const uint32_t at = from + c * 1024 + lane * 16;
      load_to_lds<16>(d, buffer_at(true, at < to, (uint32_t)r * K * (uint32_t)sizeof(X) + at, 0), base + r * pitch + c * 1024);
    }
  }
  if constexpr (P > 1) {
    if (t < 16 * MT) rmax[t] = 0u;
  }
  const int64_t tiles = (N + 15) / 16, stride = SHARE ? gridDim.x : (int64_t)gridDim.x * kFWaves;
  const int64_t tile0 = SHARE ? blockIdx.x : (int64_t)blockIdx.x * kFWaves + wave;
  const int KG = K / G;
  const int c0 = SHARE ? chunks * wave / kFWaves : 0;  // this wave's chunks
  const int nc = SHARE ? chunks * (wave + 1) / kFWaves - c0 : chunks;
  const int64_t total = tile0 < tiles ? ((tiles - 1 - tile0) / stride + 1) * nc : 0;  // chunks of this wave
  int64_t ft = tile0;  // the tile and the chunk that are asked for next
  int fc = 0;
  auto fetch = [&](Chunk<G>& f) {
    int64_t n = ft * 16 + col;  // this lane's row
    if (n >= N) n = N - 1;
    const int k = k0 + (c0 + fc) * kChunk;
    const uint8_t* at_w = codes + n * (K / 2) + k / 2 + p * 16;
    const int64_t g = n * KG + k / G;
    if constexpr (!RAGGED) {
      f.w[0] = *reinterpret_cast<const u32x4*>(at_w);
      f.w[1] = *reinterpret_cast<const u32x4*>(at_w + 64);
      __builtin_memcpy(f.s, scales + g, 2 * GC);
      if constexpr (KIND == kZeros) {
        if constexpr (GC == 2) {
          uint16_t z;
          __builtin_memcpy(&z, zeros + g, 2);
          f.z[0] = z;
        } else {
          __builtin_memcpy(f.z, zeros + g, GC);
        }
      }
    } else {  // the last chunk of a row may be a part of one
      f = Chunk<G>{};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (k + h * 128 + p * 32 < K) f.w[h] = *reinterpret_cast<const u32x4*>(at_w + h * 64);
#pragma unroll
      for (int j = 0; j < GC; ++j)
        if (k + j * G < K) {
          f.s[j / 2] |= (uint32_t)scales[g + j] << (16 * (j & 1));
          if (ZEROS) f.z[j / 4] |= (uint32_t)zeros[g + j] << (8 * (j & 3));
        }
    }
    const bool end = ++fc == nc;
    fc = end ? 0 : fc;
    ft = end ? ft + stride : ft;
  };
  Chunk<G> ring[kDeep];
#pragma unroll
  for (int d = 0; d < kDeep; ++d)
    if (d < total) fetch(ring[d]);
  wait_loads<0>();
  __syncthreads();
  if ((k_end - k0) % kChunk) {  // past the end of K anything may lie there
    const int from = (k_end - k0) * (int)sizeof(X), per = (chunks * kChunk * (int)sizeof(X) - from) / 16;
    for (int u = t; u < M * per; u += kFThreads)
      *reinterpret_cast<u32x4*>(xs + u / per * pitch + from + u % per * 16) = (u32x4){0, 0, 0, 0};
    if constexpr (P == 1) __syncthreads();  // else those of the parts
  }
  if constexpr (P > 1) {  // eight values of x become their two parts, in place
    const int per = (k_end - k0) / 8, units = M * per;
    for (int u = t; u < units; u += kFThreads) {
      const int r = u / per;
      const u32x4* v = reinterpret_cast<const u32x4*>(xs + r * pitch + (u - r * per) * 32);
      uint32_t most = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t b = v[h][j] & 0x7FFFFFFFu;  // by bits: a NaN's are above an infinity's
          most = b > most ? b : most;
        }
      atomicMax(&rmax[r], most);
    }
    __syncthreads();
    for (int u = t; u < units; u += kFThreads) {
      const int r = u / per;
      u32x4* v = reinterpret_cast<u32x4*>(xs + r * pitch + (u - r * per) * 32);
      u32x4 hi, lo;
      split8(__builtin_bit_cast(f32x4, v[0]), __builtin_bit_cast(f32x4, v[1]), of_exponent(row_factor(rmax[r])), hi, lo);
      v[0] = lo;
      v[1] = hi;
    }
    __syncthreads();
  }
  // the eight values from k on of row 16 m + col (rows past M repeat row 0)
  const uint8_t* my_x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) my_x[m] = xs + (m * 16 + col < M ? m * 16 + col : 0) * pitch;
  auto load_x = [&](int m, int k, int part) {
    return *reinterpret_cast<const u32x4*>(my_x[m] + k * (int)sizeof(X) + part * 16);
  };
  for (int c = wave; c < 2 * chunks; c += kFWaves) {  // halves
    const u32x4 ones = {Mfma<X>::ones, Mfma<X>::ones, Mfma<X>::ones, Mfma<X>::ones};
#pragma unroll
    for (int j = 0; j < GP; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 of_x = {0, 0, 0, 0};
#pragma unroll
        for (int i = j * (4 / GP); i < (j + 1) * (4 / GP); ++i)
#pragma unroll
          for (int part = 0; part < P; ++part)
            of_x = Mfma<X>::mul16(load_x(m, c * 128 + place_of<G>(p, i), part), ones, of_x);
        if (col == 0) table[(c * GP + j) * MT * 4 + m * 4 + p] = of_x;  // rows 16 m + 4 p + (0, 1, 2, 3)
      }
  }
  __syncthreads();
  f32x4 acc[MT] = {};
  auto multiply = [&](Chunk<G>& f, int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      regroup<G>(f.w[h]);
#pragma unroll
      for (int jj = 0; jj < GP; ++jj) {
        const int j = h * GP + jj;  // group of the chunk
        f32x4 sum[MT] = {};
#pragma unroll
        for (int i = jj * (4 / GP); i < (jj + 1) * (4 / GP); ++i) {
          const int k = c * kChunk + h * 128 + place_of<G>(p, i);
          const u32x4 b = codes_of<X>(f.w[h][i]);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int part = 0; part < P; ++part) sum[m] = Mfma<X>::mul16(load_x(m, k, part), b, sum[m]);
        }
        const float s = __uint_as_float(j & 1 ? f.s[j / 2] & 0xFFFF0000u : f.s[j / 2] << 16);
        const float z = ZEROS ? (float)(f.z[j / 4] >> (8 * (j & 3)) & 0xFFu) : 8.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const f32x4 of_x = table[(c * GC + j) * MT * 4 + m * 4 + p];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][r] = __builtin_fmaf(s, __builtin_fmaf(-z, of_x[r], sum[m][r]), acc[m][r]);
        }
      }
    }
  };
  // the bias of a tile's weight row, asked for a tile ahead
  auto bias_of = [&](int64_t tile) {
    const int64_t n = tile * 16 + (SHARE ? t >> 2 & 15 : col);
    return bias ? bias[n < N ? n : N - 1] : 0.0f;
  };
  float add = bias_of(tile0 < tiles ? tile0 : 0);
  auto store = [&](int m, int64_t n, float y) {  // row m's sum for weight row n
    if constexpr (P > 1) y *= of_exponent(254u - row_factor(rmax[m]));
    if (!SHARE && parts) {
      parts[((int64_t)blockIdx.y * M + m) * N + n] = y;
    } else {
      if (out_f32) store1(static_cast<float*>(out) + m * pitch_out + n, y + add);
      else store1(static_cast<uint16_t*>(out) + m * pitch_out + n, y + add);
    }
  };
  int buf = 0;
  auto finish = [&](int64_t tile) {
    if constexpr (SHARE) {
      red[(buf * kFWaves + wave) * 64 + lane] = acc[0];
      __syncthreads();
      if (t < 256) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kFWaves; ++w) y += reinterpret_cast<const float*>(red)[(buf * kFWaves + w) * 256 + t];
        // float t of a partial tile: register t % 4 of lane t / 4
        const int m = (t >> 6) * 4 + (t & 3);
        const int64_t n = tile * 16 + (t >> 2 & 15);
        if (m < M && n < N) store(m, n, y);
      }
      buf ^= 1;  // the next tile's sums go elsewhere: its barrier stands between this one's reads and their reuse
    } else {
      const int64_t n = tile * 16 + col;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = m * 16 + p * 4 + r;
          if (row < M && n < N) store(row, n, acc[m][r]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = (f32x4){0, 0, 0, 0};
    add = bias_of(tile + stride < tiles ? tile + stride : tile);
  };
  if (nc == 0) {
    if constexpr (SHARE)
      for (int64_t tile = tile0; tile < tiles; tile += stride) finish(tile);
    return;
  }
  int64_t tile = tile0, it = 0;
  int c = 0;
  auto step = [&](Chunk<G>& f) {
    multiply(f, c0 + c);
    ++it;
    if (++c == nc) {
      finish(tile);
      c = 0;
      tile += stride;
    }
  };
  // Whole rounds of the ring, with no branch around a load: behind one the compiler would not know how many are on
  // their way, and wait for nearly all.
  while (it + 2 * kDeep <= total) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      step(ring[d]);
      fetch(ring[d]);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (it >= total) return;
      const bool more = it + kDeep < total;
      step(ring[d]);
      if (r == 0 && more) fetch(ring[d]);
    }
}

template <typename X, int G, int KIND>
void launch_share(const Int4Few& c, hipStream_t s) {
  const int64_t tiles = (c.N + 15) / 16;
  const bool half = share_bytes(c.M, c.K, G, sizeof(X)) <= kFewHalf;
  const int64_t most = device_cus() * (half ? 2 : 1);
  const dim3 grid((unsigned)(tiles < most ? tiles : most));
#define BSQ_FEW(BYTES)                                                                                              \
  hipLaunchKernelGGL((k_linear_int4_few<X, G, 1, true, KIND, BYTES>), grid, dim3(kFThreads), 0, s,                  \
                     static_cast<const X*>(c.x), c.codes, c.scales, c.zeros, c.bias, (int)c.M, c.N, (int)c.K, (int)c.K, \
                     nullptr, c.pitch_out, c.out, c.out_f32)
  if (half) BSQ_FEW(kFewHalf);
  else BSQ_FEW(kFewLds);
#undef BSQ_FEW
}

template <typename X, int G, int KIND>
void launch_slabs(const Int4Few& c, hipStream_t s) {
  const int64_t tiles = (c.N + 15) / 16, groups = (tiles + kFWaves - 1) / kFWaves;
  int64_t most = device_cus() / c.splits;  // workgroups of a slab
  if (most < 1) most = 1;
  const dim3 grid((unsigned)(groups < most ? groups : most), (unsigned)c.splits);
#define BSQ_FEW(MT)                                                                                                    \
  hipLaunchKernelGGL((k_linear_int4_few<X, G, MT, false, KIND, kSlabLds + 256 * MT + 8192>), grid, dim3(kFThreads), 0, s, \
                     static_cast<const X*>(c.x), c.codes, c.scales, c.zeros, c.bias, (int)c.M, c.N, (int)c.K,          \
                     (int)c.slab, c.splits > 1 ? c.parts : nullptr, c.pitch_out, c.out, c.out_f32)
  if (c.mt == 1) BSQ_FEW(1);
  else if (c.mt == 2) BSQ_FEW(2);
  else BSQ_FEW(4);
#undef BSQ_FEW
}

template <typename X, int G>
void run(const Int4Few& c, bool share, hipStream_t s) {
  if (c.K % kChunk) share ? launch_share<X, G, kRagged>(c, s) : launch_slabs<X, G, kRagged>(c, s);
  else if (c.zeros) share ? launch_share<X, G, kZeros>(c, s) : launch_slabs<X, G, kZeros>(c, s);
  else share ? launch_share<X, G, kPlain>(c, s) : launch_slabs<X, G, kPlain>(c, s);
}
template <typename X>
void run(const Int4Few& c, bool share, hipStream_t s) {
  if (c.group == 32) run<X, 32>(c, share, s);
  else if (c.group == 64) run<X, 64>(c, share, s);
  else run<X, 128>(c, share, s);
}

}  // namespace

void bsqh::int4_share(const Int4Few& c, hipStream_t s) {
  c.dtype == BSQ_F32 ? run<float>(c, true, s) : run<uint16_t>(c, true, s);
}
void bsqh::int4_slabs(const Int4Few& c, hipStream_t s) {
  c.dtype == BSQ_F32 ? run<float>(c, false, s) : run<uint16_t>(c, false, s);
}
