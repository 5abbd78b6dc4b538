// Products of few rows with weights in the layer's layout, [K][N] with N
// contiguous: the gated block's serving form. The weights' bytes are what
// such a product costs, so they are read once, where they are (no turning, no
// padding), straight into registers.
//
// A wave takes 64 columns and steps of 32 k. In bf16 a lane loads four columns
// of eight consecutive k (8-byte loads, 16 lanes side by side cover 128
// bytes of a row) and turns the 8 x 4 block in registers, one byte-select
// for two elements: fragment j holds column 4 l + j (l = lane % 16) for k
// 8 (lane / 16) .. + 7, which is the operand of mfma 16x16x32. In fp32 a lane
// loads four columns of k = 4 i + lane / 16 for i = 0..7, each an operand of
// mfma 16x16x4 as it is. The weights go in as the first operand, so lane L
// ends up with token L % 16 and, over the four fragments, the 16 consecutive
// columns 16 (L / 16) .. + 15. The waves of a workgroup share K; their sums are
// added in LDS in wave order. One token through weights of 2048 x 8192 (three
// times 33.5 MB): 23 to 30 us, 3.4 to 4.4 TB/s; turning them for the tiles
// first takes 37 us alone. From 17 rows of bf16 on the weights' repeated way
// through L2 costs more than tiles (gated_ffn.hip, kFewRows).
#pragma once

#include "block.h"

namespace moe {

constexpr int kSkinnyCols = 64, kSkinnyStep = 32, kSkinnyWaves = 8;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

// The weights of one step: rows k.., columns n .. n + 3 of a lane.
template <typename T>
struct SkinnyW;
template <>
struct SkinnyW<bf16_t> {
  u32x2 r[8];
  __device__ void load(const bf16_t* w, int64_t ld, int k0, int K, int n, int N, int lane) {
    const int k = k0 + 8 * (lane >> 4);
    const bf16_t* p = w + k * ld + n;
    if (k0 + kSkinnyStep <= K && n + 4 <= N) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = *reinterpret_cast<const u32x2_a2*>(p + i * ld);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t e[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) e[q] = (k + i < K && n + q < N) ? p[i * ld + q] : 0u;
      r[i] = (u32x2){e[0] | (e[1] << 16), e[2] | (e[3] << 16)};
    }
  }
  // Fragment j: column j of the eight rows.
  __device__ bf16x8_t frag(int j) const {
    u32x4 o;
#pragma unroll
    for (int m = 0; m < 4; ++m)
      o[m] = __builtin_amdgcn_perm(r[2 * m + 1][j / 2], r[2 * m][j / 2],
                                   (j & 1) ? 0x07060302u : 0x05040100u);
    return __builtin_bit_cast(bf16x8_t, o);
  }
};
template <>
struct SkinnyW<float> {
  u32x4 r[8];
  __device__ void load(const float* w, int64_t ld, int k0, int K, int n, int N, int lane) {
    const int k = k0 + (lane >> 4);
    const float* p = w + k * ld + n;
    if (k0 + kSkinnyStep <= K && n + 4 <= N) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = load_any(p + 4 * i * ld);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        r[i][q] = (k + 4 * i < K && n + q < N) ? __float_as_uint(p[4 * i * ld + q]) : 0u;
  }
};

// The rows of one step: token row of a lane, k as in SkinnyW.
template <typename T>
struct SkinnyX;
template <>
struct SkinnyX<bf16_t> {
  u32x4 v;
  __device__ void load(const bf16_t* row, int k0, int K, int lane) {
    v = load_piece(row, k0 + 8 * (lane >> 4), K);
  }
};
template <>
struct SkinnyX<float> {
  float v[8];
  __device__ void load(const float* row, int k0, int K, int lane) {
    const int k = k0 + (lane >> 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + 4 * i < K ? row[k + 4 * i] : 0.0f;
  }
};

// acc[j] += fragment j of w times the rows.
__device__ __forceinline__ void skinny_step(const SkinnyW<bf16_t>& w, const SkinnyX<bf16_t>& x,
                                            f32x4_t (&acc)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.frag(j), __builtin_bit_cast(bf16x8_t, x.v),
                                                     acc[j], 0, 0, 0);
}
__device__ __forceinline__ void skinny_step(const SkinnyW<float>& w, const SkinnyX<float>& x,
                                            f32x4_t (&acc)[4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w.r[i][j]), x.v[i], acc[j], 0, 0, 0);
}

// One operand: rows x [rows][K] (row stride ldx) and, where kLow, their low
// halves (put_hidden in gated_ffn.hip); kW weight matrices [K][N].
template <typename T, int kW>
struct SkinnyArgs {
  const T* x;
  const T* low;
  int64_t ldx;
  const T* w[kW];
  int64_t rows;
  int K, N;
  int k_parts;  // slices of K, one per blockIdx.z
};

// Sums of this workgroup's columns over its slice of K, for 16 rows: after the
// call thread t holds, for v = 0, 1, those of column t % 64 and row t / 64 +
// 8 v of the tile, all kW of them. In LDS register
// 4 q + j of a lane stands at 65 (4 q + j) + lane: both sides use all banks.
constexpr int kSkinnyLds = 16 * 65;
template <typename T, int kW, bool kLow>
__device__ __forceinline__ void skinny_sums(const SkinnyArgs<T, kW>& a, float (*lds)[kSkinnyLds],
                                            float (&sum)[2][kW]) {
  // the wave's number as a scalar: a step past the end has to be branched over,
  // for MFMAs run whatever lanes are on
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = blockIdx.x * kSkinnyCols + 4 * (lane & 15);
  const int steps = (a.K + kSkinnyStep - 1) / kSkinnyStep;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * blockIdx.z / a.k_parts);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (blockIdx.z + 1) / a.k_parts);
  int64_t r = static_cast<int64_t>(blockIdx.y) * 16 + (lane & 15);
  r = r < a.rows ? r : a.rows - 1;  // computed, not stored
  const T* row = a.x + r * a.ldx;
  const T* low = kLow ? a.low + r * a.ldx : nullptr;
  f32x4_t acc[kW][4];
#pragma unroll
  for (int m = 0; m < kW; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};

  SkinnyW<T> w[2][kW];
  SkinnyX<T> x[2], xl[2];
  auto load = [&](int set, int s) {
#pragma unroll
    for (int m = 0; m < kW; ++m) w[set][m].load(a.w[m], a.N, s * kSkinnyStep, a.K, n, a.N, lane);
    x[set].load(row, s * kSkinnyStep, a.K, lane);
    if (kLow) xl[set].load(low, s * kSkinnyStep, a.K, lane);
  };
  auto multiply = [&](int set) {
#pragma unroll
    for (int m = 0; m < kW; ++m) {
      skinny_step(w[set][m], x[set], acc[m]);
      if (kLow) skinny_step(w[set][m], xl[set], acc[m]);
    }
  };
  // two steps in flight
  int s = s0 + wave;
  if (s < s1) load(0, s);
  for (; s < s1; s += 2 * kSkinnyWaves) {
    if (s + kSkinnyWaves < s1) load(1, s + kSkinnyWaves);
    multiply(0);
    if (s + 2 * kSkinnyWaves < s1) load(0, s + 2 * kSkinnyWaves);
    if (s + kSkinnyWaves < s1) multiply(1);
  }

  const int c = lane;  // column that this thread adds up
#pragma unroll
  for (int m = 0; m < kW; ++m) {
    // register q of fragment j is column 4 q + j of the lane's 16
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) lds[wave][(4 * q + j) * 65 + lane] = acc[m][j][q];
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float t = 0.0f;
#pragma unroll
      for (int u = 0; u < kSkinnyWaves; ++u) t += lds[u][(c & 15) * 65 + (c >> 4) * 16 + wave + 8 * v];
      sum[v][m] = t;
    }
    __syncthreads();
  }
}

}  // namespace moe
