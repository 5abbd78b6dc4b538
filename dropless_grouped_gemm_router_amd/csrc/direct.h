// fp32 products of moderate size whose operands are taken from memory as they
// are, whichever of their dimensions the product runs over:
//
//   C[m][n] = sum_k S(m, k) F(n, k)
//
// mfma 16x16x4 wants one number a lane and operand: row lane % 16, k lane / 16. A
// 16-byte load gives a lane either four k of a row (kAlong: rows of consecutive k)
// or four rows of a k (kAcross: consecutive rows), and which of the four goes into
// which MFMA is free as long as both sides agree: step e of 16 k takes k 4 (lane /
// 16) + e, and the 64 rows of a tile are dealt to its four fragments so that the
// loads are what they are. So there is no turning, no padding and no LDS before the
// products, and a backward pass whose two products need both orders is one launch.
//
// A workgroup makes a tile of 64 x 64; its eight waves share k, 16 at a time, and
// their sums are added in LDS in wave order. A step is 64 MFMAs (2048 clocks) for 8
// KB of loads (12 where a slope is multiplied in). Measured at 777 x 500 x 1001: the
// forward product with its epilogue 22 us (35 TF; 208 tiles of four steps a wave on 256
// CUs: latency), its two backward products with dbias 33 us (47 TF), where tiles
// through LDS (mm.h) with what they need before and after took 34 and 51. Those win
// once there are tiles for many goes: they reach 154 TF, and here each wave loads its
// own operands, four times what a shared tile loads.
#pragma once

#include "block.h"

namespace moe {

constexpr int kDirTile = 64, kDirWaves = 8, kDirStep = 16, kDirThreads = 64 * kDirWaves;

enum { kAlong = 0, kAcross = 1 };

// One operand: kAlong p[row][k], kAcross p[k][row], `ld` between the outer ones;
// `rows` rows and K k. scale: null, or numbers of the same order that it is
// multiplied by, `ld_scale` between the outer ones. The inner dimension is four or
// more, and all of it is below 2^32 bytes.
struct DirOperand {
  const float* p;
  int64_t ld;
  const float* scale;
  int64_t ld_scale;
  int64_t rows;
};

// The rows of a tile that lane group i (lane % 16) of fragment j has: as the
// second operand a lane keeps row i of each fragment, as the first operand it
// ends up with rows 4 g + q (g: lane / 16) of each.
template <int kOrder, bool kFirst>
__device__ __forceinline__ int dir_row(int j, int i) {
  if (kOrder == kAcross) return 4 * i + j;
  // first operand: 4 j + q of 16 g, so that a lane's are 16 in a row
  return kFirst ? 16 * (i / 4) + 4 * j + i % 4 : 16 * j + i;
}

// Where a lane's four loads of a step start, and how many numbers lie between
// steps; the last step of a K that is no multiple of 16, and tiles that go past the
// last row (kAcross), are told apart by conditions that all lanes share.
template <int kOrder, bool kFirst, bool kScale>
struct DirPlaces {
  uint32_t p[4], s[kScale ? 4 : 1];  // bytes from the operand's start: below 2^32
  int64_t step, step_scale;
  int past;  // kAcross: numbers of the lane's piece behind the last row
  bool ragged;
  __device__ DirPlaces(const DirOperand& o, int64_t row0, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const uint32_t ld = static_cast<uint32_t>(o.ld), lds = static_cast<uint32_t>(o.ld_scale);
    step = kOrder == kAlong ? kDirStep : kDirStep * o.ld;
    step_scale = kOrder == kAlong ? kDirStep : kDirStep * o.ld_scale;
    ragged = kOrder == kAcross && row0 + kDirTile > o.rows;
    const int c = kOrder == kAcross ? static_cast<int>(row0) + 4 * i : 0;
    past = kOrder == kAcross ? c + 4 - static_cast<int>(o.rows) : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (kOrder == kAlong) {
        int64_t r = row0 + dir_row<kOrder, kFirst>(u, i);
        r = r < o.rows ? r : o.rows - 1;  // computed, not stored
        p[u] = (static_cast<uint32_t>(r) * ld + 4 * g) * 4;
        if constexpr (kScale) s[u] = (static_cast<uint32_t>(r) * lds + 4 * g) * 4;
      } else {
        const uint32_t at = past > 0 ? static_cast<uint32_t>(o.rows) - 4 : c;
        p[u] = ((4 * g + u) * ld + at) * 4;
        if constexpr (kScale) s[u] = ((4 * g + u) * lds + at) * 4;
      }
    }
  }
};
// 16 bytes at a byte offset from an address that all lanes share.
__device__ __forceinline__ u32x4 dir_load(const float* base, uint32_t offset) {
  return load_any(reinterpret_cast<const float*>(reinterpret_cast<const char*>(base) + offset));
}

template <int kOrder, bool kFirst, bool kScale>
struct DirLoads {
  typedef DirPlaces<kOrder, kFirst, kScale> Places;
  u32x4 v[4], s[kScale ? 4 : 1];
  // Bytes that a lane's load is moved back by, so as not to go past K.
  __device__ static uint32_t back(int64_t left, int u, int g, int64_t ld) {
    const int over = (kOrder == kAlong ? 4 * g + 4 : 4 * g + u + 1) - static_cast<int>(left);
    return over > 0 ? over * 4u * (kOrder == kAlong ? 1u : static_cast<uint32_t>(ld)) : 0u;
  }
  // Step `at` of k: all 16 of it.
  __device__ void load(const DirOperand& o, const Places& w, int64_t at) {
    const float* p = o.p + at * w.step;
    const float* s0 = o.scale + at * w.step_scale;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = dir_load(p, w.p[u]);
      if constexpr (kScale) s[u] = dir_load(s0, w.s[u]);
    }
  }
  // The same, of fewer: `left` numbers from K. A piece may start before the step.
  __device__ void load_last(const DirOperand& o, const Places& w, int64_t at, int64_t left, int g) {
    const uint32_t p = static_cast<uint32_t>(at * w.step * 4), s0 = static_cast<uint32_t>(at * w.step_scale * 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = dir_load(o.p, w.p[u] + p - back(left, u, g, o.ld));
      if constexpr (kScale) s[u] = dir_load(o.scale, w.s[u] + s0 - back(left, u, g, o.ld_scale));
    }
  }
  // Moves a piece that was loaded `past` numbers too early to its place; zeros behind it.
  __device__ static void trim(u32x4& x, int past) {
    if (past & 1) x = (u32x4){x[1], x[2], x[3], 0u};
    if (past & 2) x = (u32x4){x[2], x[3], 0u, 0u};
    if (past >= 4) x = (u32x4){0u, 0u, 0u, 0u};
  }
  // The scales multiplied in, and rows in their places. (A product of two numbers that
  // were moved alike is the moved product.)
  __device__ void settle(const Places& w) {
    if constexpr (kScale) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[u][q] = __float_as_uint(__uint_as_float(v[u][q]) * __uint_as_float(s[u][q]));
    }
    if (w.ragged && w.past > 0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) trim(v[u], w.past);
    }
  }
  // Zeros from K on, in the last step.
  __device__ void settle_last(int64_t left, int g) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (kOrder == kAlong) {
        const int past = 4 * g + 4 - static_cast<int>(left);
        if (past > 0) trim(v[u], past);
      } else if (4 * g + u >= left) {
        v[u] = (u32x4){0u, 0u, 0u, 0u};
      }
    }
  }
  __device__ float get(int j, int e) const { return __uint_as_float(kOrder == kAlong ? v[j][e] : v[e][j]); }
};

// Sums of the tile at (m0, n0) over steps s0 .. s1 - 1 of k: thread t ends up with
// row m0 + t / 8, columns n0 + 8 (t % 8) .. + 7. lds: kDirLds floats, free after the
// call's last barrier. kColumns: also the sums over k of F itself, for the 64
// columns, in `cols` (LDS, [kDirWaves][64] floats, to be added by the caller after
// the call).
constexpr int kDirLds = kDirWaves * 64 * 64;
template <int kS, int kF, bool kScaleS, bool kScaleF, bool kColumns>
__device__ __forceinline__ void dir_tile(const DirOperand& S, const DirOperand& F, int64_t K, int64_t m0, int64_t n0,
                                         int64_t s0, int64_t s1, bool columns, float* lds, float (*cols)[64],
                                         float (&out)[8]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  f32x4_t acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
  float total[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  DirLoads<kS, false, kScaleS> sv[2];
  DirLoads<kF, true, kScaleF> fv[2];
  const DirPlaces<kS, false, kScaleS> sp(S, m0, lane);
  const DirPlaces<kF, true, kScaleF> fp(F, n0, lane);
  auto load = [&](int set, int64_t s) {
    sv[set].load(S, sp, s);
    fv[set].load(F, fp, s);
  };
  auto multiply = [&](int set) {
    if (kColumns && columns) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[j] += fv[set].get(j, e);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(fv[set].get(b, e), sv[set].get(a, e), acc[a][b], 0, 0, 0);
  };
  auto settle = [&](int set) {
    sv[set].settle(sp);
    fv[set].settle(fp);
  };
  // whole steps, the next one's loads under way; then the last one, of fewer k
  const int64_t whole = K / kDirStep, end = s1 < whole ? s1 : whole;
  int64_t s = s0 + wave;
  if (s < end) load(0, s);
  for (; s < end; s += 2 * kDirWaves) {
    const int64_t n1 = s + kDirWaves, n2 = s + 2 * kDirWaves;
    load(1, n1 < end ? n1 : s);  // one that is not there is not multiplied
    settle(0);
    multiply(0);
    if (n1 >= end) break;
    load(0, n2 < end ? n2 : s);
    settle(1);
    multiply(1);
  }
  if (s1 > whole && wave == (whole - s0) % kDirWaves) {
    const int64_t left = K - whole * kDirStep;
    sv[0].load_last(S, sp, whole, left, g);
    fv[0].load_last(F, fp, whole, left, g);
    settle(0);
    sv[0].settle_last(left, g);
    fv[0].settle_last(left, g);
    multiply(0);
  }
  // register 16 a + 4 b + q of lane l at [.][l]
  float* mine = lds + wave * 4096 + lane;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) mine[(16 * a + 4 * b + q) * 64] = acc[a][b][q];
  if (kColumns && columns) {
    // kAcross: column 4 i + j; over the four lane groups first
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float other;
      total[j] = lane16(total[j], &other);
      total[j] += other;
      total[j] = lane32(total[j], &other);
      total[j] += other;
      if (g == 0) cols[wave][4 * i + j] = total[j];
    }
  }
  __syncthreads();
  const int m = threadIdx.x >> 3, n8 = (threadIdx.x & 7) * 8;
  // row m is row `mi` of fragment `a`; column n is register (b, q) of lane group n / 16
  const int a = kS == kAcross ? m % 4 : m / 16, mi = kS == kAcross ? m / 4 : m % 16;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int r = (n8 + u) % 16;
    const int b = kF == kAcross ? r % 4 : r / 4, q = kF == kAcross ? r / 4 : r % 4;
    const float* p = lds + (16 * a + 4 * b + q) * 64 + (n8 + u) / 16 * 16 + mi;
    float v = p[0];
#pragma unroll
    for (int w = 1; w < kDirWaves; ++w) v += p[w * 4096];
    out[u] = v;
  }
}

}  // namespace moe
