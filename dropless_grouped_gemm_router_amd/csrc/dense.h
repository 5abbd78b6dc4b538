// What the dense products share (gated_ffn.hip, linear.hip): activations,
// layout changes, the choice of tiles and slices, weight gradients.
#pragma once

#include <algorithm>

#include "gemm_wgrad.h"
#include "mm.h"
#include "skinny.h"

namespace moe {

constexpr int64_t kCUs = 256;

constexpr int64_t pad128(int64_t v) { return (v + 127) / 128 * 128; }

// ------------------------------------------------------------- activations

template <int kAct>
__device__ __forceinline__ float act_value(float a, float* slope) {
  if (kAct == MOE_ACT_NONE) {
    *slope = 1.0f;
    return a;
  }
  if (kAct == MOE_ACT_RELU) {
    *slope = a > 0.0f ? 1.0f : 0.0f;
    return a < 0.0f ? 0.0f : a;  // NaN stays
  }
  if (kAct == MOE_ACT_GELU) {
    const float cdf = 0.5f * (1.0f + erff(a * 0.70710678118654752f));
    *slope = cdf + a * 0.39894228040143268f * __expf(-0.5f * a * a);
    return a * cdf;
  }
  if (kAct == MOE_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 is the logistic function of 2 u
    const float k = 0.79788456080286536f, c = 0.044715f;
    const float s = sigmoid_f(2.0f * k * (a + c * a * a * a));
    const float bend = s * (1.0f - s);  // 0 where a^2 may overflow
    *slope = bend > 0.0f ? s + a * 2.0f * bend * k * (1.0f + 3.0f * c * a * a) : s;
    return a * s;
  }
  const float s = sigmoid_f(a), v = a * s;
  *slope = __builtin_fmaf(v, 1.0f - s, s);
  return v;
}

// ---------------------------------------------------------- layout changes

// dst[n][kp] from src[k][n] (row stride ld): 64 x 64 blocks through LDS; zeros
// for k >= K (kp: K rounded up to 128). Up to four matrices in one launch, the
// flat block index running over them.
struct TurnJob {
  const void* src;
  void* dst;
  int64_t K, ld, kp;
  int N;
  int64_t end;  // exclusive end of the job's blocks
};
struct TurnJobs {
  TurnJob job[4];
  int n;
  u32x4* zero;  // kTrZeroBytes to clear, or null

  void add(const void* src, void* dst, int64_t K, int N, int64_t ld) {
    const int64_t blocks = pad128(K) / 64 * ((N + 63) / 64);
    job[n] = TurnJob{src, dst, K, ld, pad128(K), N, (n ? job[n - 1].end : 0) + blocks};
    ++n;
  }
};
template <typename T>
__global__ __launch_bounds__(256) void turn_kernel(const TurnJobs jobs) {
  constexpr int V = Piece<T>::V, P = 64 / V;  // pieces of a block's row
  __shared__ T tile[64][64 + 4 / sizeof(T)];
  const int64_t blk = blockIdx.x;
  if (blk == 0 && jobs.zero && threadIdx.x < kTrZeroBytes / 16)
    jobs.zero[threadIdx.x] = (u32x4){0u, 0u, 0u, 0u};
  int which = 0;
  while (blk >= jobs.job[which].end) ++which;
  const TurnJob& b = jobs.job[which];
  const int64_t local = blk - (which ? jobs.job[which - 1].end : 0);
  const int across = (b.N + 63) / 64;
  const int n0 = static_cast<int>(local % across) * 64;
  const int64_t k0 = local / across * 64;
  const T* src = static_cast<const T*>(b.src);
  T* dst = static_cast<T*>(b.dst);
  for (int i = threadIdx.x; i < 64 * P; i += 256) {
    const int k = i / P, c = i % P * V;
    u32x4 v = (u32x4){0u, 0u, 0u, 0u};
    if (k0 + k < b.K && n0 + c < b.N) v = load_piece(src + (k0 + k) * b.ld, n0 + c, b.N);
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int q = 0; q < V; ++q) tile[k][c + q] = e[q];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * P; i += 256) {
    const int n = i / P, c = i % P * V;
    if (n0 + n >= b.N) continue;  // kp is a multiple of 128: whole blocks of k
    u32x4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int q = 0; q < V; ++q) e[q] = tile[c + q][n];
    *reinterpret_cast<u32x4*>(dst + (n0 + n) * b.kp + k0 + c) = v;
  }
}

// dst[r][wp] = src[r][w], zeros from w on: up to five matrices in one launch.
struct PadJob {
  const void* src;
  void* dst;
  int64_t end;  // exclusive end of the job's 16-byte pieces
  int w, wp;
};
struct PadJobs {
  PadJob job[5];
  int n;
};
template <typename T>
__global__ __launch_bounds__(256) void pad_rows_kernel(const PadJobs jobs) {
  constexpr int V = Piece<T>::V;
  const int64_t total = jobs.job[jobs.n - 1].end;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    int j = 0;
    while (i >= jobs.job[j].end) ++j;
    const PadJob& b = jobs.job[j];
    const int64_t local = i - (j ? jobs.job[j - 1].end : 0);
    const int per = b.wp / V;
    const int64_t r = local / per;
    const int c = static_cast<int>(local % per) * V;
    *reinterpret_cast<u32x4*>(static_cast<T*>(b.dst) + r * b.wp + c) =
        load_piece(static_cast<const T*>(b.src) + r * b.w, c, b.w);
  }
}

template <typename T>
struct OpOf {
  typedef OpBf16 type;
};
template <>
struct OpOf<float> {
  typedef OpF32 type;
};

template <typename T>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ part, int parts,
                                                            int64_t cells, T* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= cells) return;
  float v = 0.0f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p) v += part[p * cells + i];
  put(out + i, v);
}

// A weight gradient in bf16 operands that needs no slices of the tokens (few
// tokens, or weights with tiles enough): the ring of wgrad_tr_kernel, but each
// tile is written once, in the gradient's type and cropped, instead of as
// fp32 sums that another launch reads again (2048 x 8192: 10 bytes an element
// against 2). Rows of the gradient past M, and columns past N of each half
// (gate and up side by side), are not stored.
struct GradDirect {
  const bf16_t *a, *b;
  int64_t lda, ldb, rows;
  int tiles_m, tiles_n, M, N, half;
  void *out, *out2;
};
template <typename Cfg, typename G>
__global__ __launch_bounds__(Cfg::NT) void grad_direct_kernel(const GradDirect p,
                                                              const bf16_t* __restrict__ zero) {
  constexpr int BM = Cfg::BM, BN = Cfg::BN, NS = Cfg::NS;
  __shared__ __attribute__((aligned(1024))) char smem[NS * Cfg::STAGE];
  const int w = xcd_remap(blockIdx.x, gridDim.x);
  const int mt = w / p.tiles_n, nt = w % p.tiles_n;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  const int a_col = mt * BM, b_col = nt * BN;
  int a_off[2][2], b_off[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a_off[i][h] = tr_frag_off<Cfg::A_PITCH>(wm * 64 + i * 32, lane, h);
      b_off[i][h] = Cfg::A_BYTES + tr_frag_off<Cfg::B_PITCH>(wn * 64 + i * 32, lane, h);
    }
  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
  const int nk = static_cast<int>((p.rows + kTrKT - 1) / kTrKT);
  auto issue = [&](int st) {
    char* buf = smem + (st % NS) * Cfg::STAGE;
    const int64_t row0 = static_cast<int64_t>(st) * kTrKT;
    tr_issue<Cfg::A_CPR, Cfg::A_LOADS>(buf, p.a, p.lda, a_col, row0, p.rows, zero, wave, lane);
    tr_issue<Cfg::B_CPR, Cfg::B_LOADS>(buf + Cfg::A_BYTES, p.b, p.ldb, b_col, row0, p.rows, zero, wave, lane);
  };
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) issue(st);
  for (int s = 0; s < nk; ++s) {
    tr_wait_vm<Cfg::LOADS * (NS - 2)>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    issue(s + NS - 1);
    const uint32_t buf = lds_base + (s % NS) * Cfg::STAGE;
#pragma unroll
    for (int ks = 0; ks < kTrKT / 16; ++ks) {
      uint32_t ad[8];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ad[2 * i + h] = buf + ks * 16 * Cfg::A_PITCH + a_off[i][h];
          ad[4 + 2 * i + h] = buf + ks * 16 * Cfg::B_PITCH + b_off[i][h];
        }
      tr_v4i16 v[8];
      tr_read_kstep(ad, v);
      bf16x8_t af[2], bf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        af[i] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[2 * i], v[2 * i + 1], 0, 1, 2, 3, 4, 5, 6, 7));
        bf[i] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[4 + 2 * i], v[5 + 2 * i], 0, 1, 2, 3, 4, 5, 6, 7));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
    }
  }
  // the loads past the end land before the workgroup's LDS is reused below
  tr_wait_vm<0>();
  __syncthreads();
  // 32 x 32 blocks through LDS of this wave: whole pieces of a row of the
  // gradient per store
  constexpr int kPitch = 36;  // floats
  static_assert(Cfg::NT / 64 * 32 * kPitch * 4 <= NS * Cfg::STAGE, "blocks fit");
  float* block = reinterpret_cast<float*>(smem) + wave * 32 * kPitch;
  const int r32 = lane & 31, g = lane >> 5;
  const bool second = b_col >= p.half;
  G* out = static_cast<G*>(second ? p.out2 : p.out);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int rr = 0; rr < 4; ++rr)
        *reinterpret_cast<float4*>(block + r32 * kPitch + 8 * rr + 4 * g) =
            make_float4(acc[i][j][4 * rr], acc[i][j][4 * rr + 1], acc[i][j][4 * rr + 2], acc[i][j][4 * rr + 3]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int n = b_col - (second ? p.half : 0) + wn * 64 + j * 32 + (lane & 3) * 8;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = (lane >> 2) + 16 * k, m = a_col + wm * 64 + i * 32 + r;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = block[r * kPitch + (lane & 3) * 8 + q];
        if (m < p.M && n < p.N) store8<G, false>(out + static_cast<int64_t>(m) * p.N, n, p.N, v);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// Weight gradients from the slices' partial sums [splits][mp][ld], cropped
// to M x N at column `col` and rounded once: the slices are added in order.
// Up to three gradients in one launch; `wide` ones are fp32 whatever G is.
struct SliceJob {
  const float* part;
  int splits;
  int64_t stride;  // floats between slices
  int64_t ld;
  int M, N;
  void* out;
  int64_t end;     // exclusive end of the job's four-column pieces
  bool wide;
};
struct SliceJobs {
  SliceJob job[3];
  int n;
};
template <typename G>
__global__ __launch_bounds__(256) void slice_sum_kernel(const SliceJobs jobs) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < jobs.job[jobs.n - 1].end;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    int which = 0;
    while (i >= jobs.job[which].end) ++which;
    const SliceJob& b = jobs.job[which];
    const int64_t local = i - (which ? jobs.job[which - 1].end : 0);
    const int per = (b.N + 3) / 4;
    const int64_t m = local / per;
    const int n = static_cast<int>(local % per) * 4;
    const float* src = b.part + m * b.ld + n;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kBatch = 8;
    int s = 0;
    for (; s + kBatch <= b.splits; s += kBatch) {
      float4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) v[u] = *reinterpret_cast<const float4*>(src + (s + u) * b.stride);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        acc.x += v[u].x; acc.y += v[u].y; acc.z += v[u].z; acc.w += v[u].w;
      }
    }
    for (; s < b.splits; ++s) {
      const float4 v = *reinterpret_cast<const float4*>(src + s * b.stride);
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    const float v[4] = {acc.x, acc.y, acc.z, acc.w};
    auto store = [&](auto* out) {
      auto* dst = out + m * b.N + n;
      if (n + 4 <= b.N && b.N % 4 == 0) {
        store4(dst, v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < b.N) put(dst + q, v[q]);
      }
    };
    if (b.wide) store(static_cast<float*>(b.out));
    else store(static_cast<G*>(b.out));
  }
}

template <typename G>
__global__ __launch_bounds__(256) void zero_kernel(G* __restrict__ p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = G{};
}

inline int slices(int64_t rows, int64_t tiles) {
  int64_t k = (512 + tiles - 1) / tiles;
  k = k < 1 ? 1 : (k > 64 ? 64 : k);
  const int64_t most = (rows + 63) / 64;  // a stage of 64 rows each at least
  return static_cast<int>(k > most ? (most < 1 ? 1 : most) : k);
}

// Tile size by the number of tiles: the largest that still gives every CU
// one, since a tile's bytes through a CU's 64-byte-a-clock load path are what
// bounds it (128 x 128: as many clocks as its MFMAs take). 256 x 256 needs a
// long K (stages of 128 bytes) to pay for an epilogue that nothing overlaps:
// with K 512 gate and up of 131072 tokens take 460 us against 418 in 256 x
// 128, with K 2048 to 8192 546 against 630. 16384 tokens, 512 x 1024: gate and
// up 63 us in 128 x 128, 55 in 256 x 128. fp32 (its MFMAs take 16 times as
// long for the same bytes) keeps to 128 x 128 at most. Few rows do not fill
// the larger ones: 128 tokens, 4096 x 16384, forward and backward: 482 us in 64
// x 64 tiles, 594 without this rule.
enum TileSize { kSmall, kMid, kTall, kBig };
inline TileSize tile_of(size_t elem, int64_t M, int64_t cols, int64_t stages) {
  auto count = [&](int m, int n) { return (M + m - 1) / m * ((cols + n - 1) / n); };
  if (M <= (elem == 2 ? 128 : 64)) return kSmall;
  if (elem == 2 && stages >= 16 && count(256, 256) >= kCUs) return kBig;
  if (elem == 2 && count(256, 128) >= kCUs) return kTall;
  return count(128, 128) >= kCUs ? kMid : kSmall;
}
// Slices of K of a plain product: two workgroups a CU, four stages each at
// least (777 x 500 with K 2048 in fp32: 104 tiles of 64 x 64).
inline int parts_of(size_t elem, int64_t M, int64_t N, int64_t stages) {
  if (tile_of(elem, M, N, stages) != kSmall) return 1;
  const int64_t tiles = (M + 63) / 64 * ((N + 63) / 64);
  if (tiles == 0) return 1;  // no tokens
  int64_t k = tiles < kCUs ? 2 * kCUs / tiles : 1;
  if (k > stages / 4) k = stages / 4;
  return static_cast<int>(k < 1 ? 1 : (k > 16 ? 16 : k));
}

inline unsigned blocks_for(int64_t items) {
  const int64_t b = (items + 255) / 256;
  return static_cast<unsigned>(b < 1 ? 1 : (b > 8192 ? 8192 : b));
}

template <typename T>
void turn(const char* name, const TurnJobs& jobs, hipStream_t s) {
  MOE_LAUNCH(name, turn_kernel<T>, dim3(static_cast<unsigned>(jobs.job[jobs.n - 1].end)), dim3(256), 0, s, jobs);
}

// The matrix itself, or the place of its copy with rows padded to a multiple
// of 128, which `jobs` then makes.
template <typename T>
const void* padded(PadJobs& jobs, const void* src, char* dst, int64_t rows, int w) {
  const int wp = static_cast<int>(pad128(w));
  if (w == wp) return src;
  const int64_t start = jobs.n ? jobs.job[jobs.n - 1].end : 0;
  jobs.job[jobs.n++] = PadJob{src, dst, start + rows * (wp / Piece<T>::V), w, wp};
  return dst;
}
template <typename T>
void pad(const char* name, const PadJobs& jobs, hipStream_t s) {
  if (jobs.n)
    MOE_LAUNCH(name, pad_rows_kernel<T>, dim3(blocks_for(jobs.job[jobs.n - 1].end)), dim3(256),
               0, s, jobs);
}

template <typename T>
MmArgs rows_of(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t M, int N, int64_t K) {
  MmArgs p{};
  p.a = static_cast<const char*>(a);
  p.a_pitch = lda * static_cast<int64_t>(sizeof(T));
  p.b = static_cast<const char*>(b);
  p.b_pitch = ldb * static_cast<int64_t>(sizeof(T));
  p.nk = static_cast<int>(K * static_cast<int64_t>(sizeof(T)) / 128);
  p.M = M;
  p.N = N;
  return p;
}

template <typename G>
void grad_direct(const char* name, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t mp,
                 int64_t np, int64_t rows, int M, int N, int64_t half, void* out, void* out2,
                 const void* zero, hipStream_t s) {
  GradDirect p{static_cast<const bf16_t*>(a), static_cast<const bf16_t*>(b), lda, ldb, rows, 0,
               static_cast<int>(np / 128), M, N, static_cast<int>(half), out, out2};
  // as wgrad_tr: 256-row tiles where they divide and still give every CU one
  const bool tall = mp % 256 == 0 && mp / 256 * (np / 128) >= kCUs;
  p.tiles_m = static_cast<int>(mp / (tall ? 256 : 128));
  const dim3 grid(p.tiles_m * p.tiles_n);
  const bf16_t* z = static_cast<const bf16_t*>(zero);
  if (tall)
    MOE_LAUNCH(name, (grad_direct_kernel<TrCfg<256, 3>, G>), grid, dim3(512), 0, s, p, z);
  else
    MOE_LAUNCH(name, (grad_direct_kernel<TrCfg<128, 4>, G>), grid, dim3(256), 0, s, p, z);
}

// Partial sums of a^T b over the slices of the rows, [splits][mp][np] (bf16).
template <typename T>
void grad_slices(const char* name, const void* a, int64_t lda, const void* b, int64_t ldb,
                 int64_t mp, int64_t np, int64_t rows, int splits, float* part, const void* zero,
                 hipStream_t s) {
  WgradArgs w{};
  w.a = a;
  w.lda = lda;
  w.b = b;
  w.ldb = ldb;
  w.M = static_cast<int>(mp);
  w.N = static_cast<int>(np);
  w.rows_total = rows;
  w.splits = splits;
  w.c = part;
  w.nsplit = w.N;
  w.ldc = np;
  w.c_group_stride = mp * np;
  wgrad_tr<true>(name, w, splits, static_cast<const bf16_t*>(zero), s);
}

}  // namespace moe
