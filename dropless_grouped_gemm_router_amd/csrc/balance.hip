// Balance loss and z loss of the router, with the experts' loads, forward and
// backward.
//
//   l = x W, p = softmax(l), lse = log sum exp(l); over the n kept tokens
//   loss = c1 sum_e f_e mean(p_e) + c2 mean(lse^2),  f = counts / (n k), c1 = balance E
//   dl = p (c1 (f - sum_j f_j p_j) + 2 c2 lse) / n,  dx = dl W^T, dW = x^T dl
//
// Bound by reading x once in the forward, and in the backward by reading x and
// writing dx. The gradient by the logits needs the counts, which the routing
// already fixes, and nothing else of the batch: a first launch counts, the pass
// over x then makes p and dl while the logits are in registers, and the backward
// starts from dl (fp32: a quarter of x's bytes at 64 experts of 512 columns in bf16)
// instead of multiplying by W again.
//
// Precision. bf16: x is exact in bf16 and W is the sum of three bf16 numbers, all
// of fp32's 24 bits, so three bf16 MFMAs make the logits as fp32 products would,
// at a fifth of fp32 MFMAs' time. In the backward dl is the sum of three for dW, x
// being exact, and of two for dx, as W is there: dx is off by 2^-16 before it is
// rounded to bf16. fp32: fp32 MFMAs throughout.
#include "block.h"
#include "skinny.h"

namespace moe {

namespace {

constexpr int kCountBlocks = 64, kCountThreads = 1024;

// Experts are padded to 32 or 64: EB blocks of 32.
inline int expert_blocks(int E) { return E <= 32 ? 1 : 2; }

struct BalArgs {
  int64_t T;
  int E, k, d;
  float c1, c2;           // balance * E, 2 * z
  const uint8_t* mask;    // or null
  const int32_t* parts;   // [kCountBlocks][64] counts by expert, [kCountBlocks] kept tokens
  int count_blocks;
  float* stats;           // [workgroups][65]: sums of p by expert, of lse^2
  // few tokens, inference (nothing waits for the counts): the logits' workgroups
  // count their own tokens and split W themselves; else null
  const int32_t* idx;
  int32_t* own;           // [workgroups][65]: counts by expert, kept tokens
  const float* w;
};

// ---------------------------------------------------- counts, and W in operands

// W as the logits' first MFMA operand: 16 bytes a lane, lane l holding expert
// 32 eb + l % 32 for k 8 (l / 32) .. + 7 of a step of 16 (fp32: 4 (l / 32) .. + 3
// of 8); bf16: three numbers that add up to W, in three such pieces.
template <typename T>
__device__ void split_router(const float* __restrict__ w, int d, int E, int EB, u32x4* __restrict__ out, int i) {
  constexpr int V = Piece<T>::V, S = sizeof(T) == 2 ? 3 : 1;
  const int lane = i % 64, eb = i / 64 % EB, step = i / 64 / EB;
  const int e = 32 * eb + lane % 32, k0 = step * 2 * V + V * (lane / 32);
  if (k0 >= d) return;
  float v[V];
#pragma unroll
  for (int q = 0; q < V; ++q) v[q] = w[static_cast<int64_t>(k0 + q) * E + (e < E ? e : 0)];  // without a branch
#pragma unroll
  for (int q = 0; q < V; ++q) v[q] = e < E ? v[q] : 0.0f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const u32x4 p = Piece<T>::narrow(v);
    out[((static_cast<int64_t>(step) * EB + eb) * S + s) * 64 + lane] = p;
    float back[V];
    Piece<T>::widen(p, back);
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] -= back[q];
  }
}

// W as the first operand of dx = dl W^T, for the backward: 64 columns of x at a
// time, four fragments of 16, 16 bytes a lane.
// bf16: fragment j's row i is column 32 (j / 2) + 8 (i / 4) + 4 (j % 2) + i % 4, so
// that a lane ends up with eight consecutive columns of two fragments; lane l
// holds row l % 16 for experts 32 b + 8 (l / 16) .. + 7, the number and what is left
// of it. fp32: row i is column 16 j + i, experts 16 b + 4 (l / 16) .. + 3. Pieces
// [columns / 64][j][b][2 or 1][lane].
template <typename T>
__device__ void turn_router(const float* __restrict__ w, int d, int E, int EB, u32x4* __restrict__ out, int i) {
  constexpr bool kHalves = sizeof(T) == 2;
  constexpr int V = Piece<T>::V;
  const int lane = i % 64, BN = kHalves ? EB : 2 * EB, b = i / 64 % BN, j = i / 64 / BN % 4;
  const int c0 = i / 256 / BN * 64, r = lane & 15, g = lane >> 4;
  if (c0 >= d) return;
  const int col = c0 + (kHalves ? 32 * (j / 2) + 8 * (r / 4) + 4 * (j % 2) + r % 4 : 16 * j + r);
  float v[V];
#pragma unroll
  for (int q = 0; q < V; ++q) {
    const int e = (kHalves ? 32 * b + 8 * g : 16 * b + 4 * g) + q;
    v[q] = w[static_cast<int64_t>(col) * E + (e < E ? e : 0)];
  }
#pragma unroll
  for (int q = 0; q < V; ++q)
    if ((kHalves ? 32 * b + 8 * g : 16 * b + 4 * g) + q >= E) v[q] = 0.0f;
  const u32x4 p = Piece<T>::narrow(v);
  if (!kHalves) {
    out[i] = p;
    return;
  }
  float back[V];
  Piece<T>::widen(p, back);
#pragma unroll
  for (int q = 0; q < V; ++q) v[q] -= back[q];
  out[static_cast<int64_t>(i / 64) * 128 + lane] = p;
  out[static_cast<int64_t>(i / 64) * 128 + 64 + lane] = Piece<T>::narrow(v);
}

// Counts by expert of the token-slots of tokens t0 .. t1 - 1 that are kept, into
// `hist` (LDS) by the calling threads, this one the i-th of `threads`; hist[64]:
// the kept tokens. Entries that are no expert are left out.
__device__ __forceinline__ void count_slots(const BalArgs& a, const int32_t* __restrict__ idx, int64_t t0, int64_t t1,
                                            int i, int threads, int* hist) {
  constexpr int kBatch = 8;
  const int64_t s1 = t1 * a.k;
  for (int64_t s0 = t0 * a.k + i; s0 < s1; s0 += kBatch * threads) {
    int e[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t s = s0 + u * threads;
      e[u] = idx[s < s1 ? s : s0];
    }
    if (a.mask) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int64_t s = s0 + u * threads;
        // slots are below 2^31
        if (!a.mask[static_cast<uint32_t>(s < s1 ? s : s0) / static_cast<uint32_t>(a.k)]) e[u] = -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (s0 + u * threads < s1 && static_cast<unsigned>(e[u]) < static_cast<unsigned>(a.E)) atomicAdd(hist + e[u], 1);
  }
  int kept = 0;
  if (a.mask) {
    for (int64_t t = t0 + i; t < t1; t += threads) kept += a.mask[t] != 0;
  } else if (i == 0) {
    kept = static_cast<int>(t1 - t0);
  }
  if (kept) atomicAdd(hist + 64, kept);
}

// Workgroups below count_blocks count their share of the tokens; the others
// lay W out, for the backward too where there is a place for it.
template <typename T>
__global__ __launch_bounds__(kCountThreads) void balance_count_kernel(const BalArgs a,
                                                                     const int32_t* __restrict__ idx,
                                                                     const float* __restrict__ w, int EB,
                                                                     u32x4* __restrict__ wf,
                                                                     u32x4* __restrict__ wb,
                                                                     int32_t* __restrict__ parts) {
  constexpr int kWaves = kCountThreads / 64;
  __shared__ int hist[kWaves][65];
  if (static_cast<int>(blockIdx.x) >= a.count_blocks) {
    // as many pieces for the backward as for the logits
    const int i = (blockIdx.x - a.count_blocks) * kCountThreads + threadIdx.x;
    const int pieces = a.d / (2 * Piece<T>::V) * EB * 64;
    if (i < pieces) split_router<T>(w, a.d, a.E, EB, wf, i);
    else if (wb) turn_router<T>(w, a.d, a.E, EB, wb, i - pieces);
    return;
  }
  for (int i = threadIdx.x; i < kWaves * 65; i += kCountThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int64_t t0 = a.T * blockIdx.x / a.count_blocks, t1 = a.T * (blockIdx.x + 1) / a.count_blocks;
  count_slots(a, idx, t0, t1, threadIdx.x, kCountThreads, hist[threadIdx.x >> 6]);
  __syncthreads();
  if (threadIdx.x < 65) {
    int v = 0;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) v += hist[u][threadIdx.x];
    parts[threadIdx.x < 64 ? blockIdx.x * 64 + threadIdx.x : kCountBlocks * 64 + blockIdx.x] = v;
  }
}

// ------------------------------------------------------------------- logits

__device__ __forceinline__ bool kept_token(const BalArgs& a, int64_t t) {
  return t < a.T && (!a.mask || a.mask[t]);
}

template <typename T>
struct BalOp;
template <>
struct BalOp<bf16_t> {
  static constexpr int S = 3;
  __device__ static void step(const u32x4 (&w)[3], const u32x4& x, f32x16_t& acc) {
    const bf16x8_t xv = __builtin_bit_cast(bf16x8_t, x);
    // the smallest products first
#pragma unroll
    for (int s = 2; s >= 0; --s)
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, w[s]), xv, acc, 0, 0, 0);
  }
};
template <>
struct BalOp<float> {
  static constexpr int S = 1;
  __device__ static void step(const u32x4 (&w)[1], const u32x4& x, f32x16_t& acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w[0][e]), __uint_as_float(x[e]), acc, 0, 0, 0);
  }
};

// The kept gradient by the logits of eight experts of a token (one lane) or,
// in fp32, of four; the two lanes of a token hold experts in turns of four.
__device__ __forceinline__ void store_dl(float* row, int eb, int g, const float (&dl)[16]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
    store4(row + 32 * eb + 8 * r + 4 * g, dl[4 * r], dl[4 * r + 1], dl[4 * r + 2], dl[4 * r + 3]);
}

// The same of eight consecutive experts of token t in one lane.
__device__ __forceinline__ void store_dl8(float* saved, int64_t t, int EP, int e0, const float (&dl)[8]) {
  float* row = saved + t * EP + e0;
  store4(row, dl[0], dl[1], dl[2], dl[3]);
  store4(row + 4, dl[4], dl[5], dl[6], dl[7]);
}

// Logits of 32 tokens from row0 on over lines first, first + step, ...: MFMA 32x32
// with W first, so a lane ends up with 16 EB experts of token lane % 32 and the lane
// 32 further with the others. x goes from memory straight into operands (a row's
// 128 bytes over four loads), W's operands come from the caches; both are loaded
// a line ahead, W's each into the place of the one that has just been multiplied.
// kRaw: W as it is, split on the way into the products.
template <typename T, int EB, bool kRaw>
__device__ __forceinline__ void logits(const BalArgs& a, const T* __restrict__ x, const u32x4* __restrict__ wf,
                                       int64_t row0, int first, int step, f32x16_t (&acc)[EB]) {
  constexpr int S = BalOp<T>::S, kLine = 128 / sizeof(T), V = Piece<T>::V;
  const int lane = threadIdx.x & 63, g = lane >> 5, r32 = lane & 31;
#pragma unroll
  for (int b = 0; b < EB; ++b)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[b][q] = 0.0f;
  const int lines = a.d / kLine;
  if (first >= lines) return;
  const int64_t r = row0 + r32;
  const T* row = x + (r < a.T ? r : a.T - 1) * a.d + g * (16 / static_cast<int>(sizeof(T)));
  u32x4 xv[2][4], wv[kRaw ? 1 : 4][EB][S];
  float raw[kRaw ? 4 : 1][EB][V];
  auto load_x = [&](int set, int line) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      xv[set][q] = *reinterpret_cast<const u32x4*>(row + line * kLine + q * (kLine / 4));
  };
  auto load_w = [&](int q, int line) {
#pragma unroll
    for (int b = 0; b < EB; ++b) {
      if constexpr (kRaw) {
        const int e = 32 * b + r32;
        const float* p = a.w + static_cast<int64_t>((line * 4 + q) * 2 * V + V * g) * a.E + (e < a.E ? e : 0);
#pragma unroll
        for (int j = 0; j < V; ++j) raw[q][b][j] = p[static_cast<int64_t>(j) * a.E];
      } else {
#pragma unroll
        for (int s = 0; s < S; ++s)
          wv[q][b][s] = wf[((static_cast<int64_t>(line * 4 + q)) * EB * S + b * S + s) * 64 + lane];
      }
    }
  };
  auto multiply = [&](int set, bool more, int next) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int b = 0; b < EB; ++b) {
        if constexpr (kRaw) {
          // experts past E take the first's weights; nothing reads their logits
#pragma unroll
          for (int s = 0; s < S; ++s) {
            wv[0][b][s] = Piece<T>::narrow(raw[q][b]);
            float back[V];
            Piece<T>::widen(wv[0][b][s], back);
#pragma unroll
            for (int j = 0; j < V; ++j) raw[q][b][j] -= back[j];
          }
        }
        BalOp<T>::step(wv[kRaw ? 0 : q][b], xv[set][q], acc[b]);
      }
      if (more) load_w(q, next);
    }
  };
  load_x(0, first);
#pragma unroll
  for (int q = 0; q < 4; ++q) load_w(q, first);
  for (int line = first; line < lines; line += 2 * step) {
    const int n1 = line + step, n2 = line + 2 * step;
    if (n1 < lines) load_x(1, n1);
    multiply(0, n1 < lines, n1);
    if (n1 >= lines) break;
    if (n2 < lines) load_x(0, n2);
    multiply(1, n2 < lines, n2);
  }
}

// The same of 32 RT tokens a wave, all lines (an even number of them: d_model is a
// multiple of 128), with W's operands of a line going through LDS once for the NW
// waves of a workgroup: [2][4 EB S] pieces of 1 KB in turns, the next line's on
// their way in registers while a line is multiplied. Where every wave read W
// through the vector cache, 24 KB a line beside its own 8 KB of x, 131072 tokens
// took 47 us; so 33. No conditions on the loads: they cost the loop their order
// (104 us).
template <typename T, int EB, int RT, int NW>
__device__ __forceinline__ void logits_shared(const BalArgs& a, const T* __restrict__ x,
                                              const u32x4* __restrict__ wf, int64_t row0, u32x4* lds,
                                              f32x16_t (&acc)[RT][EB]) {
  constexpr int S = BalOp<T>::S, kLine = 128 / sizeof(T), kPieces = 4 * EB * S, kEach = kPieces / NW;
  static_assert(kPieces % NW == 0, "pieces");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, r32 = lane & 31;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int b = 0; b < EB; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][b][q] = 0.0f;
  const int lines = a.d / kLine;
  const T* rows[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = row0 + 32 * i + r32;
    rows[i] = x + (r < a.T ? r : a.T - 1) * a.d + g * (16 / static_cast<int>(sizeof(T)));
  }
  u32x4 xv[2][RT][4], w[kEach];
  auto load_x = [&](int set, int line) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        xv[set][i][q] = *reinterpret_cast<const u32x4*>(rows[i] + line * kLine + q * (kLine / 4));
  };
  auto load_w = [&](int line) {
#pragma unroll
    for (int u = 0; u < kEach; ++u) w[u] = wf[(static_cast<int64_t>(line) * kPieces + wave * kEach + u) * 64 + lane];
  };
  auto store_w = [&](int set) {
#pragma unroll
    for (int u = 0; u < kEach; ++u) lds[(set * kPieces + wave * kEach + u) * 64 + lane] = w[u];
  };
  auto multiply = [&](int set) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int b = 0; b < EB; ++b) {
        u32x4 f[S];
#pragma unroll
        for (int s = 0; s < S; ++s) f[s] = lds[(set * kPieces + (q * EB + b) * S + s) * 64 + lane];
#pragma unroll
        for (int i = 0; i < RT; ++i) BalOp<T>::step(f, xv[set][i][q], acc[i][b]);
      }
  };
  load_w(0);
  load_x(0, 0);
  store_w(0);
  __syncthreads();
  int line = 0;
  for (; line + 2 < lines; line += 2) {
    load_w(line + 1);
    load_x(1, line + 1);
    multiply(0);
    store_w(1);
    __syncthreads();
    load_w(line + 2);
    load_x(0, line + 2);
    multiply(1);
    store_w(0);
    __syncthreads();
  }
  load_w(line + 1);
  load_x(1, line + 1);
  multiply(0);
  store_w(1);
  __syncthreads();
  multiply(1);
}

// Counts of the experts and the number of kept tokens from the count blocks',
// by all NT threads: the loads early, the sums when they are needed.
template <int NT>
struct Tallies {
  static constexpr int kWaves = NT / 64, kEach = kCountBlocks / kWaves;
  static_assert(kCountBlocks == 64 && kCountBlocks % kWaves == 0, "a lane has a block's kept tokens");
  int v[kEach], n;
  __device__ void load(const BalArgs& a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int p = wave + u * kWaves;
      v[u] = a.parts[(p < a.count_blocks ? p : 0) * 64 + lane];
    }
    n = a.parts[kCountBlocks * 64 + (lane < a.count_blocks ? lane : 0)];
  }
  // sums: [kWaves][64], whole after the caller's next barrier; returns n (at most
  // 2^31, exact in every lane).
  __device__ int put(const BalArgs& a, int (*sums)[64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int c = 0;
#pragma unroll
    for (int u = 0; u < kEach; ++u) c += wave + u * kWaves < a.count_blocks ? v[u] : 0;
    sums[wave][lane] = c;
    int k = lane < a.count_blocks ? n : 0;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) k += __shfl_xor(k, o);
    return k;
  }
  __device__ static int count(const int (*sums)[64], int e) {
    int c = 0;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) c += sums[u][e];
    return c;
  }
  __device__ static float share(const BalArgs& a, const int (*sums)[64], int e, int n) {
    return n > 0 ? static_cast<float>(count(sums, e)) / (static_cast<float>(n) * static_cast<float>(a.k)) : 0.0f;
  }
};
__device__ __forceinline__ float one_over(int n) { return n > 0 ? 1.0f / static_cast<float>(n) : 0.0f; }

// Many tokens: 64 a wave, whose softmax stays in the registers that the
// products leave it in. 131072 tokens of 64 experts x 512 bf16: 33 us for 134 MB (4.1
// TB/s; MFMA 40% busy, three bf16 products for one).
template <typename T, int EB>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void balance_logits_kernel(const BalArgs a, const T* __restrict__ x, const u32x4* __restrict__ wf,
                           float* __restrict__ saved) {
  constexpr int EP = 32 * EB, RT = 2, NW = 4;
  __shared__ float sums[NW][EP + 1];
  __shared__ int tallies[NW][64];
  __shared__ __attribute__((aligned(16))) float share[64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, r32 = lane & 31;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * NW + wave) * 32 * RT;
  float inv_n = 0.0f;
  if (saved) {
    Tallies<64 * NW> t;
    t.load(a);
    const int n = t.put(a, tallies);
    inv_n = one_over(n);
    __syncthreads();
    if (threadIdx.x < 64) share[threadIdx.x] = t.share(a, tallies, threadIdx.x, n);
    // the products' barriers lie before the shares' use
  }
  f32x16_t acc[RT][EB];
  __shared__ u32x4 lds[2 * 4 * EB * BalOp<T>::S * 64];
  logits_shared<T, EB, RT, NW>(a, x, wf, row0, lds, acc);

  float psum[EB][16], zsum = 0.0f;
#pragma unroll
  for (int b = 0; b < EB; ++b)
#pragma unroll
    for (int q = 0; q < 16; ++q) psum[b][q] = 0.0f;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t t = row0 + 32 * i + r32;
    const bool keep = kept_token(a, t);
    float other, most = -__builtin_inff();
#pragma unroll
    for (int b = 0; b < EB; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (32 * b + 8 * (q / 4) + 4 * g + q % 4 < a.E) most = fmaxf(most, acc[i][b][q]);
    most = lane32(most, &other);
    most = fmaxf(most, other);
    float p[EB][16], total = 0.0f;
#pragma unroll
    for (int b = 0; b < EB; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        p[b][q] = 32 * b + 8 * (q / 4) + 4 * g + q % 4 < a.E ? __expf(acc[i][b][q] - most) : 0.0f;
        total += p[b][q];
      }
    total = lane32(total, &other);
    total += other;
    const float inv = 1.0f / total, lse = most + logf(total);
#pragma unroll
    for (int b = 0; b < EB; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        p[b][q] *= inv;
        if (keep) psum[b][q] += p[b][q];
      }
    if (keep && g == 0) zsum += lse * lse;
    if (!saved) continue;
    float f[EB][16], inner = 0.0f;
#pragma unroll
    for (int b = 0; b < EB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 v = *reinterpret_cast<const float4*>(share + 32 * b + 8 * r + 4 * g);
        f[b][4 * r] = v.x; f[b][4 * r + 1] = v.y; f[b][4 * r + 2] = v.z; f[b][4 * r + 3] = v.w;
      }
#pragma unroll
    for (int b = 0; b < EB; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q) inner = __builtin_fmaf(f[b][q], p[b][q], inner);
    inner = lane32(inner, &other);
    inner += other;
    const float zed = a.c2 * lse;
#pragma unroll
    for (int b = 0; b < EB; ++b) {
      float dl[16];
#pragma unroll
      for (int q = 0; q < 16; ++q)
        dl[q] = keep ? p[b][q] * __builtin_fmaf(a.c1, f[b][q] - inner, zed) * inv_n : 0.0f;
      if (t < a.T) store_dl(saved + t * EP, b, g, dl);
    }
  }
  // sums over the wave's 32 lanes, then over the waves
#pragma unroll
  for (int b = 0; b < EB; ++b)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float other, v = row16_sum(psum[b][q]);
      v = lane16(v, &other);
      v += other;
      if (r32 == 0) sums[wave][32 * b + 8 * (q / 4) + 4 * g + q % 4] = v;
    }
  zsum = wave_sum(zsum);
  if (lane == 0) sums[wave][EP] = zsum;
  __syncthreads();
  if (threadIdx.x <= EP) {
    float v = 0.0f;
#pragma unroll
    for (int u = 0; u < NW; ++u) v += sums[u][threadIdx.x];
    // the last one is the sum of lse^2
    a.stats[static_cast<int64_t>(blockIdx.x) * 65 + (static_cast<int>(threadIdx.x) == EP ? 64 : threadIdx.x)] = v;
  }
}

// Fewer tokens: 32 a workgroup, whose KS waves share the columns. Their sums go
// through LDS, from where the softmax takes eight experts of a token a lane,
// 4 EB lanes to a token, so that all waves work on it.
template <typename T, int EB, int KS, bool kRaw>
__global__ __launch_bounds__(64 * KS) void balance_logits_few_kernel(const BalArgs a, const T* __restrict__ x,
                                                                     const u32x4* __restrict__ wf,
                                                                     float* __restrict__ saved) {
  constexpr int EP = 32 * EB, L = 4 * EB, kTokens = 64 / L, kPitch = 66;
  constexpr int kUsed = 32 / kTokens < KS ? 32 / kTokens : KS, kPasses = 32 / kTokens / kUsed;
  __shared__ float part[KS][16 * EB * kPitch];
  __shared__ float sums[KS][EP + 1];
  __shared__ int tallies[KS][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 32;
  __shared__ int hist[65];
  if constexpr (kRaw) {
    if (threadIdx.x < 65) hist[threadIdx.x] = 0;
    __syncthreads();
    count_slots(a, a.idx, row0, row0 + 32 < a.T ? row0 + 32 : a.T, threadIdx.x, 64 * KS, hist);
  }
  Tallies<64 * KS> counts;
  if (saved) counts.load(a);
  f32x16_t acc[EB];
  logits<T, EB, kRaw>(a, x, wf, row0, wave, KS, acc);
  const int n = saved ? counts.put(a, tallies) : 0;
#pragma unroll
  for (int b = 0; b < EB; ++b)
#pragma unroll
    for (int q = 0; q < 16; ++q) part[wave][(b * 16 + q) * kPitch + lane] = acc[b][q];
  __syncthreads();
  // lane: eight experts e0.. of a token
  const int m = lane % L, e0 = 8 * m;
  float psum[8], zsum = 0.0f, f[8];
  const float inv_n = one_over(n);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    psum[q] = 0.0f;
    f[q] = saved ? counts.share(a, tallies, e0 + q, n) : 0.0f;
  }
  // a sum over the lanes of a token, and over those of an octet of experts
  auto over_token = [&](float v) {
    v += dpp<0xb1>(v);  // lane ^ 1
    v += dpp<0x4e>(v);  // lane ^ 2
    if (L == 8) v += dpp<0x141>(v);  // half row mirrored
    return v;
  };
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    if (wave >= kUsed) break;
    const int tok = (pass * kUsed + wave) * kTokens + lane / L;
    const int64_t t = row0 + tok;
    const bool keep = kept_token(a, t);
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // expert e0 + q of the products' layout: register 16 (m / 4) + 4 (m % 4) + q % 4, lane 32 (q / 4) + tok
      const int at = (4 * m + q % 4) * kPitch + 32 * (q / 4) + tok;
      v[q] = part[0][at];
#pragma unroll
      for (int s = 1; s < KS; ++s) v[q] += part[s][at];
    }
    float most = -__builtin_inff();
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (e0 + q < a.E) most = fmaxf(most, v[q]);
    most = fmaxf(most, dpp<0xb1>(most));
    most = fmaxf(most, dpp<0x4e>(most));
    if (L == 8) most = fmaxf(most, dpp<0x141>(most));
    float p[8], total = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      p[q] = e0 + q < a.E ? __expf(v[q] - most) : 0.0f;
      total += p[q];
    }
    total = over_token(total);
    const float inv = 1.0f / total, lse = most + logf(total);
    float inner = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      p[q] *= inv;
      if (keep) psum[q] += p[q];
      inner = __builtin_fmaf(f[q], p[q], inner);
    }
    if (keep && m == 0) zsum += lse * lse;
    if (!saved) continue;
    inner = over_token(inner);
    const float zed = a.c2 * lse;
    float dl[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) dl[q] = keep ? p[q] * __builtin_fmaf(a.c1, f[q] - inner, zed) * inv_n : 0.0f;
    if (t < a.T) store_dl8(saved, t, EP, e0, dl);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float other, s = psum[q];
    if (L == 4) s += dpp<0x141>(dpp<0x1b>(s));  // lane ^ 4: quad reversed, half row mirrored
    s += dpp<0x128>(s);  // lane ^ 8: row rotated by eight
    s = lane16(s, &other);
    s += other;
    s = lane32(s, &other);
    s += other;
    if (lane < L) sums[wave][e0 + q] = s;
  }
  zsum = wave_sum(zsum);
  if (lane == 0) sums[wave][EP] = zsum;
  __syncthreads();
  if (threadIdx.x <= EP) {
    float v = 0.0f;
#pragma unroll
    for (int u = 0; u < kUsed; ++u) v += sums[u][threadIdx.x];
    a.stats[static_cast<int64_t>(blockIdx.x) * 65 + (static_cast<int>(threadIdx.x) == EP ? 64 : threadIdx.x)] = v;
  }
  if (kRaw && threadIdx.x < 65) a.own[static_cast<int64_t>(blockIdx.x) * 65 + threadIdx.x] = hist[threadIdx.x];
}

// The results from the workgroups' sums, and from their counts or the count
// blocks': 16 threads to an expert.
__global__ __launch_bounds__(1024) void balance_loss_kernel(const BalArgs a, int groups, float balance, float z,
                                                            int32_t* __restrict__ counts,
                                                            float* __restrict__ mean_prob,
                                                            float* __restrict__ loss) {
  __shared__ float sums[16][64], zeds[16];
  __shared__ int tallies[16][64], kept[16];
  const int e = threadIdx.x % 64, j = threadIdx.x / 64;
  Tallies<1024> t;
  if (!a.own) t.load(a);
  float v = 0.0f, zed = 0.0f;
  int c = 0, k = 0;
  if (a.own) {
#pragma unroll 16
    for (int p = j; p < groups; p += 16) c += a.own[static_cast<int64_t>(p) * 65 + e];
    for (int p = threadIdx.x; p < groups; p += 1024) k += a.own[static_cast<int64_t>(p) * 65 + 64];
  }
  if (e < a.E) {
#pragma unroll 16
    for (int p = j; p < groups; p += 16) v += a.stats[static_cast<int64_t>(p) * 65 + e];
  }
  for (int p = threadIdx.x; p < groups; p += 1024) zed += a.stats[static_cast<int64_t>(p) * 65 + 64];
  sums[j][e] = v;
  zed = wave_sum(zed);
  if (e == 0) zeds[j] = zed;
  int n = 0;
  if (a.own) {
    tallies[j][e] = c;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) k += __shfl_xor(k, o);
    if (e == 0) kept[j] = k;
  } else {
    n = t.put(a, tallies);
  }
  __syncthreads();
  if (j) return;
  float p = 0.0f, zz = 0.0f;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    p += sums[u][e];
    zz += zeds[u];
    if (a.own) n += kept[u];
  }
  p *= one_over(n);
  zz *= one_over(n);
  if (e < a.E) {
    mean_prob[e] = p;
    counts[e] = t.count(tallies, e);
  }
  const float total = static_cast<float>(a.E) * wave_sum(e < a.E ? t.share(a, tallies, e, n) * p : 0.0f);
  if (e == 0) {
    loss[0] = __builtin_fmaf(balance, total, z * zz);
    loss[1] = total;
    loss[2] = zz;
  }
}

// ----------------------------------------------------------------- backward

// dx and partial sums of dW for 128 columns: two waves side by side, four pairs
// of them over the tokens, 32 at a time. dl of these goes through LDS, where
// each wave takes it twice: token rows for dx = dl W^T (W of its 64 columns stays
// in registers) and, turned, expert rows for dW = dl^T x, whose 64 x 64 sums stay
// in registers too. x comes from memory straight into operands (skinny.h).
constexpr int kGradCols = 128, kGradSets = 4, kGradThreads = 512;

struct BalGradArgs {
  int64_t T;
  int d;
  int ranges;          // of the tokens: a partial dW each
  const uint8_t* mask;
  const float* gloss;  // or null
  bool add;
};

// W of a wave's 64 columns (turn_router) and dl's LDS rows.
template <typename T, int EB>
struct BalGrad;

template <int EB>
struct BalGrad<bf16_t, EB> {
  // dl goes in as three bf16 numbers, each what the ones before it round away. dx,
  // rounded to bf16, takes two; dW takes all (two, off by 2^-18 at most, made it
  // 1.5e-6 to 2.9e-6 off in the 2-norm). ROW: bytes of a token's dl in memory, BYTES: here.
  static constexpr int EP = 32 * EB, ROW = 4 * EP, BYTES = 6 * EP;
  u32x4 hi[4][EB], lo[4][EB];
  __device__ void load(const u32x4* wb, int c0, int lane) {
    const u32x4* p = wb + static_cast<int64_t>(c0 / 64) * 4 * EB * 128 + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < EB; ++b) {
        hi[j][b] = p[(j * EB + b) * 128];
        lo[j][b] = p[(j * EB + b) * 128 + 64];
      }
  }
  // 16-byte chunk c of number `part` of token row r: spread over the banks, the same
  // way in the three
  __device__ static int at(int part, int r, int c) {
    return part * 64 * EP + r * 2 * EP + ((c ^ (r & (EP / 8 - 1))) << 4);
  }
  // dl of experts 4 c .. + 3 of token row r.
  __device__ static void put_dl(char* lds, int r, int c, const u32x4& dl) {
    float v[4];
    Piece<float>::widen(dl, v);
    u32x2 part[3];
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      part[u] = (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      v[0] -= bf16lo(part[u][0]);
      v[1] -= bf16hi(part[u][0]);
      v[2] -= bf16lo(part[u][1]);
      v[3] -= bf16hi(part[u][1]);
    }
#pragma unroll
    for (int u = 0; u < 3; ++u) *reinterpret_cast<u32x2*>(lds + at(u, r, c >> 1) + (c & 1) * 8) = part[u];
  }
  // dx of 16 tokens (rows r0..): v[h] are columns c0 + 32 h + 8 (lane / 16) .. + 7
  // of token lane % 16.
  __device__ void dx(const char* lds, int r0, int lane, float (&v)[2][8]) const {
    const int r = r0 + (lane & 15), g = lane >> 4;
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < EB; ++b) {
      const bf16x8_t dh = *reinterpret_cast<const bf16x8_t*>(lds + at(0, r, 4 * b + g));
      const bf16x8_t dlo = *reinterpret_cast<const bf16x8_t*>(lds + at(1, r, 4 * b + g));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, lo[j][b]), dh, acc[j], 0, 0, 0);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, hi[j][b]), dlo, acc[j], 0, 0, 0);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, hi[j][b]), dh, acc[j], 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j / 2][4 * (j % 2) + q] = acc[j][q];
  }
  // dW: expert rows 16 m + i of the 32 tokens, each of the three, times x.
  __device__ static void dw(const char* lds, const SkinnyW<bf16_t>& x, int lane, f32x4_t (&acc)[4][2 * EB]) {
    typedef short v4i16 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
    const int s = lane & 15, g = lane >> 4;
    bf16x8_t xf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xf[j] = x.frag(j);
#pragma unroll
    for (int m = 0; m < 6 * EB; ++m) {
      const int c = 16 * (m % (2 * EB)) + 4 * (s & 3), r = 8 * g + (s >> 2), part = m / (2 * EB);
      const char* p0 = lds + at(part, r, c >> 3) + (c & 7) * 2;
      const char* p1 = lds + at(part, r + 4, c >> 3) + (c & 7) * 2;
      const v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p0));
      const v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p1));
      const bf16x8_t dl = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j][m % (2 * EB)] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dl, xf[j], acc[j][m % (2 * EB)], 0, 0, 0);
    }
  }
  // Expert of register q of sums m.
  __device__ static int expert(int m, int q, int lane) { return 16 * m + 4 * (lane >> 4) + q; }
};

template <int EB>
struct BalGrad<float, EB> {
  static constexpr int EP = 32 * EB, ROW = 4 * EP, BYTES = ROW;
  // Step s takes element s % 4 of the lane groups' 16 bytes s / 4 on both sides:
  // experts 16 (s / 4) + 4 (lane / 16) + s % 4.
  f32x4_t w[4][2 * EB];
  __device__ void load(const u32x4* wb, int c0, int lane) {
    const u32x4* p = wb + static_cast<int64_t>(c0 / 64) * 8 * EB * 64 + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < 2 * EB; ++b) w[j][b] = __builtin_bit_cast(f32x4_t, p[(j * 2 * EB + b) * 64]);
  }
  __device__ static int at(int r, int c) { return r * ROW + ((c ^ (r & (ROW / 16 - 1))) << 4); }
  __device__ static void put_dl(char* lds, int r, int c, const u32x4& dl) {
    *reinterpret_cast<u32x4*>(lds + at(r, c)) = dl;
  }
  // v[h]: columns c0 + 16 (2 h) + 4 (lane / 16) .. + 3, then 16 further on
  __device__ void dx(const char* lds, int r0, int lane, float (&v)[2][8]) const {
    const int r = r0 + (lane & 15), g = lane >> 4;
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < 2 * EB; ++b) {
      const f32x4_t dl = *reinterpret_cast<const f32x4_t*>(lds + at(r, 4 * b + g));
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[j][b][q], dl[q], acc[j], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j / 2][4 * (j % 2) + q] = acc[j][q];
  }
  // Sums m take experts 4 i + m of every 64 (32 with one block: 2 i + m).
  __device__ static void dw(const char* lds, const SkinnyW<float>& x, int lane, f32x4_t (&acc)[4][2 * EB]) {
    const int s = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + g;
      float dl[2 * EB];
      const char* p = lds + at(r, s * EB / 2) + (EB == 1 ? (s & 1) * 8 : 0);
#pragma unroll
      for (int m = 0; m < 2 * EB; ++m) dl[m] = reinterpret_cast<const float*>(p)[m];
#pragma unroll
      for (int m = 0; m < 2 * EB; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x4f32(dl[m], __uint_as_float(x.r[i][j]), acc[j][m], 0, 0, 0);
    }
  }
  __device__ static int expert(int m, int q, int lane) { return 2 * EB * (4 * (lane >> 4) + q) + m; }
};

// x of 32 tokens from `rows` on (`left` of them there) and the four columns of
// a lane, without a branch: tokens past the last are read as the last.
__device__ __forceinline__ void load_tokens(SkinnyW<bf16_t>& x, const bf16_t* rows, int d, int left, int col, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t r = min(8 * (lane >> 4) + i, left - 1);
    x.r[i] = *reinterpret_cast<const u32x2*>(rows + (r * d + col));
  }
}
__device__ __forceinline__ void load_tokens(SkinnyW<float>& x, const float* rows, int d, int left, int col, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t r = min(4 * i + (lane >> 4), left - 1);
    x.r[i] = *reinterpret_cast<const u32x4*>(rows + (r * d + col));
  }
}
// Zeros for the tokens that are not there or that the mask leaves out (they
// may hold NaN): a byte a token in LDS, all ones or zeros.
__device__ __forceinline__ void drop_tokens(SkinnyW<bf16_t>& x, const char* keep, int lane) {
  const uint2 k = *reinterpret_cast<const uint2*>(keep + 8 * (lane >> 4));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int word = static_cast<int>(i < 4 ? k.x : k.y);
    x.r[i] &= static_cast<uint32_t>((word << (24 - 8 * (i % 4))) >> 24);
  }
}
__device__ __forceinline__ void drop_tokens(SkinnyW<float>& x, const char* keep, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x.r[i] &= static_cast<uint32_t>(static_cast<int>(keep[4 * i + (lane >> 4)]));
}

// 16384 tokens of 64 experts x 512 bf16: 17 us for 38 MB (7.4), MFMA 22% busy: five
// or six turns of a workgroup, each waiting for its x; 4999 x 1152 fp32 27 us, MFMA 44%
// (two blocks of experts in fp32 put 16 bytes a thread into scratch memory).
template <typename T, int EB>
__global__ __launch_bounds__(kGradThreads) __attribute__((amdgpu_waves_per_eu(2)))
void balance_grad_kernel(const BalGradArgs a, const T* __restrict__ x, const u32x4* __restrict__ wb,
                         const float* __restrict__ saved, T* dx, float* __restrict__ partial) {
  typedef BalGrad<T, EB> G;
  constexpr int EP = 32 * EB, kPieces = 32 * G::ROW / 16;       // 16-byte pieces of 32 tokens
  constexpr int kLoads = kGradSets * kPieces / kGradThreads;    // of a thread
  constexpr int kBuf = kGradSets * 32 * G::BYTES;
  static_assert(kGradSets * kPieces % kGradThreads == 0 && kPieces % 64 == 0, "loads");
  // the sums of three sets, a quarter at a time, share the place
  constexpr int kSums = (kGradSets - 1) * 2 * 2 * EB * 4 * 64 * 4;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kBuf > kSums ? 2 * kBuf : kSums];
  __shared__ __attribute__((aligned(16))) char kept[2][kGradSets * 32];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int set = wave / 2;
  const int slices = a.d / kGradCols;
  const int logical = xcd_remap(blockIdx.x, gridDim.x);
  const int range = logical / slices, c0 = logical % slices * kGradCols + 64 * (wave & 1);
  const int64_t chunks = (a.T + 31) / 32;
  const int64_t k0 = chunks * range / a.ranges, k1 = chunks * (range + 1) / a.ranges;
  const float scale = a.gloss ? a.gloss[0] : 1.0f;
  G weights;
  weights.load(wb, c0, lane);
  f32x4_t acc[4][2 * EB];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int m = 0; m < 2 * EB; ++m) acc[j][m] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};

  // dl of the next chunks, a token's 16-byte pieces side by side, and whether a
  // token counts; tokens past the end and chunks past the range as zeros
  u32x4 dl[kLoads];
  uint32_t keep = 0;  // 0: no
  auto load_dl = [&](int64_t k) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * kGradThreads + threadIdx.x, r = i % kPieces / (G::ROW / 16);
      const int64_t t = (k + i / kPieces) * 32 + r;
      const bool there = k + i / kPieces < k1 && t < a.T;
      const u32x4 v = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(saved) +
                                                      (there ? t : 0) * G::ROW + i % (G::ROW / 16) * 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) dl[u][q] = there ? v[q] : 0u;
    }
    if (threadIdx.x < kGradSets * 32) {
      const int64_t t = k * 32 + threadIdx.x;
      keep = t < a.T;
      if (a.mask && t < a.T) keep = a.mask[t];
    }
  };
  auto store_lds = [&](int to) {
    char* buf = smem + to * kBuf;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * kGradThreads + threadIdx.x, r = i % kPieces / (G::ROW / 16);
      G::put_dl(buf + i / kPieces * 32 * G::BYTES, r, i % (G::ROW / 16), dl[u]);
    }
    if (threadIdx.x < kGradSets * 32) kept[to][threadIdx.x] = keep ? '\xff' : '\0';
  };
  SkinnyW<T> xv;
  auto load_x = [&](int64_t k) {
    // a chunk past the range: the last one again, not used
    const int64_t t0 = min(k + set, chunks - 1) * 32;
    const int left = static_cast<int>(a.T - t0 < 32 ? a.T - t0 : 32);
    load_tokens(xv, x + t0 * a.d, a.d, left, c0 + 4 * (lane & 15), lane);
  };
  auto work = [&](int from, int64_t k) {
    const char* lds = smem + from * kBuf + set * 32 * G::BYTES;
    const int64_t t0 = (k + set) * 32;
    if (k + set < k1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[2][8];
        weights.dx(lds, 16 * h, lane, v);
        const int64_t t = t0 + 16 * h + (lane & 15);
        if (t >= a.T) continue;
        T* row = dx + t * a.d + c0;
        constexpr int V = Piece<T>::V;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int q = 0; q < 8 / V; ++q) {
            const int c = sizeof(T) == 2 ? 32 * n + 8 * (lane >> 4) : 16 * (2 * n + q) + 4 * (lane >> 4);
            float e[V], old[V];
            u32x4 o = (u32x4){0u, 0u, 0u, 0u};
            if (a.add) o = *reinterpret_cast<const u32x4*>(row + c);
            Piece<T>::widen(o, old);
#pragma unroll
            for (int m = 0; m < V; ++m) e[m] = __builtin_fmaf(scale, v[n][q * V + m], old[m]);
            *reinterpret_cast<u32x4*>(row + c) = Piece<T>::narrow(e);
          }
      }
      drop_tokens(xv, kept[from] + 32 * set, lane);
      G::dw(lds, xv, lane, acc);
    }
  };
  load_dl(k0);
  load_x(k0);
  store_lds(0);
  __syncthreads();
  // buffers in turn: the one that is written was last read before the last
  // barrier; x of the next tokens is on its way through the barrier and dx
  int buf = 0;
  for (int64_t k = k0; k < k1; k += kGradSets, buf ^= 1) {
    load_dl(k + kGradSets);
    work(buf, k);
    load_x(k + kGradSets);
    store_lds(buf ^ 1);
    __syncthreads();
  }
  // the sets' sums in order, a fragment of columns at a time, then out
  float* sums = reinterpret_cast<float*>(smem);
  float* out = partial + static_cast<int64_t>(range) * a.d * EP;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j) __syncthreads();
    if (set > 0) {
#pragma unroll
      for (int m = 0; m < 2 * EB; ++m)
        *reinterpret_cast<f32x4_t*>(sums + (((wave - 2) * 2 * EB + m) * 64 + lane) * 4) = acc[j][m];
    }
    __syncthreads();
    if (set == 0) {
#pragma unroll
      for (int m = 0; m < 2 * EB; ++m) {
        f32x4_t v = acc[j][m];
#pragma unroll
        for (int u = 0; u < kGradSets - 1; ++u)
          v += *reinterpret_cast<const f32x4_t*>(sums + (((2 * u + wave) * 2 * EB + m) * 64 + lane) * 4);
        // column of x: 4 (lane % 16) + j
        float* row = out + static_cast<int64_t>(c0 + 4 * (lane & 15) + j) * EP;
        if (sizeof(T) == 2) {
          *reinterpret_cast<f32x4_t*>(row + G::expert(m, 0, lane)) = v;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) row[G::expert(m, q, lane)] = v[q];
        }
      }
    }
  }
}

// dW [d][E] from the ranges' partial sums [ranges][d][EP], in order within 16
// threads, these then in order: four experts a thread.
__global__ __launch_bounds__(256) void balance_sum_kernel(const float* __restrict__ partial, int ranges, int d,
                                                          int E, int EP, const float* __restrict__ gloss,
                                                          bool add, float* __restrict__ dw) {
  __shared__ float4 sums[16][16];
  const int c = threadIdx.x % 16, j = threadIdx.x / 16;
  const int64_t cells = static_cast<int64_t>(d) * EP / 4, i = static_cast<int64_t>(blockIdx.x) * 16 + c;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int p = j; p < ranges; p += 16) {
    const float4 o = *reinterpret_cast<const float4*>(partial + (p * cells + i) * 4);
    v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
  }
  sums[j][c] = v;
  __syncthreads();
  if (j) return;
#pragma unroll
  for (int u = 1; u < 16; ++u) {
    const float4 o = sums[u][c];
    v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
  }
  const float scale = gloss ? gloss[0] : 1.0f, s[4] = {v.x, v.y, v.z, v.w};
  const int64_t row = i * 4 / EP;
  const int e = static_cast<int>(i * 4 % EP);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (e + q < E) {
      float* p = dw + row * E + e + q;
      *p = add ? __builtin_fmaf(scale, s[q], *p) : scale * s[q];
    }
}

__global__ __launch_bounds__(256) void balance_zero_kernel(float* p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// ------------------------------------------------------------------ layouts

// Tokens of a logits workgroup: 256 with whole rows of 64 tokens a wave, or 32
// with waves that share the columns, which fill the chip with fewer tokens. bf16,
// 64 experts x 512: 32768 tokens 21.3 and 17.9 us, 50000 22.6 and 26.2; fp32 50000
// 48.4 and 44.8, 65536 49 and 58 (fp32 MFMAs take longer: less is won by sharing W).
constexpr int64_t kManyTokens = 40960, kManyTokensF32 = 57344;
int logits_rows(int64_t T, int dtype) { return T >= (dtype == MOE_BF16 ? kManyTokens : kManyTokensF32) ? 256 : 32; }

// Ranges of the tokens: one workgroup a CU, not more (a few more took 4999 x 1152
// fp32 45 us, in two goes).
int grad_ranges(const moe_balance& b) {
  const int64_t slices = b.d_model / kGradCols, chunks = (b.tokens + 31) / 32;
  int64_t r = 256 / slices;
  const int64_t most = (chunks + kGradSets - 1) / kGradSets;
  if (r > most) r = most;
  return static_cast<int>(r < 1 ? 1 : r);
}

// Up to how many tokens the workgroups of an inference call split W and count
// themselves, a launch less: bf16, 64 experts x 512, 200 tokens 10.1 and 13.6 us,
// 8192 13.1 and 15.4; x 2048, 8192 tokens 24.3 and 24.8. (With 256-token workgroups
// the last kernel would have 512 counts an expert to add: 131072 tokens, 45 and 41.5.)
constexpr int64_t kRawTokens = 8192;

struct BalLayout {
  size_t parts, stats, own, wf, partial, total;
};
BalLayout bal_layout(const moe_balance& b) {
  BalLayout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  const size_t EP = 32 * expert_blocks(b.experts), d = b.d_model;
  L.parts = take(kCountBlocks * 65 * sizeof(int32_t));
  const int64_t rows = logits_rows(b.tokens, b.dtype);
  L.stats = take((b.tokens + rows - 1) / rows * 65 * sizeof(float));
  L.own = take(b.tokens <= kRawTokens ? (b.tokens + rows - 1) / rows * 65 * sizeof(int32_t) : 0);
  L.wf = take(d * EP * (b.dtype == MOE_BF16 ? 6 : 4));
  L.total = o;
  o = 0;  // the backward has the place for itself
  L.partial = take(static_cast<size_t>(grad_ranges(b)) * d * EP * sizeof(float));
  if (o > L.total) L.total = o;
  return L;
}

// Bytes of dl in `saved`; W for the backward is behind it.
size_t saved_rows_bytes(const moe_balance& b) {
  return align_up(static_cast<size_t>(b.tokens) * 32 * expert_blocks(b.experts) * 4, 256);
}

template <typename T, int EB>
void launch_logits(const BalArgs& a, const T* x, const u32x4* wf, float* saved, hipStream_t s) {
  const int rows = logits_rows(a.T, sizeof(T) == 2 ? MOE_BF16 : MOE_FP32);
  const dim3 grid(static_cast<unsigned>((a.T + rows - 1) / rows));
  if (rows == 256)
    MOE_LAUNCH("balance_logits", (balance_logits_kernel<T, EB>), grid, dim3(256), 0, s, a, x, wf, saved);
  else if (a.w)
    MOE_LAUNCH("balance_logits", (balance_logits_few_kernel<T, EB, 4, true>), grid, dim3(256), 0, s, a, x, wf, saved);
  else
    MOE_LAUNCH("balance_logits", (balance_logits_few_kernel<T, EB, 4, false>), grid, dim3(256), 0, s, a, x, wf, saved);
}

template <typename T>
hipError_t balance_t(const moe_balance& b, const void* x, const float* w, const int32_t* idx, const uint8_t* mask,
                     int32_t* counts, float* mean_prob, float* loss, void* saved, void* ws, hipStream_t s) {
  const BalLayout L = bal_layout(b);
  char* W = static_cast<char*>(ws);
  const int EB = expert_blocks(b.experts);
  int32_t* parts = reinterpret_cast<int32_t*>(W + L.parts);
  u32x4* wf = reinterpret_cast<u32x4*>(W + L.wf);
  u32x4* wb = saved ? reinterpret_cast<u32x4*>(static_cast<char*>(saved) + saved_rows_bytes(b)) : nullptr;
  BalArgs a{b.tokens, b.experts, b.top_k, b.d_model, b.balance * static_cast<float>(b.experts), 2.0f * b.z, mask,
            parts, 0, reinterpret_cast<float*>(W + L.stats), nullptr, nullptr, nullptr};
  int groups = 0;
  if (b.tokens > 0) {
    if (!saved && b.tokens <= kRawTokens) {
      a.idx = idx;
      a.own = reinterpret_cast<int32_t*>(W + L.own);
      a.w = w;
    } else {
      const int64_t blocks = (b.tokens * b.top_k + 8 * kCountThreads - 1) / (8 * kCountThreads);
      a.count_blocks = static_cast<int>(blocks > kCountBlocks ? kCountBlocks : blocks);
      const int pieces = b.d_model / (2 * Piece<T>::V) * EB * 64 * (wb ? 2 : 1);
      MOE_LAUNCH("balance_count", balance_count_kernel<T>,
                 dim3(a.count_blocks + (pieces + kCountThreads - 1) / kCountThreads), dim3(kCountThreads), 0, s, a,
                 idx, w, EB, wf, wb, parts);
    }
    if (EB == 1) launch_logits<T, 1>(a, static_cast<const T*>(x), wf, static_cast<float*>(saved), s);
    else launch_logits<T, 2>(a, static_cast<const T*>(x), wf, static_cast<float*>(saved), s);
    const int rows = logits_rows(b.tokens, b.dtype);
    groups = static_cast<int>((b.tokens + rows - 1) / rows);
  }
  MOE_LAUNCH("balance_loss", balance_loss_kernel, dim3(1), dim3(1024), 0, s, a, groups, b.balance, b.z, counts,
             mean_prob, loss);
  return hipGetLastError();
}

template <typename T, int EB>
hipError_t balance_bwd_t(const moe_balance& b, const void* x, const uint8_t* mask, const void* saved,
                         const float* gloss, bool add, void* dx, float* dw, void* ws, hipStream_t s) {
  const int ranges = grad_ranges(b), EP = 32 * EB;
  float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + bal_layout(b).partial);
  const BalGradArgs a{b.tokens, b.d_model, ranges, mask, gloss, add};
  const u32x4* wb = reinterpret_cast<const u32x4*>(static_cast<const char*>(saved) + saved_rows_bytes(b));
  MOE_LAUNCH("balance_grad", (balance_grad_kernel<T, EB>), dim3(b.d_model / kGradCols * ranges), dim3(kGradThreads), 0, s, a,
             static_cast<const T*>(x), wb, static_cast<const float*>(saved), static_cast<T*>(dx), partial);
  MOE_LAUNCH("balance_sum", balance_sum_kernel, dim3(b.d_model * EP / 4 / 16), dim3(256), 0, s, partial, ranges,
             b.d_model, b.experts, EP, gloss, add, dw);
  return hipGetLastError();
}

}  // namespace

size_t balance_ws_bytes(const moe_balance& b) { return bal_layout(b).total; }
size_t balance_saved_bytes(const moe_balance& b) {
  return saved_rows_bytes(b) + static_cast<size_t>(b.d_model) * 32 * expert_blocks(b.experts) * 4;
}

hipError_t launch_balance(const moe_balance& b, const void* x, const float* w, const int32_t* idx,
                          const uint8_t* mask, int32_t* counts, float* mean_prob, float* loss, void* saved, void* ws,
                          hipStream_t s) {
  return b.dtype == MOE_BF16 ? balance_t<bf16_t>(b, x, w, idx, mask, counts, mean_prob, loss, saved, ws, s)
                             : balance_t<float>(b, x, w, idx, mask, counts, mean_prob, loss, saved, ws, s);
}

hipError_t launch_balance_bwd(const moe_balance& b, const void* x, const uint8_t* mask, const void* saved,
                              const float* gloss, bool add, void* dx, float* dw, void* ws,
                              hipStream_t s) {
  if (b.tokens == 0) {
    const int64_t n = static_cast<int64_t>(b.d_model) * b.experts;
    if (!add)
      MOE_LAUNCH("balance_zero", balance_zero_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, dw, n);
    return hipGetLastError();
  }
  const bool wide = expert_blocks(b.experts) == 2;
  if (b.dtype == MOE_BF16)
    return wide ? balance_bwd_t<bf16_t, 2>(b, x, mask, saved, gloss, add, dx, dw, ws, s)
                : balance_bwd_t<bf16_t, 1>(b, x, mask, saved, gloss, add, dx, dw, ws, s);
  return wide ? balance_bwd_t<float, 2>(b, x, mask, saved, gloss, add, dx, dw, ws, s)
              : balance_bwd_t<float, 1>(b, x, mask, saved, gloss, add, dx, dw, ws, s);
}

}  // namespace moe
