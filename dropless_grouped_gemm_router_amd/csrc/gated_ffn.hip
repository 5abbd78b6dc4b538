// Dense gated feed-forward block, forward and backward.
//
//   a = x Wg, b = x Wu, h = act(a) b, out = h Wd
//   dh = dout Wd^T, da = dh b act'(a), db = dh act(a)
//   dx = da Wg^T + db Wu^T, dWg = x^T da, dWu = x^T db, dWd = h^T dout
//
// Both projections, the activation and the product are one kernel (gate and
// up columns of a tile sit in matching registers); so are the product with
// Wd^T and the activation's gradient. The weights come [d][h] and [h][d]:
// the forward's products run over their leading dimension, so they are
// turned K-contiguous into the workspace first; the backward's data
// gradients read them as they are, and so does the forward in bf16 with widths
// in multiples of 64, up to some thousand tokens (in_place). The weight
// gradients reduce over tokens, in slices whose partial sums are added in a
// fixed order.
//
// Widths that are no multiple of 128 take zero-padded copies of the operands
// in the workspace (x and dout, and the weights the backward reads), with the
// hidden values kept at the padded width.
//
// 16384 tokens, 512 x 1024, bf16, forward and backward: 247 to 271 us (155
// GFLOP; at this depth a tile's loop and its epilogue, which writes and reads
// as many bytes, take turns: gate and up keep the MFMA pipes 23% busy and move
// 3.0 TB/s). 8192 tokens, 2048 x 8192: 2.5 ms, 0.99 PFLOP/s.
#include <algorithm>

#include "gemm_wgrad.h"
#include "mm.h"
#include "skinny.h"

namespace moe {

namespace {

// Tokens up to which the forward takes the serving form, bf16 and fp32. The
// serving form and tiles take, bf16, 16 tokens, 2048 x 8192: 25.0 and 27.8 us,
// 1024 x 4096: 14.1 and 13.4; 32 tokens: 29.3 and 28.5, 18.1 and 14.0; where
// tiles have the weights turned first, 17 tokens, 2047 x 8191: 88 and 76, 500 x
// 1001: 22.6 and 18.6. fp32, 64 tokens, 1024 x 4096: 39 and 52, 2048 x 2048: 55
// and 73; 128 tokens: 66 and 58, 63 and 77; 512 x 1024: 22 and 28.
// In bf16 the tiles round the hidden values for the second product, as the
// layer's experts do, and the serving form does not: from 17 tokens on the
// result is 2.35e-3 off 64 bits in the 2-norm instead of 1.66e-3, which its own
// rounding is. Two halves in the tiles too would be a third more MFMAs and two
// more bytes a hidden value.
constexpr int64_t kFewRows = 16, kFewRowsF32 = 128;
constexpr int64_t kCUs = 256;

constexpr int64_t pad128(int64_t v) { return (v + 127) / 128 * 128; }
size_t elem_bytes(const moe_ffn& f) { return f.dtype == MOE_BF16 ? 2 : 4; }

// ------------------------------------------------------------- activations

template <int kAct>
__device__ __forceinline__ float act_value(float a, float* slope) {
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

// ----------------------------------------------------------------- products

struct FfnOut {
  void* c;       // plain: the result
  int64_t ldc;
  void* h;       // gated: the hidden values
  // What the backward needs of the pre-activations: f = act(a) and
  // p = b act'(a), so that da = dh p and db = dh f. In bf16 each is rounded to
  // 20 bits and kept as its high half (f, p) and the next four mantissa bits,
  // both in one byte of `low`: 5 bytes a pair instead of 4, and off by 2^-12 at
  // most instead of the 2^-8 of a bf16 number, which leaves the roundings of
  // da, db and the result as the only ones that count in the gradients.
  void *f, *p;
  uint8_t* low;
  int64_t ld;    // columns kept of the hidden matrices (a multiple of 128)
  void* dab;     // gradient: da and db, a row of each side by side
  u32x4* zero;   // null, or a zero row that kTurned tiles write (else turn_kernel does)
};

// Half a step of the kept 20 bits, added before the rest is cut off: the
// nearest kept value, the larger one of two that are as near. (Without it
// every value would come out shorter, by 1.8e-4 on average, and so would the
// gradients over however many tokens.) No test is needed: an infinity's bits
// below the 20th are cut again, and a NaN changes only if the upper 12 of its
// mantissa's bits are all set, which those of bf16 operands (16 low bits zero)
// and the hardware's own are not.
__device__ __forceinline__ uint32_t kept20(float v) { return __float_as_uint(v) + 0x800u; }

// What is kept of eight values of f and p.
__device__ __forceinline__ void keep8(const FfnOut& o, int64_t at, const float (&f)[8],
                                      const float (&p)[8], const bf16_t*) {
  u32x4 fh, ph;
  uint32_t lo[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 8; q += 2) {
    const uint32_t a = kept20(f[q]), b = kept20(f[q + 1]);
    const uint32_t c = kept20(p[q]), d = kept20(p[q + 1]);
    fh[q / 2] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    ph[q / 2] = __builtin_amdgcn_perm(d, c, 0x07060302u);
    // byte 1 of each: its high nibble follows the 16 bits that are kept
    const uint32_t fl = __builtin_amdgcn_perm(b, a, 0x0c0c0501u), pl = __builtin_amdgcn_perm(d, c, 0x0c0c0501u);
    const uint32_t both = ((fl >> 4) & 0x0f0fu) | (pl & 0xf0f0u);
    lo[q / 4] |= (q & 2) ? both << 16 : both;
  }
  *reinterpret_cast<u32x4*>(static_cast<bf16_t*>(o.f) + at) = fh;
  *reinterpret_cast<u32x4*>(static_cast<bf16_t*>(o.p) + at) = ph;
  *reinterpret_cast<uint2*>(o.low + at) = make_uint2(lo[0], lo[1]);
}
__device__ __forceinline__ void keep8(const FfnOut& o, int64_t at, const float (&f)[8],
                                      const float (&p)[8], const float*) {
  store4(static_cast<float*>(o.f) + at, f[0], f[1], f[2], f[3]);
  store4(static_cast<float*>(o.f) + at + 4, f[4], f[5], f[6], f[7]);
  store4(static_cast<float*>(o.p) + at, p[0], p[1], p[2], p[3]);
  store4(static_cast<float*>(o.p) + at + 4, p[4], p[5], p[6], p[7]);
}

template <typename T>
struct Kept;
template <>
struct Kept<bf16_t> {
  u32x4 f, p;
  uint2 low;
  __device__ void load(const FfnOut& o, int64_t at) {
    f = *reinterpret_cast<const u32x4*>(static_cast<const bf16_t*>(o.f) + at);
    p = *reinterpret_cast<const u32x4*>(static_cast<const bf16_t*>(o.p) + at);
    low = *reinterpret_cast<const uint2*>(o.low + at);
  }
  __device__ void get(int q, float* fv, float* pv) const {
    const uint32_t lo = ((q < 4 ? low.x : low.y) >> (8 * (q % 4))) & 0xffu;
    const uint32_t a = (q & 1) ? f[q / 2] & 0xffff0000u : f[q / 2] << 16;
    const uint32_t b = (q & 1) ? p[q / 2] & 0xffff0000u : p[q / 2] << 16;
    *fv = __uint_as_float(a | ((lo & 15u) << 12));
    *pv = __uint_as_float(b | ((lo >> 4) << 12));
  }
};
template <>
struct Kept<float> {
  float f[8], p[8];
  __device__ void load(const FfnOut& o, int64_t at) {
    load4(static_cast<const float*>(o.f) + at, f);
    load4(static_cast<const float*>(o.f) + at + 4, f + 4);
    load4(static_cast<const float*>(o.p) + at, p);
    load4(static_cast<const float*>(o.p) + at + 4, p + 4);
  }
  __device__ void get(int q, float* fv, float* pv) const {
    *fv = f[q];
    *pv = p[q];
  }
};

enum { kPlain = 0, kGated = 1, kGatedGrad = 2, kPart = 3 };  // kPart: a K slice's sums, fp32

template <typename T>
struct OpOf {
  typedef OpBf16 type;
};
template <>
struct OpOf<float> {
  typedef OpF32 type;
};

// The callbacks of mm_drain; kFull: every column of the tile is below p.N.
// Else columns past p.N are left out, or, up to its padded width o.ld, are
// written as zeros in a hidden matrix.
template <typename T, typename Cfg, int kMode, int kAct, bool kFull>
struct FfnRows {
  static constexpr int kJ = Cfg::WN / MmStrip<Cfg>::CB;
  static constexpr bool kGrad = kMode == kGatedGrad;
  const MmArgs& p;
  const FfnOut& o;
  const MmTile& t;
  int base, n[kJ];
  Kept<T> kept[kGrad ? 2 : 1][kGrad ? mm_passes<Cfg, false>() : 1];

  __device__ void cols(int j, int c) { n[j] = base + c; }
  __device__ void start(int, int, int) {}
  __device__ void pre(int set, int j, int k, int m) {
    if constexpr (kGrad) {
      if (kFull || n[j] < o.ld) kept[set][k].load(o, (t.row0 + m) * o.ld + n[j]);
    }
  }
  __device__ void row(int set, int, int j, int k, int m, const uint32_t (&v)[8]) {
    const int64_t row = t.row0 + m;
    if constexpr (!kGrad) {
      float y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = __uint_as_float(v[q]);
      if constexpr (kMode == kPart)
        store8<float, kFull>(static_cast<float*>(o.c) + (t.part * p.M + row) * o.ldc, n[j], p.N, y);
      else
        store8<T, kFull>(static_cast<T*>(o.c) + row * o.ldc, n[j], p.N, y);
    } else {
      if (!kFull && n[j] >= o.ld) return;
      float da[8], db[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float fv, pv;
        kept[set][k].get(q, &fv, &pv);
        const float dh = __uint_as_float(v[q]);
        const bool in = kFull || n[j] + q < p.N;
        da[q] = in ? dh * pv : 0.0f;
        db[q] = in ? dh * fv : 0.0f;
      }
      T* dst = static_cast<T*>(o.dab) + row * 2 * o.ld;
      store8<T, true>(dst, n[j], 0, da);
      store8<T, true>(dst + o.ld, n[j], 0, db);
    }
  }
  __device__ void row(int, int, int j, int, int m, const uint32_t (&g)[8], const uint32_t (&u)[8]) {
    if (!kFull && n[j] >= o.ld) return;
    float h[8], f[8], s[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool in = kFull || n[j] + q < p.N;
      const float b = __uint_as_float(u[q]);
      float slope;
      const float fv = act_value<kAct>(__uint_as_float(g[q]), &slope);
      h[q] = in ? fv * b : 0.0f;
      f[q] = in ? fv : 0.0f;
      s[q] = in ? b * slope : 0.0f;
    }
    store8<T, true>(static_cast<T*>(o.h) + (t.row0 + m) * o.ld, n[j], 0, h);
    if (o.f) keep8(o, (t.row0 + m) * o.ld + n[j], f, s, static_cast<const T*>(nullptr));
  }
};

template <typename T, typename Cfg, int kMode, int kAct, bool kTurned>
__global__ __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(Cfg::WPE)))
void ffn_tile_kernel(const MmArgs p, const FfnOut o) {
  __shared__ __attribute__((aligned(1024))) char smem[MmStrip<Cfg>::LDS];
  f32x16_t acc[Cfg::WM][Cfg::WN];
  MmTile t;
  constexpr bool kPaired = kMode == kGated;
  if (kTurned && o.zero && blockIdx.x == 0 && threadIdx.x < kTrZeroBytes / 16)
    o.zero[threadIdx.x] = (u32x4){0u, 0u, 0u, 0u};
  if (!mm_find<Cfg>(p, &t)) return;
  constexpr int kCols = kPaired ? Cfg::BN / 2 : Cfg::BN;
  auto go = [&](auto full) {
    FfnRows<T, Cfg, kMode, kAct, decltype(full)::value> rows{p, o, t, t.nt * kCols};
    mm_begin<Cfg, kPaired>(t.rows, rows);
    mm_drain<Cfg, kPaired>(smem, acc, t.rows, rows);
  };
  mm_tile<typename OpOf<T>::type, Cfg, kPaired, kTurned>(p, smem, t, acc);
  if ((t.nt + 1) * kCols <= p.N) go(std::true_type{});
  else go(std::false_type{});
}

// ------------------------------------------------------------ few tokens

// Hidden values of the serving form. In bf16 they are kept as the sum of two
// bf16 numbers (high and low half: 2^-17 instead of 2^-9): the second
// product is bound by the weights' bytes, so the second MFMA is free.
__device__ __forceinline__ void put_hidden(bf16_t* high, bf16_t* low, float v) {
  const bf16_t h = f32_to_bf16(v);
  *high = h;
  // an infinite or NaN high half says it all
  const float rest = v - bf16_to_f32(h);
  *low = (__float_as_uint(rest) & 0x7f800000u) == 0x7f800000u ? 0 : f32_to_bf16(rest);
}
__device__ __forceinline__ void put_hidden(float* high, float*, float v) { *high = v; }

// One value of f and p as keep8 keeps eight.
__device__ __forceinline__ void keep1(const FfnOut& o, int64_t at, float f, float p, const bf16_t*) {
  const uint32_t a = kept20(f), b = kept20(p);
  static_cast<bf16_t*>(o.f)[at] = static_cast<bf16_t>(a >> 16);
  static_cast<bf16_t*>(o.p)[at] = static_cast<bf16_t>(b >> 16);
  o.low[at] = static_cast<uint8_t>(((a >> 12) & 0x0fu) | ((b >> 8) & 0xf0u));
}
__device__ __forceinline__ void keep1(const FfnOut& o, int64_t at, float f, float p, const float*) {
  static_cast<float*>(o.f)[at] = f;
  static_cast<float*>(o.p)[at] = p;
}

// Training (o.f): also what the backward needs, over the padded width o.ld
// (columns past N come out as zeros: no weights are read for them), and the
// backward's row of zeros.
template <typename T, int kAct>
__global__ __launch_bounds__(512) void ffn_rows_gate_up_kernel(const SkinnyArgs<T, 2> a, T* high, T* low,
                                                               const FfnOut o, u32x4* zero) {
  __shared__ float lds[kSkinnyWaves][kSkinnyLds];
  float sum[2][2];
  if (zero && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kTrZeroBytes / 16)
    zero[threadIdx.x] = (u32x4){0u, 0u, 0u, 0u};
  skinny_sums<T, 2, false>(a, lds, sum);
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int64_t row = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x >> 6) + 8 * v;
    const int n = blockIdx.x * kSkinnyCols + (threadIdx.x & 63);
    if (row >= a.rows) continue;
    const float b = sum[v][1];
    float slope;
    const float f = act_value<kAct>(sum[v][0], &slope), h = f * b;
    if (n < a.N) put_hidden(high + row * a.N + n, low + row * a.N + n, h);
    if (o.f) {
      put(static_cast<T*>(o.h) + row * o.ld + n, h);
      keep1(o, row * o.ld + n, f, b * slope, static_cast<const T*>(nullptr));
    }
  }
}

// part: null (one slice of K): out is written; else the slices' sums
// [k_parts][rows][N].
template <typename T>
__global__ __launch_bounds__(512) void ffn_rows_down_kernel(const SkinnyArgs<T, 1> a, T* out, float* part) {
  __shared__ float lds[kSkinnyWaves][kSkinnyLds];
  float sum[2][1];
  skinny_sums<T, 1, sizeof(T) == 2>(a, lds, sum);
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int64_t row = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x >> 6) + 8 * v;
    const int n = blockIdx.x * kSkinnyCols + (threadIdx.x & 63);
    if (row >= a.rows || n >= a.N) continue;
    if (part) part[(blockIdx.z * a.rows + row) * a.N + n] = sum[v][0];
    else put(out + row * a.N + n, sum[v][0]);
  }
}

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

// The three weight gradients in fp32, in one launch: products over the
// tokens of turned operands, [rows of the gradient][tokens] each.
struct GradArgs {
  MmArgs p[3];
  FfnOut o[3];
  int end[3];  // exclusive end of each product's tiles
};
template <typename Cfg, int kMode>
__global__ __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(Cfg::WPE)))
void ffn_grad_kernel(const GradArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[MmStrip<Cfg>::LDS];
  int w = xcd_remap(blockIdx.x, gridDim.x);
  const int part = w / a.end[2];
  w %= a.end[2];
  const int which = w < a.end[0] ? 0 : (w < a.end[1] ? 1 : 2);
  const MmArgs& p = a.p[which];
  const FfnOut& o = a.o[which];
  f32x16_t acc[Cfg::WM][Cfg::WN];
  MmTile t;
  if (!mm_place<Cfg>(p, w - (which ? a.end[which - 1] : 0), part, &t)) return;
  mm_tile<OpF32, Cfg, false>(p, smem, t, acc);
  auto go = [&](auto full) {
    FfnRows<float, Cfg, kMode, 0, decltype(full)::value> rows{p, o, t, t.nt * Cfg::BN};
    mm_begin<Cfg, false>(t.rows, rows);
    mm_drain<Cfg, false>(smem, acc, t.rows, rows);
  };
  if ((t.nt + 1) * Cfg::BN <= p.N) go(std::true_type{});
  else go(std::false_type{});
}

// Weight gradients from the slices' partial sums [splits][mp][ld], cropped
// to M x N at column `col` and rounded once: the slices are added in order.
// Up to three gradients in one launch.
struct SliceJob {
  const float* part;
  int splits;
  int64_t stride;  // floats between slices
  int64_t ld;
  int M, N;
  void* out;
  int64_t end;     // exclusive end of the job's four-column pieces
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
    G* dst = static_cast<G*>(b.out) + m * b.N + n;
    if (n + 4 <= b.N && b.N % 4 == 0) {
      store4(dst, v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < b.N) put(dst + q, v[q]);
    }
  }
}

template <typename G>
__global__ __launch_bounds__(256) void zero_kernel(G* __restrict__ p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = G{};
}

// ------------------------------------------------------------------ layouts

int parts_of(size_t elem, int64_t M, int64_t N, int64_t stages);
int grad_parts(const moe_ffn& f);
bool in_place(const moe_ffn& f);

struct FfnBlockLayout {
  // forward workspace: turned weights, padded x, hidden values (inference)
  size_t tg, tu, td, xp, h;
  // backward workspace
  size_t dyp, wgp, wup, wdp, dab, part_gu, part_d;
  size_t xt, dabt, ht, dyt;  // fp32: operands of the weight gradients, turned
  // serving form: hidden values (both halves) and the second product's slices
  size_t rows_h, rows_part;
  size_t k_sums;  // sums of the slices of K of a plain product
  size_t total;
  int splits_gu, splits_d, k_parts, grad_parts;
};

int slices(int64_t rows, int64_t tiles) {
  int64_t k = (512 + tiles - 1) / tiles;
  k = k < 1 ? 1 : (k > 64 ? 64 : k);
  const int64_t most = (rows + 63) / 64;  // a stage of 64 rows each at least
  return static_cast<int>(k > most ? (most < 1 ? 1 : most) : k);
}

// Whether the forward takes the serving form (training too: what it keeps is
// the same, and the weights are not turned).
bool few_rows(const moe_ffn& f) { return f.tokens <= (f.dtype == MOE_BF16 ? kFewRows : kFewRowsF32); }

FfnBlockLayout ffn_block_layout(const moe_ffn& f, bool training) {
  FfnBlockLayout L{};
  const size_t es = elem_bytes(f);
  const size_t T = f.tokens, d = f.d_model, h = f.d_hidden, dp = pad128(d), hp = pad128(h);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  if (few_rows(f)) {
    L.rows_h = take(T * h * es * (es == 2 ? 2 : 1));
    // slices of K so that every CU has a workgroup, of two steps a wave at least
    const int64_t blocks = f.tokens == 0 ? 1 : (f.d_model + kSkinnyCols - 1) / kSkinnyCols * ((f.tokens + 15) / 16);
    const int64_t most = (f.d_hidden + 2 * kSkinnyStep * kSkinnyWaves - 1) / (2 * kSkinnyStep * kSkinnyWaves);
    const int64_t want = (256 + blocks - 1) / blocks;
    L.k_parts = static_cast<int>(want < most ? want : most);
    L.rows_part = take(L.k_parts > 1 ? L.k_parts * T * d * sizeof(float) : 0);
    L.total = o;
    if (!training) return L;
    o = 0;  // the backward has the place for itself
  }
  L.xp = take(d == dp ? 0 : T * dp * es);
  const size_t start = o;
  if (!few_rows(f) && !in_place(f)) {
    L.tg = take(h * dp * es);
    L.tu = take(h * dp * es);
    L.td = take(d * hp * es);
  }
  if (!training) L.h = take(T * hp * es);
  auto sums = [&](int64_t K) {
    const int n = parts_of(es, f.tokens, d, K * es / 128);
    return n > 1 ? n * T * d * sizeof(float) : 0;
  };
  L.k_sums = take(sums(hp));
  L.total = std::max(L.total, o);
  if (training) {
    // the backward reuses the turned weights' place
    o = start;
    L.dyp = take(d == dp ? 0 : T * dp * es);
    L.wgp = take(h == hp ? 0 : d * hp * es);
    L.wup = take(h == hp ? 0 : d * hp * es);
    L.wdp = take(d == dp ? 0 : h * dp * es);
    L.dab = take(T * 2 * hp * es);
    if (f.dtype == MOE_BF16) {
      const int64_t tiles = static_cast<int64_t>(dp / 128) * (hp / 128);
      L.splits_gu = slices(f.tokens, 2 * tiles);
      L.splits_d = slices(f.tokens, tiles);
      L.part_gu = take(L.splits_gu > 1 ? static_cast<size_t>(L.splits_gu) * 2 * dp * hp * sizeof(float) : 0);
      L.part_d = take(L.splits_d > 1 ? static_cast<size_t>(L.splits_d) * dp * hp * sizeof(float) : 0);
    } else {
      const size_t tp = pad128(f.tokens);
      L.xt = take(d * tp * es);
      L.dabt = take(2 * hp * tp * es);
      L.ht = take(h * tp * es);
      L.dyt = take(d * tp * es);
      L.grad_parts = grad_parts(f);
      const size_t n = L.grad_parts > 1 ? L.grad_parts : 0;
      L.part_gu = take(n * 2 * d * ((h + 3) / 4 * 4) * sizeof(float));
      L.part_d = take(n * h * ((d + 3) / 4 * 4) * sizeof(float));
    }
    // one place for the sums of either pass
    L.k_sums = std::max(o, L.total);
    L.total = L.k_sums + std::max(sums(hp), sums(2 * hp));
  }
  return L;
}

// `zero`: a row of zeros for the weight gradients' loads past the last token.
struct SavedLayout {
  size_t h, f, p, low, zero, total;
};
SavedLayout saved_layout(const moe_ffn& f) {
  const size_t cells = static_cast<size_t>(f.tokens) * pad128(f.d_hidden);
  const size_t n = align_up(cells * elem_bytes(f), 256);
  const size_t zero = 3 * n + (f.dtype == MOE_BF16 ? align_up(cells, 256) : 0);
  return SavedLayout{0, n, 2 * n, 3 * n, zero, zero + kTrZeroBytes};
}

FfnOut saved_out(const SavedLayout& S, char* saved, int64_t hp) {
  FfnOut o{};
  o.h = saved + S.h;
  o.f = saved + S.f;
  o.p = saved + S.p;
  o.low = reinterpret_cast<uint8_t*>(saved + S.low);
  o.ld = hp;
  return o;
}

// ----------------------------------------------------------------- launches

template <typename T, typename Cfg, int kMode, int kAct, bool kTurned = false>
void tiles_at(const char* name, const MmArgs& a, const FfnOut& o, hipStream_t s) {
  MmArgs p = a;
  const int per = kMode == kGated ? Cfg::BN / 2 : Cfg::BN;
  // the hidden matrices are written to their padded width
  const int64_t n = kMode == kPlain || kMode == kPart ? p.N : o.ld;
  p.tiles_n = static_cast<int>((n + per - 1) / per);
  p.nk *= 128 / Cfg::ROW;
  p.k_split *= 128 / Cfg::ROW;
  const int64_t grid = (p.M + Cfg::BM - 1) / Cfg::BM * p.tiles_n * (p.parts > 1 ? p.parts : 1);
  MOE_LAUNCH(name, (ffn_tile_kernel<T, Cfg, kMode, kAct, kTurned>), dim3(static_cast<unsigned>(grid)),
             dim3(Cfg::NT), 0, s, p, o);
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
TileSize tile_of(size_t elem, int64_t M, int64_t cols, int64_t stages) {
  auto count = [&](int m, int n) { return (M + m - 1) / m * ((cols + n - 1) / n); };
  if (M <= (elem == 2 ? 128 : 64)) return kSmall;
  if (elem == 2 && stages >= 16 && count(256, 256) >= kCUs) return kBig;
  if (elem == 2 && count(256, 128) >= kCUs) return kTall;
  return count(128, 128) >= kCUs ? kMid : kSmall;
}
// Slices of K of a plain product: two workgroups a CU, four stages each at
// least (777 x 500 with K 2048 in fp32: 104 tiles of 64 x 64).
int parts_of(size_t elem, int64_t M, int64_t N, int64_t stages) {
  if (tile_of(elem, M, N, stages) != kSmall) return 1;
  const int64_t tiles = (M + 63) / 64 * ((N + 63) / 64);
  if (tiles == 0) return 1;  // no tokens
  int64_t k = tiles < kCUs ? 2 * kCUs / tiles : 1;
  if (k > stages / 4) k = stages / 4;
  return static_cast<int>(k < 1 ? 1 : (k > 16 ? 16 : k));
}

// Whether the forward's tiles read the weights where they are (mm_tile,
// kTurned), in 64 x 64 or 128 x 128: bf16, widths that fill stages, and not so
// many tokens that turning the weights once for the larger tiles is less.
// Turned first and in place, 300 tokens, 1024 x 4096: 35.1 and 28.4 us; 1000
// tokens, 2048 x 8192: 154 and 145, 4000: 441 and 439, 8192: 790 and 925;
// 8192 tokens, 1024 x 4096: 258 and 243; 16384 tokens, 512 x 1024: 93 and 91,
// 32768: 147 and 152. Narrower ones at the limit, inference and training: 131072
// tokens, 64 x 256: 70 and 49, 93 and 61; 65536, 128 x 1024: 111 and 93, 159 and
// 162; 32768, 256 x 1024: 79 and 76, 97 and 96; the one that loses, 16384, 256 x
// 4096: 147 and 146, 237 and 255.
constexpr int64_t kInPlace = int64_t{1} << 23;  // elements of x
bool in_place(const moe_ffn& f) {
  if (f.dtype != MOE_BF16 || f.d_model % 64 || f.d_hidden % 64) return false;
  return f.tokens * f.d_model <= kInPlace;
}

template <typename T, int kMode, int kAct>
void tiles(const char* name, const MmArgs& p, const FfnOut& o, hipStream_t s, bool turned = false) {
  const int64_t cols = kMode == kGated ? 2 * static_cast<int64_t>(p.N) : p.N;
  if constexpr (sizeof(T) == 2 && (kMode == kPlain || kMode == kGated)) {
    if (turned) {
      if (tile_of(2, p.M, cols, p.nk) == kSmall) tiles_at<T, MmSmall, kMode, kAct, true>(name, p, o, s);
      else tiles_at<T, MmMid, kMode, kAct, true>(name, p, o, s);
      return;
    }
  }
  switch (tile_of(sizeof(T), p.M, cols, p.nk)) {
    case kSmall: return tiles_at<T, MmSmall, kMode, kAct>(name, p, o, s);
    case kMid: return tiles_at<T, MmMid, kMode, kAct>(name, p, o, s);
    default: break;
  }
  if constexpr (sizeof(T) == 2) {
    if (tile_of(sizeof(T), p.M, cols, p.nk) == kBig) return tiles_at<T, MmBig, kMode, kAct>(name, p, o, s);
    tiles_at<T, MmTall, kMode, kAct>(name, p, o, s);
  }
}

// Tiles of the fp32 weight gradients in tiles of t, and the slices of the
// tokens: one and a half workgroups a CU, four stages each at least.
int64_t grad_tiles(const moe_ffn& f, int t) {
  return 3 * ((f.d_model + t - 1) / t) * static_cast<int64_t>((f.d_hidden + t - 1) / t);
}
int grad_parts(const moe_ffn& f) {
  const int64_t tiles = grad_tiles(f, 64), stages = pad128(f.tokens) / 32;
  int64_t k = (kCUs * 3 / 2 + tiles - 1) / tiles;
  if (k > stages / 4) k = stages / 4;
  return static_cast<int>(k < 1 ? 1 : (k > 64 ? 64 : k));
}

// A plain product [M][N], over slices of K (sums in `part`) where it has few
// tiles.
template <typename T>
void product(const char* name, const MmArgs& a, void* out, float* part, hipStream_t s, bool turned = false) {
  MmArgs p = a;
  FfnOut o{};
  o.ldc = p.N;
  p.parts = parts_of(sizeof(T), p.M, p.N, p.nk);
  if (p.parts == 1) {
    o.c = out;
    return tiles<T, kPlain, 0>(name, p, o, s, turned);
  }
  o.c = part;
  if constexpr (sizeof(T) == 2) {
    if (turned) tiles_at<T, MmSmall, kPart, 0, true>(name, p, o, s);
  }
  if (!turned) tiles_at<T, MmSmall, kPart, 0>(name, p, o, s);
  const int64_t cells = p.M * p.N;
  MOE_LAUNCH("ffn_join", join_kernel<T>, dim3(static_cast<unsigned>((cells + 255) / 256)), dim3(256), 0, s,
             part, p.parts, cells, static_cast<T*>(out));
}

template <typename T, int kMode>
void tiles_act(const char* name, int act, const MmArgs& p, const FfnOut& o, hipStream_t s, bool turned) {
  switch (act) {
    case MOE_ACT_SILU: return tiles<T, kMode, MOE_ACT_SILU>(name, p, o, s, turned);
    case MOE_ACT_GELU: return tiles<T, kMode, MOE_ACT_GELU>(name, p, o, s, turned);
    case MOE_ACT_GELU_TANH: return tiles<T, kMode, MOE_ACT_GELU_TANH>(name, p, o, s, turned);
    default: return tiles<T, kMode, MOE_ACT_RELU>(name, p, o, s, turned);
  }
}

unsigned blocks_for(int64_t items) {
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
void pad(const PadJobs& jobs, hipStream_t s) {
  if (jobs.n)
    MOE_LAUNCH("ffn_pad_rows", pad_rows_kernel<T>, dim3(blocks_for(jobs.job[jobs.n - 1].end)), dim3(256),
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

template <typename T>
hipError_t ffn_rows_t(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                      const void* wd, void* saved, void* out, void* ws, hipStream_t s) {
  const FfnBlockLayout L = ffn_block_layout(f, saved != nullptr);
  char *W = static_cast<char*>(ws), *SV = static_cast<char*>(saved);
  const int d = f.d_model, h = f.d_hidden;
  T* high = reinterpret_cast<T*>(W + L.rows_h);
  T* low = sizeof(T) == 2 ? high + f.tokens * h : nullptr;
  const unsigned tall = static_cast<unsigned>((f.tokens + 15) / 16);
  SkinnyArgs<T, 2> a{static_cast<const T*>(x), nullptr, d,
                     {static_cast<const T*>(wg), static_cast<const T*>(wu)}, f.tokens, d, h, 1};
  FfnOut o{};
  u32x4* zero = nullptr;
  if (SV) {
    const SavedLayout S = saved_layout(f);
    o = saved_out(S, SV, pad128(h));
    zero = reinterpret_cast<u32x4*>(SV + S.zero);
  }
  const dim3 ga((SV ? pad128(h) : h + kSkinnyCols - 1) / kSkinnyCols, tall);
  switch (f.act) {
#define MOE_ROWS(ACT)                                                                              \
  case ACT:                                                                                        \
    MOE_LAUNCH("ffn_rows_gate_up", (ffn_rows_gate_up_kernel<T, ACT>), ga, dim3(512), 0, s, a, \
               high, low, o, zero);                                                                         \
    break
    MOE_ROWS(MOE_ACT_SILU);
    MOE_ROWS(MOE_ACT_GELU);
    MOE_ROWS(MOE_ACT_GELU_TANH);
    MOE_ROWS(MOE_ACT_RELU);
#undef MOE_ROWS
  }
  float* part = L.k_parts > 1 ? reinterpret_cast<float*>(W + L.rows_part) : nullptr;
  SkinnyArgs<T, 1> b{high, low, h, {static_cast<const T*>(wd)}, f.tokens, h, d, L.k_parts};
  MOE_LAUNCH("ffn_rows_down", (ffn_rows_down_kernel<T>),
             dim3((d + kSkinnyCols - 1) / kSkinnyCols, tall, L.k_parts), dim3(512), 0, s, b,
             static_cast<T*>(out), part);
  if (part) {
    const int64_t cells = f.tokens * d;
    MOE_LAUNCH("ffn_join", join_kernel<T>, dim3(static_cast<unsigned>((cells + 255) / 256)),
               dim3(256), 0, s, part, L.k_parts, cells, static_cast<T*>(out));
  }
  return hipGetLastError();
}

template <typename T>
hipError_t ffn_fwd_t(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                     const void* wd, void* saved, void* out, void* ws, hipStream_t s) {
  if (few_rows(f)) return ffn_rows_t<T>(f, x, wg, wu, wd, saved, out, ws, s);
  const FfnBlockLayout L = ffn_block_layout(f, saved != nullptr);
  const SavedLayout S = saved_layout(f);
  char *W = static_cast<char*>(ws), *SV = static_cast<char*>(saved);
  const int d = f.d_model, h = f.d_hidden;
  const int64_t dp = pad128(d), hp = pad128(h);
  u32x4* zero = SV ? reinterpret_cast<u32x4*>(SV + S.zero) : nullptr;
  const bool there = in_place(f);  // the weights stay there
  MmArgs p;
  if (there) {
    p = rows_of<T>(x, d, wg, h, f.tokens, h, d);
    p.half = static_cast<const char*>(wu) - static_cast<const char*>(wg);
  } else {
    TurnJobs jobs{};
    jobs.zero = zero;
    jobs.add(wg, W + L.tg, d, h, h);
    jobs.add(wu, W + L.tu, d, h, h);
    jobs.add(wd, W + L.td, h, d, d);
    turn<T>("ffn_turn_weights", jobs, s);
    PadJobs pads{};
    const void* xp = padded<T>(pads, x, W + L.xp, f.tokens, d);
    pad<T>(pads, s);
    p = rows_of<T>(xp, dp, W + L.tg, dp, f.tokens, h, dp);
    p.half = static_cast<int64_t>(L.tu) - static_cast<int64_t>(L.tg);
  }
  FfnOut o{};
  if (SV) o = saved_out(S, SV, hp);
  else o.h = W + L.h;
  o.ld = hp;
  if (there) o.zero = zero;
  tiles_act<T, kGated>("ffn_gate_up", f.act, p, o, s, there);
  MmArgs q = there ? rows_of<T>(o.h, hp, wd, d, f.tokens, d, h)
                   : rows_of<T>(o.h, hp, W + L.td, hp, f.tokens, d, hp);
  product<T>("ffn_down", q, out, reinterpret_cast<float*>(W + L.k_sums), s, there);
  return hipGetLastError();
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

template <typename Cfg, int kMode>
void launch_grad(GradArgs& a, int parts, hipStream_t s) {
  int64_t tiles = 0;
  for (int i = 0; i < 3; ++i) {
    MmArgs& p = a.p[i];
    p.tiles_n = (p.N + Cfg::BN - 1) / Cfg::BN;
    p.nk *= 128 / Cfg::ROW;
    tiles += (p.M + Cfg::BM - 1) / Cfg::BM * p.tiles_n;
    a.end[i] = static_cast<int>(tiles);
  }
  MOE_LAUNCH("ffn_bwd_wgrad", (ffn_grad_kernel<Cfg, kMode>), dim3(static_cast<unsigned>(tiles * parts)),
             dim3(Cfg::NT), 0, s, a);
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

template <typename T, typename G>
hipError_t ffn_bwd_t(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                     const void* wd, const void* saved, const void* dy, void* dx, void* dwg,
                     void* dwu, void* dwd, void* ws, hipStream_t s) {
  const FfnBlockLayout L = ffn_block_layout(f, true);
  const SavedLayout S = saved_layout(f);
  char* W = static_cast<char*>(ws);
  const char* SV = static_cast<const char*>(saved);
  const int d = f.d_model, h = f.d_hidden;
  const int64_t dp = pad128(d), hp = pad128(h), tok = f.tokens;
  PadJobs pads{};
  [[maybe_unused]] const void* xp = x;
  if constexpr (std::is_same<T, bf16_t>::value) xp = padded<T>(pads, x, W + L.xp, tok, d);
  const void* dyp = padded<T>(pads, dy, W + L.dyp, tok, d);
  const void* wdp = padded<T>(pads, wd, W + L.wdp, h, d);
  const void* wgp = padded<T>(pads, wg, W + L.wgp, d, h);
  const void* wup = padded<T>(pads, wu, W + L.wup, d, h);
  pad<T>(pads, s);

  MmArgs p = rows_of<T>(dyp, dp, wdp, dp, tok, h, dp);
  FfnOut o = saved_out(S, const_cast<char*>(SV), hp);
  o.dab = W + L.dab;
  tiles<T, kGatedGrad, 0>("ffn_bwd_down", p, o, s);

  MmArgs q = rows_of<T>(W + L.dab, 2 * hp, wgp, hp, tok, d, hp);
  q.k_split = q.nk;
  q.nk *= 2;
  q.a2 = W + L.dab + hp * sizeof(T);
  q.b2 = static_cast<const char*>(wup);
  product<T>("ffn_bwd_gate_up", q, dx, reinterpret_cast<float*>(W + L.k_sums), s);

  float* gu = reinterpret_cast<float*>(W + L.part_gu);
  float* dn = reinterpret_cast<float*>(W + L.part_d);
  SliceJobs jobs{};
  int64_t end = 0;
  auto job = [&](const float* part, int splits, int64_t stride, int64_t ld, int M, int N, void* out) {
    end += static_cast<int64_t>(M) * ((N + 3) / 4);
    jobs.job[jobs.n++] = SliceJob{part, splits, stride, ld, M, N, out, end};
  };
  if constexpr (std::is_same<T, bf16_t>::value) {
    const void* zero = SV + S.zero;
    if (L.splits_gu == 1) {
      grad_direct<G>("ffn_bwd_wgrad_gate_up", xp, dp, W + L.dab, 2 * hp, dp, 2 * hp, tok, d, h, hp, dwg,
                     dwu, zero, s);
    } else {
      grad_slices<T>("ffn_bwd_wgrad_gate_up", xp, dp, W + L.dab, 2 * hp, dp, 2 * hp, tok, L.splits_gu,
                     gu, zero, s);
      job(gu, L.splits_gu, 2 * dp * hp, 2 * hp, d, h, dwg);
      job(gu + hp, L.splits_gu, 2 * dp * hp, 2 * hp, d, h, dwu);
    }
    if (L.splits_d == 1) {
      grad_direct<G>("ffn_bwd_wgrad_down", SV + S.h, hp, dyp, dp, hp, dp, tok, h, d, dp, dwd, dwd, zero, s);
    } else {
      grad_slices<T>("ffn_bwd_wgrad_down", SV + S.h, hp, dyp, dp, hp, dp, tok, L.splits_d, dn, zero, s);
      job(dn, L.splits_d, dp * hp, dp, h, d, dwd);
    }
  } else {
    // The tiles take rows of consecutive tokens, so fp32 operands are turned
    // first (their bytes are little beside fp32 MFMAs; a stage loop that reads
    // single elements of [tokens][columns] from LDS would do without) and the
    // gradients are plain products, written in place where the tokens are not
    // cut into slices. 777 tokens, 500 x 1001: 42 us, against 64 with row
    // slices turned in registers and their partial sums.
    TurnJobs turns{};
    turns.add(x, W + L.xt, tok, d, d);
    turns.add(W + L.dab, W + L.dabt, tok, static_cast<int>(2 * hp), 2 * hp);
    turns.add(SV + S.h, W + L.ht, tok, h, hp);
    turns.add(dy, W + L.dyt, tok, d, d);
    turn<T>("ffn_bwd_turn", turns, s);
    const int64_t tp = pad128(tok);
    GradArgs a{};
    const int parts = L.grad_parts;
    const int64_t h4 = (h + 3) / 4 * 4, d4 = (d + 3) / 4 * 4;  // rows of the slices' sums
    auto grad = [&](int i, const char* A, const char* B, int M, int N, void* out, float* sums, int64_t ld) {
      a.p[i] = rows_of<T>(A, tp, B, tp, M, N, tp);
      a.p[i].parts = parts;
      a.o[i].c = parts > 1 ? sums : out;
      a.o[i].ldc = parts > 1 ? ld : N;
      if (parts > 1) job(sums, parts, M * ld, ld, M, N, out);
    };
    const char* dabt = W + L.dabt;
    grad(0, W + L.xt, dabt, d, h, dwg, gu, h4);
    grad(1, W + L.xt, dabt + hp * tp * sizeof(T), d, h, dwu, gu + parts * d * h4, h4);
    grad(2, W + L.ht, W + L.dyt, h, d, dwd, dn, d4);
    if (parts > 1) launch_grad<MmSmall, kPart>(a, parts, s);
    else if (grad_tiles(f, 128) >= kCUs) launch_grad<MmMid, kPlain>(a, 1, s);
    else launch_grad<MmSmall, kPlain>(a, 1, s);
  }
  if (jobs.n)
    MOE_LAUNCH("ffn_slice_sum", slice_sum_kernel<G>, dim3(blocks_for(end)), dim3(256), 0, s, jobs);
  return hipGetLastError();
}

}  // namespace

size_t ffn_block_ws_bytes(const moe_ffn& f, bool training) {
  // a training workspace serves inference too
  size_t n = ffn_block_layout(f, false).total;
  if (training) n = std::max(n, ffn_block_layout(f, true).total);
  return align_up(n < 256 ? 256 : n, 256);
}
size_t ffn_block_saved_bytes(const moe_ffn& f) { return saved_layout(f).total; }

hipError_t launch_ffn_block(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                            const void* wd, void* saved, void* out, void* ws, hipStream_t s) {
  return f.dtype == MOE_BF16 ? ffn_fwd_t<bf16_t>(f, x, wg, wu, wd, saved, out, ws, s)
                             : ffn_fwd_t<float>(f, x, wg, wu, wd, saved, out, ws, s);
}

hipError_t launch_ffn_block_bwd(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                                const void* wd, const void* saved, const void* dy, void* dx,
                                void* dwg, void* dwu, void* dwd, void* ws, hipStream_t s) {
  if (f.tokens == 0) {
    const int64_t n = static_cast<int64_t>(f.d_model) * f.d_hidden;
    for (void* g : {dwg, dwu, dwd}) {
      if (f.grad_dtype == MOE_BF16)
        MOE_LAUNCH("ffn_zero", zero_kernel<bf16_t>, dim3(blocks_for(n)), dim3(256), 0, s,
                   static_cast<bf16_t*>(g), n);
      else
        MOE_LAUNCH("ffn_zero", zero_kernel<float>, dim3(blocks_for(n)), dim3(256), 0, s,
                   static_cast<float*>(g), n);
    }
    return hipGetLastError();
  }
  if (f.dtype != MOE_BF16)
    return ffn_bwd_t<float, float>(f, x, wg, wu, wd, saved, dy, dx, dwg, dwu, dwd, ws, s);
  return f.grad_dtype == MOE_BF16
             ? ffn_bwd_t<bf16_t, bf16_t>(f, x, wg, wu, wd, saved, dy, dx, dwg, dwu, dwd, ws, s)
             : ffn_bwd_t<bf16_t, float>(f, x, wg, wu, wd, saved, dy, dx, dwg, dwu, dwd, ws, s);
}

}  // namespace moe
