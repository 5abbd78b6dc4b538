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
// gradients read them as they are. The weight gradients reduce over tokens,
// in slices whose partial sums are added in a fixed order.
//
// Widths that are no multiple of 128 take zero-padded copies of the operands
// in the workspace (x and dout, and the weights the backward reads), with the
// hidden values kept at the padded width.
#include <algorithm>

#include "gemm_wgrad.h"
#include "mm.h"

namespace moe {

namespace {

constexpr int64_t pad128(int64_t v) { return (v + 127) / 128 * 128; }
size_t elem_bytes(const moe_ffn& f) { return f.dtype == MOE_BF16 ? 2 : 4; }

// ------------------------------------------------------------- activations

template <int kAct>
__device__ __forceinline__ float act_value(float a, float* slope) {
  if (kAct == MOE_ACT_RELU) {
    *slope = a > 0.0f ? 1.0f : 0.0f;
    return fmaxf(a, 0.0f);
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
    *slope = s + a * 2.0f * s * (1.0f - s) * k * (1.0f + 3.0f * c * a * a);
    return a * s;
  }
  const float s = sigmoid_f(a);
  *slope = s * (1.0f + a * (1.0f - s));
  return a * s;
}

// ---------------------------------------------------------- layout changes

// dst[n][kp] from src[k][n]: 32 x 32 blocks through LDS; zeros for k >= K.
template <typename T>
__global__ __launch_bounds__(256) void turn_kernel(const T* __restrict__ src, T* __restrict__ dst,
                                                   int K, int N, int64_t kp) {
  __shared__ T tile[32][33];
  const int n0 = blockIdx.x * 32, k0 = blockIdx.y * 32;
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = k0 + r + 8 * i, n = n0 + c;
    tile[r + 8 * i][c] = (k < K && n < N) ? src[static_cast<int64_t>(k) * N + n] : T{};
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + r + 8 * i, k = k0 + c;
    if (n < N && k < kp) dst[n * kp + k] = tile[c][r + 8 * i];
  }
}

// dst[r][wp] = src[r][w], zeros from w on.
template <typename T>
__global__ __launch_bounds__(256) void pad_rows_kernel(const T* __restrict__ src, T* __restrict__ dst,
                                                       int64_t rows, int w, int wp) {
  constexpr int V = Piece<T>::V;
  const int per = wp / V;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < rows * per;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / per;
    const int c = static_cast<int>(i % per) * V;
    *reinterpret_cast<u32x4*>(dst + r * wp + c) = load_piece(src + r * w, c, w);
  }
}

// ----------------------------------------------------------------- products

struct FfnOut {
  void* c;        // plain: the result
  int64_t ldc;
  void *h, *a, *b;  // gated: hidden values and (training) both pre-activations
  const void *sa, *sb;  // gradient: the pre-activations read
  void *da, *db;        // gradient: the results
  int64_t ld;           // columns kept of the hidden matrices (a multiple of 128)
};

// Columns n .. n + 3 of a row that keeps `width` columns.
template <typename T>
__device__ __forceinline__ void store4_any(T* row, int n, int64_t width, const float (&v)[4]) {
  if (n + 4 <= width && width % 4 == 0) {
    store4(row + n, v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (n + q < width) put(row + n + q, v[q]);
}

enum { kPlain = 0, kGated = 1, kGatedGrad = 2 };

template <typename T>
struct OpOf {
  typedef OpBf16 type;
};
template <>
struct OpOf<float> {
  typedef OpF32 type;
};

template <typename T, typename Cfg, int kMode, int kAct>
__global__ __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(Cfg::NT == 512 ? 2 : 1)))
void ffn_tile_kernel(const MmArgs p, const FfnOut o) {
  __shared__ __attribute__((aligned(1024))) char smem[2 * Cfg::STAGE];
  f32x16_t acc[Cfg::WM][Cfg::WN];
  MmTile t;
  if (!mm_tile<typename OpOf<T>::type, Cfg, kMode == kGated>(p, smem, &t, acc)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 5, r32 = lane & 31;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
#pragma unroll
  for (int i = 0; i < Cfg::WM; ++i) {
    const int m = (wm * Cfg::WM + i) * 32 + r32;
    if (m >= t.rows) continue;
    const int64_t row = t.row0 + m;
#pragma unroll
    for (int j = 0; j < Cfg::WN; ++j) {
      const int n0 = t.nt * Cfg::BN + (wn * Cfg::WN + j) * 32;
#pragma unroll
      for (int rr = 0; rr < (kMode == kGated ? 2 : 4); ++rr) {
        const int n = (kMode == kGated ? n0 / 2 : n0) + 8 * rr + 4 * g;
        if (kMode == kPlain) {
          const float v[4] = {acc[i][j][4 * rr], acc[i][j][4 * rr + 1], acc[i][j][4 * rr + 2],
                              acc[i][j][4 * rr + 3]};
          store4_any(static_cast<T*>(o.c) + row * o.ldc, n, o.ldc, v);
          continue;
        }
        if (n >= o.ld) continue;
        if (kMode == kGated) {
          float h[4], a[4], b[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bool in = n + q < p.N;  // zeros in the padding
            a[q] = in ? acc[i][j][4 * rr + q] : 0.0f;
            b[q] = in ? acc[i][j][4 * rr + 8 + q] : 0.0f;
            float slope;
            h[q] = act_value<kAct>(a[q], &slope) * b[q];
          }
          store4(static_cast<T*>(o.h) + row * o.ld + n, h[0], h[1], h[2], h[3]);
          if (o.a) {
            store4(static_cast<T*>(o.a) + row * o.ld + n, a[0], a[1], a[2], a[3]);
            store4(static_cast<T*>(o.b) + row * o.ld + n, b[0], b[1], b[2], b[3]);
          }
        } else {
          float a[4], b[4], da[4], db[4];
          load4(static_cast<const T*>(o.sa) + row * o.ld + n, a);
          load4(static_cast<const T*>(o.sb) + row * o.ld + n, b);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float dh = n + q < p.N ? acc[i][j][4 * rr + q] : 0.0f;
            float slope;
            const float f = act_value<kAct>(a[q], &slope);
            da[q] = dh * b[q] * slope;
            db[q] = dh * f;
          }
          store4(static_cast<T*>(o.da) + row * o.ld + n, da[0], da[1], da[2], da[3]);
          store4(static_cast<T*>(o.db) + row * o.ld + n, db[0], db[1], db[2], db[3]);
        }
      }
    }
  }
}

// Weight gradients from the slices' partial sums [splits][Mp][Np], cropped to
// M x N and rounded once: the slices are added in order.
template <typename G>
__global__ __launch_bounds__(256) void slice_sum_kernel(const float* __restrict__ part, int splits,
                                                        int64_t mp, int64_t np, int M, int N,
                                                        G* __restrict__ out) {
  const int per = (N + 3) / 4;
  const int64_t total = static_cast<int64_t>(M) * per, stride = mp * np / 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t m = i / per;
    const int n = static_cast<int>(i % per) * 4;
    const float4* src = reinterpret_cast<const float4*>(part + m * np + n);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kBatch = 8;
    int s = 0;
    for (; s + kBatch <= splits; s += kBatch) {
      float4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) v[u] = src[(s + u) * stride];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        acc.x += v[u].x; acc.y += v[u].y; acc.z += v[u].z; acc.w += v[u].w;
      }
    }
    for (; s < splits; ++s) {
      const float4 v = src[s * stride];
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    const float v[4] = {acc.x, acc.y, acc.z, acc.w};
    store4_any(out + m * N, n, N, v);
  }
}

template <typename G>
__global__ __launch_bounds__(256) void zero_kernel(G* __restrict__ p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = G{};
}

// ------------------------------------------------------------------ layouts

struct FfnBlockLayout {
  // forward workspace: turned weights, padded x, hidden values (inference)
  size_t tg, tu, td, xp, h;
  // backward workspace
  size_t dyp, wgp, wup, wdp, da, db, part, zero;
  size_t total;
  int splits_gu, splits_d;
};

int slices(int64_t rows, int64_t tiles) {
  int64_t k = (512 + tiles - 1) / tiles;
  k = k < 1 ? 1 : (k > 64 ? 64 : k);
  const int64_t most = (rows + 63) / 64;  // a stage of 64 rows each at least
  return static_cast<int>(k > most ? (most < 1 ? 1 : most) : k);
}

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
  L.xp = take(d == dp ? 0 : T * dp * es);
  const size_t start = o;
  L.tg = take(h * dp * es);
  L.tu = take(h * dp * es);
  L.td = take(d * hp * es);
  if (!training) L.h = take(T * hp * es);
  L.total = o;
  if (training) {
    // the backward reuses the turned weights' place
    o = start;
    L.dyp = take(d == dp ? 0 : T * dp * es);
    L.wgp = take(h == hp ? 0 : d * hp * es);
    L.wup = take(h == hp ? 0 : d * hp * es);
    L.wdp = take(d == dp ? 0 : h * dp * es);
    L.da = take(T * hp * es);
    L.db = take(T * hp * es);
    const int64_t tiles = static_cast<int64_t>(dp / 128) * (hp / 128);
    L.splits_gu = slices(f.tokens, 2 * tiles);
    L.splits_d = slices(f.tokens, tiles);
    const size_t gu = static_cast<size_t>(L.splits_gu) * 2, dn = L.splits_d;
    L.part = take((gu > dn ? gu : dn) * dp * hp * sizeof(float));
    L.zero = take(kTrZeroBytes);
    if (o > L.total) L.total = o;
  }
  return L;
}

struct SavedLayout {
  size_t a, b, h, total;
};
SavedLayout saved_layout(const moe_ffn& f) {
  const size_t n = align_up(static_cast<size_t>(f.tokens) * pad128(f.d_hidden) * elem_bytes(f), 256);
  return SavedLayout{0, n, 2 * n, 3 * n};
}

// ----------------------------------------------------------------- launches

template <typename T, typename Cfg, int kMode, int kAct>
void tiles_at(const char* name, const MmArgs& a, const FfnOut& o, hipStream_t s) {
  MmArgs p = a;
  const int per = kMode == kGated ? Cfg::BN / 2 : Cfg::BN;
  // the hidden matrices are written to their padded width
  const int64_t n = kMode == kPlain ? p.N : o.ld;
  p.tiles_n = static_cast<int>((n + per - 1) / per);
  const int64_t grid = (p.M + Cfg::BM - 1) / Cfg::BM * p.tiles_n;
  MOE_LAUNCH(name, (ffn_tile_kernel<T, Cfg, kMode, kAct>), dim3(static_cast<unsigned>(grid)),
             dim3(Cfg::NT), 0, s, p, o);
}

template <typename T, int kMode, int kAct>
void tiles(const char* name, const MmArgs& p, const FfnOut& o, hipStream_t s) {
  using Big = MmCfg<256, 256, 4, 2>;
  using Mid = MmCfg<128, 128, 2, 2>;
  using Low = MmCfg<32, 128, 1, 4>;
  const int64_t cols = kMode == kGated ? 2 * static_cast<int64_t>(p.N) : p.N;
  const int64_t big = (p.M + 255) / 256 * ((cols + 255) / 256);
  if (sizeof(T) == 2 && big >= cu_count()) tiles_at<T, Big, kMode, kAct>(name, p, o, s);
  else if (p.M > 32) tiles_at<T, Mid, kMode, kAct>(name, p, o, s);
  else tiles_at<T, Low, kMode, kAct>(name, p, o, s);
}

template <typename T, int kMode>
void tiles_act(const char* name, int act, const MmArgs& p, const FfnOut& o, hipStream_t s) {
  switch (act) {
    case MOE_ACT_SILU: return tiles<T, kMode, MOE_ACT_SILU>(name, p, o, s);
    case MOE_ACT_GELU: return tiles<T, kMode, MOE_ACT_GELU>(name, p, o, s);
    case MOE_ACT_GELU_TANH: return tiles<T, kMode, MOE_ACT_GELU_TANH>(name, p, o, s);
    default: return tiles<T, kMode, MOE_ACT_RELU>(name, p, o, s);
  }
}

unsigned blocks_for(int64_t items) {
  const int64_t b = (items + 255) / 256;
  return static_cast<unsigned>(b < 1 ? 1 : (b > 8192 ? 8192 : b));
}

template <typename T>
void turn(const void* src, void* dst, int K, int N, int64_t kp, hipStream_t s) {
  MOE_LAUNCH("ffn_turn_weights", turn_kernel<T>,
             dim3((N + 31) / 32, static_cast<unsigned>((kp + 31) / 32)), dim3(256), 0, s,
             static_cast<const T*>(src), static_cast<T*>(dst), K, N, kp);
}

template <typename T>
const void* padded(const void* src, char* dst, int64_t rows, int w, hipStream_t s) {
  const int wp = static_cast<int>(pad128(w));
  if (w == wp) return src;
  MOE_LAUNCH("ffn_pad_rows", pad_rows_kernel<T>, dim3(blocks_for(rows * (wp / Piece<T>::V))),
             dim3(256), 0, s, static_cast<const T*>(src), reinterpret_cast<T*>(dst), rows, w, wp);
  return dst;
}

template <typename T>
MmArgs rows_of(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t M, int N, int64_t K) {
  MmArgs p{};
  p.a = static_cast<const char*>(a);
  p.a_pitch = lda * static_cast<int64_t>(sizeof(T));
  p.b = static_cast<const char*>(b);
  p.b_pitch = ldb * static_cast<int64_t>(sizeof(T));
  p.nk = static_cast<int>(K * static_cast<int64_t>(sizeof(T)) / kMmRow);
  p.M = M;
  p.N = N;
  return p;
}

template <typename T>
hipError_t ffn_fwd_t(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                     const void* wd, void* saved, void* out, void* ws, hipStream_t s) {
  const FfnBlockLayout L = ffn_block_layout(f, saved != nullptr);
  const SavedLayout S = saved_layout(f);
  char *W = static_cast<char*>(ws), *SV = static_cast<char*>(saved);
  const int d = f.d_model, h = f.d_hidden;
  const int64_t dp = pad128(d), hp = pad128(h);
  turn<T>(wg, W + L.tg, d, h, dp, s);
  turn<T>(wu, W + L.tu, d, h, dp, s);
  turn<T>(wd, W + L.td, h, d, hp, s);
  const void* xp = padded<T>(x, W + L.xp, f.tokens, d, s);
  MmArgs p = rows_of<T>(xp, dp, W + L.tg, dp, f.tokens, h, dp);
  p.half = static_cast<int64_t>(L.tu) - static_cast<int64_t>(L.tg);
  FfnOut o{};
  o.h = SV ? SV + S.h : W + L.h;
  o.a = SV ? SV + S.a : nullptr;
  o.b = SV ? SV + S.b : nullptr;
  o.ld = hp;
  tiles_act<T, kGated>("ffn_gate_up", f.act, p, o, s);
  MmArgs q = rows_of<T>(o.h, hp, W + L.td, hp, f.tokens, d, hp);
  FfnOut c{};
  c.c = out;
  c.ldc = d;
  tiles<T, kPlain, 0>("ffn_down", q, c, s);
  return hipGetLastError();
}

template <typename T, typename G>
void grad_weight(const char* name, const void* a, int64_t lda, const void* b, int64_t ldb, int M,
                 int N, int64_t rows, int splits, float* part, const void* zero, void* out,
                 hipStream_t s) {
  const int64_t mp = pad128(M), np = pad128(N);
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
  if (std::is_same<T, bf16_t>::value) {
    wgrad_tr<true>(name, w, splits, static_cast<const bf16_t*>(zero), s);
  } else {
    const int64_t blocks = splits * (mp / 128) * (np / 128);
    MOE_LAUNCH(name, (wgrad_kernel<float, false, true>), dim3(static_cast<unsigned>(blocks)),
               dim3(256), 0, s, w);
  }
  MOE_LAUNCH("ffn_slice_sum", slice_sum_kernel<G>,
             dim3(blocks_for(static_cast<int64_t>(M) * ((N + 3) / 4))), dim3(256), 0, s, part,
             splits, mp, np, M, N, static_cast<G*>(out));
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
  const void* xp = padded<T>(x, W + L.xp, tok, d, s);
  const void* dyp = padded<T>(dy, W + L.dyp, tok, d, s);
  const void* wdp = padded<T>(wd, W + L.wdp, h, d, s);
  const void* wgp = padded<T>(wg, W + L.wgp, d, h, s);
  const void* wup = padded<T>(wu, W + L.wup, d, h, s);

  MmArgs p = rows_of<T>(dyp, dp, wdp, dp, tok, h, dp);
  FfnOut o{};
  o.sa = SV + S.a;
  o.sb = SV + S.b;
  o.da = W + L.da;
  o.db = W + L.db;
  o.ld = hp;
  tiles_act<T, kGatedGrad>("ffn_bwd_down", f.act, p, o, s);

  MmArgs q = rows_of<T>(o.da, hp, wgp, hp, tok, d, hp);
  q.k_split = q.nk;
  q.nk *= 2;
  q.a2 = static_cast<const char*>(o.db);
  q.b2 = static_cast<const char*>(wup);
  FfnOut c{};
  c.c = dx;
  c.ldc = d;
  tiles<T, kPlain, 0>("ffn_bwd_gate_up", q, c, s);

  float* part = reinterpret_cast<float*>(W + L.part);
  MOE_LAUNCH("ffn_zero", zero_kernel<uint32_t>, dim3(1), dim3(256), 0, s,
             reinterpret_cast<uint32_t*>(W + L.zero), static_cast<int64_t>(kTrZeroBytes / 4));
  grad_weight<T, G>("ffn_bwd_wgrad", xp, dp, o.da, hp, d, h, tok, L.splits_gu, part, W + L.zero, dwg, s);
  grad_weight<T, G>("ffn_bwd_wgrad", xp, dp, o.db, hp, d, h, tok, L.splits_gu, part, W + L.zero, dwu, s);
  grad_weight<T, G>("ffn_bwd_wgrad", SV + S.h, hp, dyp, dp, h, d, tok, L.splits_d, part, W + L.zero, dwd, s);
  return hipGetLastError();
}

}  // namespace

size_t ffn_block_ws_bytes(const moe_ffn& f, bool training) {
  // a training workspace serves inference too
  size_t n = ffn_block_layout(f, false).total;
  if (training) n = std::max(n, ffn_block_layout(f, true).total);
  return n < 256 ? 256 : n;
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
