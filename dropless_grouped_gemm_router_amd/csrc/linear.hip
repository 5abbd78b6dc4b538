// Matrix product with bias, activation and residual in its epilogue, forward
// and backward.
//
//   a = x W + bias, y = act(a) + residual
//   da = dy act'(a), dx = da W^T, dW = x^T da, dbias = sum_rows da
//
// The forward is one product; what follows it is done on the sums while they
// are in registers, where the tile's rows are handed out (mm_drain): the
// residual's rows are read one strip ahead, y is rounded once, and the slope
// act'(a) is kept for the backward, in bf16 in 20 bits of fixed point (slopes lie
// in [-0.13, 1.13]; 2.5 bytes a value and off by at most 6.4e-7: 6e-7 in the 2-norm of
// dbias, which is fp32 and has no other rounding. A slope of fp16, 2 bytes, made
// 2.2e-4 of that, one of a bf16 pre-activation would make 2e-3).
//
// The weights come [inputs][outputs]: the forward runs over their leading
// dimension, so it turns them K-contiguous first or, in bf16 up to some
// thousand tokens, reads them where they are (in_place); up to 16 tokens it reads
// them once, straight into MFMA operands (skinny.h), and in fp32 up to 128, once for
// every 16. The
// backward's dx reads them as they are. da is made in one pass over dy that
// also adds up dbias and pads the rows; without an activation dy itself is da.
//
// Up to 16 bf16 rows keep da unrounded, in a backward pass of one launch
// (lin_few_bwd_kernel) or, where weights are large, in tiles (lin_halves_kernel), and
// fp32 products of moderate size take both passes' operands from memory as they
// are, in one launch each (direct.h).
#include "dense.h"
#include "direct.h"

namespace moe {

namespace {

constexpr int64_t kFewRows = 16, kFewRowsF32 = 128;
// The serving form's workgroups: 16 waves over the whole of K where that is short,
// else slices of K to 8 waves each and a second launch that adds them. One row,
// bf16, one slice and slices: 1024 x 4096 7.3 and 10.5 us, 700 x 1001 7.4 and 10.8,
// 4096 x 4096 11.8 and 10.5, 8192 x 2048 20 and 11; 8 rows, 2048 x 8192 8.4 and 10.9;
// fp32, 64 rows, 512 x 2048 8.1 and 8.4, 16 rows, 1024 x 1024 12.8 and 10.9.
constexpr int kRowsWaves = 16, kShortK = 2048, kShortKF32 = 512;

// The backward of few rows in one launch; a training pass so and in tiles
// (lin_halves_kernel), us: 1 x 512 x 512 15 and 22, 16 x 512 x 4096 22 and 22, 16 x 2048 x
// 2048 24 and 25, 2 x 8192 x 2048 35 and 35; past its limits 16 x 128 x 16384 64 and 22, 16 x
// 65536 x 64 67 and 42, 16 x 4096 x 4096 56 and 37.
constexpr int kFewInputs = 8192, kFewOutputs = 4096;
constexpr int64_t kFewProducts = int64_t{1} << 26;

int64_t pad4(int64_t v) { return (v + 3) / 4 * 4; }
size_t elem_bytes(const moe_linear& l) { return l.dtype == MOE_BF16 ? 2 : 4; }
bool few_rows(const moe_linear& l) { return l.tokens <= (l.dtype == MOE_BF16 ? kFewRows : kFewRowsF32); }
// Elements between rows of the kept slopes.
int64_t slope_pitch(const moe_linear& l) { return (l.outputs + 7) / 8 * 8; }

// A kept slope of the bf16 form: 3 2^18 slope + 2^17, rounded, in 20 bits, as the
// low bits of a number from 2^23 on; 0, which no slope gives, for a NaN. Slopes of 0
// and 1 come back as they were.
__device__ __forceinline__ uint32_t slope_code(float v) {
  return __float_as_uint(fmaxf(__builtin_fmaf(v, 786432.0f, 8388608.0f + 131072.0f), 8388608.0f)) & 0xfffff;
}
__device__ __forceinline__ float slope_of(uint32_t code) {
  return code ? __builtin_fmaf(static_cast<float>(code), 1.0f / 786432.0f, -1.0f / 6.0f) : __builtin_nanf("");
}

// Where slopes are kept: [rows][ld] of T's type, fp32 numbers or the codes' high
// 16 bits, and behind these their low four, two to a byte.
template <typename T>
struct Slopes;
template <>
struct Slopes<float> {
  float* p;
  int64_t ld;
  __device__ void put8(int64_t row, int n, const float (&v)[8]) const {
    float* d = p + row * ld + n;
    store4(d, v[0], v[1], v[2], v[3]);
    store4(d + 4, v[4], v[5], v[6], v[7]);
  }
  struct Raw {
    u32x4 a, b;
  };
  __device__ Raw load8(int64_t row, int n) const {
    const u32x4* s = reinterpret_cast<const u32x4*>(p + row * ld + n);
    return Raw{s[0], s[1]};
  }
  __device__ static void get8(const Raw& r, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(q < 4 ? r.a[q] : r.b[q - 4]);
  }
  // One column a lane, the next lane having the next one; `in`: the lane has one.
  __device__ void put1(int64_t row, int n, bool in, float v) const {
    if (in) p[row * ld + n] = v;
  }
};
template <>
struct Slopes<bf16_t> {
  uint16_t* p;
  int64_t ld;
  uint8_t* low;
  __device__ void put8(int64_t row, int n, const float (&v)[8]) const {
    u32x4 h;
    uint32_t l = 0;
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
      const uint32_t a = slope_code(v[q]), b = slope_code(v[q + 1]);
      h[q / 2] = (a >> 4) | (b >> 4 << 16);
      l |= ((a & 15) | (b & 15) << 4) << 4 * q;
    }
    *reinterpret_cast<u32x4*>(p + row * ld + n) = h;
    *reinterpret_cast<uint32_t*>(low + (row * ld + n) / 2) = l;
  }
  struct Raw {
    u32x4 high;
    uint32_t low;
  };
  __device__ Raw load8(int64_t row, int n) const {
    return Raw{*reinterpret_cast<const u32x4*>(p + row * ld + n),
               *reinterpret_cast<const uint32_t*>(low + (row * ld + n) / 2)};
  }
  __device__ static void get8(const Raw& r, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      v[q] = slope_of(((q & 1 ? r.high[q / 2] >> 16 : r.high[q / 2] & 0xffff) << 4) | (r.low >> 4 * q & 15));
  }
  __device__ void put1(int64_t row, int n, bool in, float v) const {
    const uint32_t code = slope_code(v);
    const uint32_t next = __float_as_uint(dpp<0xb1>(__uint_as_float(code)));  // lane ^ 1
    if (!in) return;
    p[row * ld + n] = static_cast<uint16_t>(code >> 4);
    if (n % 2 == 0) low[(row * ld + n) / 2] = static_cast<uint8_t>((code & 15) | (next & 15) << 4);
  }
};

// act(a) and its slope. In bf16 GELU's Phi(-|a|) is exp(-a^2 / 2) R(|a|), R
// (0.5 exp(x^2 / 2) erfc(x / sqrt 2)) as t p(t), t = 1 / (1 + 0.285 x), with p of
// degree 8 fitted to the smallest largest relative error, 4.8e-7 over all x in
// fp32, so that Phi is off by at most 2.2e-7, less than the slopes' rounding (degree
// 6: 4e-6, which showed in dbias). One exponential serves
// the value and the slope. (erff's two branches, 32 times eight of them, were
// more than the compiler would unroll in a 256 x 256 tile.) fp32 takes erff.
template <typename T, int kAct>
__device__ __forceinline__ float lin_act(float a, float* slope) {
  if constexpr (kAct == MOE_ACT_GELU && sizeof(T) == 2) {
    const float x = fabsf(a), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.285f, x, 1.0f));
    float p = 0.0245698374f;
    p = __builtin_fmaf(p, t, -0.0865935981f);
    p = __builtin_fmaf(p, t, 0.0739199519f);
    p = __builtin_fmaf(p, t, 0.00349686155f);
    p = __builtin_fmaf(p, t, 0.0675795525f);
    p = __builtin_fmaf(p, t, 0.0851249918f);
    p = __builtin_fmaf(p, t, 0.104505382f);
    p = __builtin_fmaf(p, t, 0.113698572f);
    p = __builtin_fmaf(p, t, 0.113698535f);
    const float e = __expf(-0.5f * a * a), tail = e * (p * t);
    const float cdf = a < 0.0f ? tail : 1.0f - tail;
    *slope = __builtin_fmaf(a * 0.39894228f, e, cdf);
    return a * cdf;
  }
  return act_value<kAct>(a, slope);
}

template <typename T>
struct LinOut {
  void* y;           // [M][ld], or fp32 sums [parts][M][ld] of the slices of K
  int64_t ld;
  const float* bias;  // or null
  const void* res;    // [M][N], or null
  Slopes<T> slope;    // p null: not kept
  int64_t M;
  int N;
  u32x4* zero;        // null, or kTrZeroBytes that the product clears on the way
};

// Eight elements c.. of a row of n, widened; zeros behind the row.
template <typename T, bool kFull>
__device__ __forceinline__ void load8(const T* row, int c, int n, float (&v)[8]) {
  constexpr int V = Piece<T>::V;
#pragma unroll
  for (int h = 0; h < 8 / V; ++h) {
    const int at = c + h * V;
    u32x4 p = (u32x4){0u, 0u, 0u, 0u};
    if (kFull) p = load_any(row + at);
    else if (at < n) p = load_piece(row, at, n);
    float e[V];
    Piece<T>::widen(p, e);
#pragma unroll
    for (int q = 0; q < V; ++q) v[h * V + q] = e[q];
  }
}

// The callbacks of mm_drain. kPart: the slice's sums as they are; kFull: every
// column of the tile is below N.
template <typename T, typename Cfg, int kAct, bool kPart, bool kFull>
struct LinRows {
  static constexpr int kJ = Cfg::WN / MmStrip<Cfg>::CB, kPasses = mm_passes<Cfg, false>();
  static constexpr int kPieces = 8 / Piece<T>::V;
  const MmTile& t;
  const LinOut<T>& o;
  int base, n[kJ];
  float bias[kPart ? 1 : kJ][8];
  u32x4 res[kPart ? 1 : 2][kPasses][kPieces];

  __device__ void cols(int j, int c) {
    n[j] = base + c;
    if constexpr (!kPart) {
#pragma unroll
      for (int q = 0; q < 8; ++q) bias[j][q] = 0.0f;
      if (o.bias) load8<float, kFull>(o.bias, n[j], o.N, bias[j]);
    }
  }
  __device__ void start(int, int, int) {}
  __device__ void pre(int set, int j, int k, int m) {
    if constexpr (!kPart) {
      if (!o.res) return;
      const T* row = static_cast<const T*>(o.res) + (t.row0 + m) * o.N;
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        const int c = n[j] + h * Piece<T>::V;
        if (kFull) res[set][k][h] = load_any(row + c);
        else if (c < o.N) res[set][k][h] = load_piece(row, c, o.N);
      }
    }
  }
  __device__ void row(int set, int, int j, int k, int m, const uint32_t (&v)[8]) {
    const int64_t row = t.row0 + m;
    float y[8];
    if constexpr (kPart) {
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = __uint_as_float(v[q]);
      store8<float, kFull>(static_cast<float*>(o.y) + (t.part * o.M + row) * o.ld, n[j], o.N, y);
    } else {
      float slope[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = lin_act<T, kAct>(__uint_as_float(v[q]) + bias[j][q], &slope[q]);
      if (o.res) {
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
          constexpr int V = Piece<T>::V;
          float r[V];
          Piece<T>::widen(res[set][k][h], r);
#pragma unroll
          for (int q = 0; q < V; ++q) y[h * V + q] += r[q];
        }
      }
      store8<T, kFull>(static_cast<T*>(o.y) + row * o.ld, n[j], o.N, y);
      if (kAct != MOE_ACT_NONE && o.slope.p && (kFull || n[j] < o.N)) o.slope.put8(row, n[j], slope);
    }
  }
};

// One tile of x W (or of da W^T) through LDS, and what follows the sums as the tile's
// rows are handed out. 16384 x 512 x 2048 bf16 with bias, SiLU, its slopes and a
// residual: 81 us for 240 MB (47) and 34 GF (28): the loop of eight short stages, the
// epilogue's arithmetic and its bytes follow each other within a tile (MFMA 22% busy,
// 3 TB/s). The same without what follows, as the backward's dx: 42 us, 0.8 PF.
template <typename T, typename Cfg, int kAct, bool kPart, bool kTurned>
__global__ __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(Cfg::WPE)))
void lin_tile_kernel(const MmArgs p, const LinOut<T> o) {
  __shared__ __attribute__((aligned(1024))) char smem[MmStrip<Cfg>::LDS];
  f32x16_t acc[Cfg::WM][Cfg::WN];
  MmTile t;
  if (o.zero && blockIdx.x == 0 && threadIdx.x < kTrZeroBytes / 16)
    o.zero[threadIdx.x] = (u32x4){0u, 0u, 0u, 0u};
  if (!mm_find<Cfg>(p, &t)) return;
  auto go = [&](auto full) {
    LinRows<T, Cfg, kAct, kPart, decltype(full)::value> rows{t, o, t.nt * Cfg::BN};
    mm_begin<Cfg, false>(t.rows, rows);
    mm_drain<Cfg, false>(smem, acc, t.rows, rows);
  };
  mm_tile<typename OpOf<T>::type, Cfg, false, kTurned>(p, smem, t, acc);
  if ((t.nt + 1) * Cfg::BN <= p.N) go(std::true_type{});
  else go(std::false_type{});
}

// One output from its sum, a column a lane; `in`: the lane has one.
template <typename T, int kAct>
__device__ __forceinline__ void finish(const LinOut<T>& o, int64_t row, int n, bool in, float sum) {
  float slope = 0.0f;
  if (in) {
    float y = lin_act<T, kAct>(sum + (o.bias ? o.bias[n] : 0.0f), &slope);
    if (o.res) y += elem(static_cast<const T*>(o.res) + row * o.N + n);
    put(static_cast<T*>(o.y) + row * o.ld + n, y);
  }
  if (kAct != MOE_ACT_NONE && o.slope.p) o.slope.put1(row, n, in, slope);
}

// Outputs from the sums of the slices of K, added in order; blockIdx.y: the row.
template <typename T, int kAct>
__global__ __launch_bounds__(256) void lin_join_kernel(const float* __restrict__ part, int parts,
                                                       const LinOut<T> o) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int64_t row = blockIdx.y;
  const bool in = n < o.N;
  float v = 0.0f;
  if (in) {
#pragma unroll 8
    for (int p = 0; p < parts; ++p) v += part[(p * o.M + row) * o.N + n];
  }
  finish<T, kAct>(o, row, n, in, v);
}

// Few tokens. part: null (one slice of K), or the slices' sums [k_parts][rows][N].
template <typename T, int kAct, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void lin_rows_kernel(const SkinnyArgs<T, 1> a, const LinOut<T> o,
                                                               float* part) {
  __shared__ float lds[kWaves][kSkinnyLds];
  float sum[16 / kWaves][1];
  skinny_sums<T, 1, false, kWaves>(a, lds, sum);
#pragma unroll
  for (int v = 0; v < 16 / kWaves; ++v) {
    const int64_t row = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x >> 6) + kWaves * v;
    const int n = blockIdx.x * kSkinnyCols + (threadIdx.x & 63);
    const bool in = row < a.rows && n < a.N;
    if (!part) finish<T, kAct>(o, row, n, in, sum[v][0]);
    else if (in) part[(blockIdx.z * a.rows + row) * a.N + n] = sum[v][0];
  }
}

// da [rows][np] from dy [rows][n] and, kSlope, the slopes, zeros from column n
// on, and the sums of its columns, before they are rounded, over the rows of this
// workgroup's slice: part [gridDim.y][n4]. da and part may each be null. A
// workgroup takes 256 columns, 32 threads of eight side by side, of 32 rows at a
// time; a thread has four rows' loads on their way, none behind a branch. 16384 x
// 2048 bf16, 218 MB: 41 us (5.3 TB/s); in workgroups of 256 threads and single rows 60.
constexpr int kDaCols = 256, kDaRows = 32;
template <typename T, bool kSlope>
__global__ __launch_bounds__(32 * kDaRows) void lin_da_kernel(const T* __restrict__ dy, const Slopes<T> slope,
                                                              T* __restrict__ da, float* __restrict__ part,
                                                              int64_t rows, int n, int np, int n4) {
  constexpr int V = Piece<T>::V, kPieces = 8 / V, kBatch = 4;
  __shared__ float sums[kDaRows][kDaCols];
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int c = blockIdx.x * kDaCols + tx * 8;
  const int64_t r0 = rows * blockIdx.y / gridDim.y, r1 = rows * (blockIdx.y + 1) / gridDim.y;
  const int cs = min(c, static_cast<int>(slope.ld) - 8);  // slopes of columns there are
  float s[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) s[q] = 0.0f;
  for (int64_t r = r0 + ty; r < r1; r += kBatch * kDaRows) {
    u32x4 raw[kBatch][kPieces];
    typename Slopes<T>::Raw sl[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t row = min(r + u * kDaRows, r1 - 1);
#pragma unroll
      for (int h = 0; h < kPieces; ++h) raw[u][h] = load_near(dy + row * n, c + h * V, n);
      if constexpr (kSlope) sl[u] = slope.load8(row, cs);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float v[8], e[8];
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        float w[V];
        trim_piece<T>(raw[u][h], c + h * V, n);
        Piece<T>::widen(raw[u][h], w);
#pragma unroll
        for (int q = 0; q < V; ++q) v[h * V + q] = w[q];
      }
      if constexpr (kSlope) {
        Slopes<T>::get8(sl[u], e);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = c + q < n ? v[q] * e[q] : 0.0f;
      }
      if (r + u * kDaRows >= r1) break;
      if (da && c < np) store8<T, true>(da + (r + u * kDaRows) * np, c, np, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += v[q];
    }
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) sums[ty][tx * 8 + q] = s[q];
  __syncthreads();
  if (threadIdx.x >= kDaCols) return;
  const int col = blockIdx.x * kDaCols + threadIdx.x;
  float v = 0.0f;
#pragma unroll
  for (int r = 0; r < kDaRows; ++r) v += sums[r][threadIdx.x];
  if (col < n4) part[static_cast<int64_t>(blockIdx.y) * n4 + col] = v;
}

// --------------------------------------------------------- backward of few rows

// The backward pass of up to 16 bf16 rows in one launch, dy's rows times their
// slopes formed where they are used, in fp32. The first workgroups make dx, 16
// columns each: mfma 16x16x32 takes 16 rows of w and the rows of da as they lie in
// memory, eight waves share the outputs, and da goes in as two bf16 numbers, of which
// the second holds what the first one rounds away (one row's da would err in every
// term alike). In the others a wave makes 64 x 64 of dW, eight by eight a lane in
// plain fp32. 16 rows, 1024 x 1024: a training pass 18 us, with its products in tiles 22;
// the backward alone at 2048 x 2048, 1
// row to 16: 13 to 18 us (24 MB: 5), bound by the lanes' additions.
constexpr int kFewWaves = 8, kFewTile = 64, kFewCols = 16;
// da of eight columns from c on, zeros from column n on.
template <bool kSlope>
__device__ __forceinline__ void few_da(u32x4 raw, const Slopes<bf16_t>::Raw& sl, int c, int n, float (&v)[8]) {
  trim_piece<bf16_t>(raw, c, n);
  Piece<bf16_t>::widen(raw, v);
  if constexpr (kSlope) {
    float e[8];
    Slopes<bf16_t>::get8(sl, e);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = c + q < n ? v[q] * e[q] : 0.0f;
  }
}
__device__ __forceinline__ f32x4_t few_mfma(const u32x4& a, const u32x4& b, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}
template <typename G, bool kSlope>
__global__ __launch_bounds__(64 * kFewWaves) void lin_few_bwd_kernel(
    const bf16_t* __restrict__ x, const bf16_t* __restrict__ w, const bf16_t* __restrict__ dy,
    const Slopes<bf16_t> slope, bf16_t* __restrict__ dx, G* __restrict__ dw, float* __restrict__ dbias, int rows, int K,
    int N, int first) {
  typedef Slopes<bf16_t>::Raw Raw;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int last = static_cast<int>(slope.ld) - 8;  // slopes of columns there are
  if (static_cast<int>(blockIdx.x) < first) {
    constexpr int kBatch = 4;
    __shared__ float sums[kFewWaves][16 * kFewCols];
    const int k0 = blockIdx.x * kFewCols, i = lane & 15, g = lane >> 4;
    const bf16_t* wr = w + static_cast<int64_t>(min(k0 + i, K - 1)) * N;
    const int row = min(i, rows - 1);
    const bf16_t* dr = dy + static_cast<int64_t>(row) * N;
    f32x4_t acc = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f}, second = acc;
    for (int s = wave * 32 + 8 * g; s - 8 * g < N; s += kBatch * kFewWaves * 32) {
      u32x4 a[kBatch], b[kBatch];
      Raw e[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int c = s + u * kFewWaves * 32;
        a[u] = load_near(wr, c, N);
        b[u] = load_near(dr, c, N);
        if constexpr (kSlope) e[u] = slope.load8(row, min(c, last));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int c = s + u * kFewWaves * 32;
        trim_piece<bf16_t>(a[u], c, N);
        if constexpr (kSlope) {
          float v[8], rest[8];
          few_da<kSlope>(b[u], e[u], c, N, v);
          const u32x4 high = Piece<bf16_t>::narrow(v);
          Piece<bf16_t>::widen(high, rest);
#pragma unroll
          for (int q = 0; q < 8; ++q) rest[q] = v[q] - rest[q];
          second = few_mfma(a[u], Piece<bf16_t>::narrow(rest), second);
          acc = few_mfma(a[u], high, acc);
        } else {
          trim_piece<bf16_t>(b[u], c, N);
          acc = few_mfma(a[u], b[u], acc);
        }
      }
    }
    // an infinity in w or da is in the first sum; the second one's is inf - inf or inf 0
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = __builtin_isfinite(acc[q]) ? acc[q] + second[q] : acc[q];
    // column k0 + 4 (lane / 16) + q of row lane % 16
    *reinterpret_cast<f32x4_t*>(&sums[wave][lane * 4]) = acc;
    __syncthreads();
    const int t = threadIdx.x / kFewCols, k = threadIdx.x % kFewCols;
    if (t >= rows || k0 + k >= K) return;
    float v = 0.0f;
#pragma unroll
    for (int u = 0; u < kFewWaves; ++u) v += sums[u][(k / 4 * 16 + t) * 4 + k % 4];
    put(dx + static_cast<int64_t>(t) * K + k0 + k, v);
    return;
  }
  constexpr int kBatch = 2;
  const int tiles_n = (N + kFewTile - 1) / kFewTile;
  const int tile = (blockIdx.x - first) * kFewWaves + wave;
  const int k = tile / tiles_n * kFewTile + (lane >> 3) * 8, c = tile % tiles_n * kFewTile + (lane & 7) * 8;
  if (tile / tiles_n * kFewTile >= K) return;
  const bool columns = dbias && tile < tiles_n && lane < 8;
  float acc[8][8], total[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    total[q] = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) acc[r][q] = 0.0f;
  }
  for (int t = 0; t < rows; t += kBatch) {
    u32x4 a[kBatch], b[kBatch];
    Raw e[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t row = min(t + u, rows - 1);
      a[u] = load_near(x + row * K, k, K);
      b[u] = load_near(dy + row * N, c, N);
      if constexpr (kSlope) e[u] = slope.load8(row, min(c, last));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (t + u >= rows) break;
      float xs[8], v[8];
      trim_piece<bf16_t>(a[u], k, K);
      Piece<bf16_t>::widen(a[u], xs);
      few_da<kSlope>(b[u], e[u], c, N, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) total[q] += v[q];
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[r][q] = __builtin_fmaf(xs[r], v[q], acc[r][q]);
    }
  }
  if (c >= N) return;
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (k + r < K) store8<G, false>(dw + static_cast<int64_t>(k + r) * N, c, N, acc[r]);
  if (columns) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < N) dbias[c + q] = total[q];
  }
}

// Up to 16 bf16 rows past the limits of that launch take the products in tiles, with
// da as the same two bf16 numbers: `rows` rows of the first ones and behind them as
// many of the second, zeros from column N on. A tile has 64 rows and a stage of the
// weights' gradient 64 tokens, so the second ones cost no step of either product: dx
// comes as 2 rows' sums, which lin_join_halves_kernel adds, and for dW x goes in
// twice, behind its padding's zeros; the second time without infinities and NaN, whose
// products the first numbers make. dbias is added up on the way, in fp32.
// Training passes, us, and what they were with one rounded da: 16 x 4096 x 4096 37
// (40), 1 x 4096 x 8192 54 (57), 16 x 128 x 16384 22 (26): no launch for dbias's slices.
constexpr int kHalvesCols = 128;
__global__ __launch_bounds__(256) void lin_halves_kernel(const bf16_t* __restrict__ dy, const Slopes<bf16_t> slope,
                                                         bf16_t* __restrict__ da, float* __restrict__ dbias,
                                                         const bf16_t* __restrict__ x, bf16_t* __restrict__ xs,
                                                         int rows, int K, int kp, int N, int np) {
  typedef Piece<bf16_t> P;
  __shared__ float sums[16][kHalvesCols];
  // 16 rows of 16 pieces: of da first, of x behind it
  const int t = threadIdx.x / 16, tx = threadIdx.x % 16, across = np / kHalvesCols;
  if (static_cast<int>(blockIdx.x) >= across) {
    const int c = (blockIdx.x - across) * kHalvesCols + tx * 8;
    if (t >= rows) return;
    const u32x4 v = load_piece(x + static_cast<int64_t>(t) * K, c, K);
    bf16_t* to = xs + static_cast<int64_t>(t) * kp + c;
    *reinterpret_cast<u32x4*>(to) = v;
    float e[8];
    P::widen(v, e);
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = __builtin_isfinite(e[q]) ? e[q] : 0.0f;
    *reinterpret_cast<u32x4*>(to + static_cast<int64_t>(rows) * kp) = P::narrow(e);
    return;
  }
  const int c = blockIdx.x * kHalvesCols + tx * 8, row = min(t, rows - 1);
  float v[8], rest[8];
  few_da<true>(load_near(dy + static_cast<int64_t>(row) * N, c, N),
               slope.load8(row, min(c, static_cast<int>(slope.ld) - 8)), c, N, v);
  const u32x4 high = P::narrow(v);
  P::widen(high, rest);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    sums[t][tx * 8 + q] = v[q];
    rest[q] = __builtin_isfinite(rest[q]) ? v[q] - rest[q] : 0.0f;
  }
  if (t < rows) {
    bf16_t* to = da + static_cast<int64_t>(t) * np + c;
    *reinterpret_cast<u32x4*>(to) = high;
    *reinterpret_cast<u32x4*>(to + static_cast<int64_t>(rows) * np) = P::narrow(rest);
  }
  if (!dbias) return;
  __syncthreads();
  const int n = blockIdx.x * kHalvesCols + threadIdx.x;
  if (threadIdx.x >= kHalvesCols || n >= N) return;
  float total = 0.0f;
  for (int r = 0; r < rows; ++r) total += sums[r][threadIdx.x];
  dbias[n] = total;
}

// dx [rows][K] from the sums [parts][2 rows][K] of the slices and of da's two numbers;
// an infinity of w or da is in the first one's.
__global__ __launch_bounds__(256) void lin_join_halves_kernel(const float* __restrict__ part, int parts, int rows,
                                                              int K, bf16_t* __restrict__ dx) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= K) return;
  const int64_t row = blockIdx.y;
  float first = 0.0f, second = 0.0f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    first += part[(int64_t{2} * p * rows + row) * K + n];
    second += part[((int64_t{2} * p + 1) * rows + row) * K + n];
  }
  put(dx + row * K + n, __builtin_isfinite(first) ? first + second : first);
}

// ---------------------------------------------------- fp32 of moderate size

// The products of one launch, their tiles one after the other; parts > 1: sums of
// slices of k, [parts][M][ld], added by another launch.
struct DirProduct {
  DirOperand s, f;
  int64_t K;
  int64_t M;
  int N;
  int tiles_n, parts;
  int64_t end;  // exclusive end of its workgroups
  float* out;   // or the slices' sums
  int64_t ld;
};
// This workgroup's tile and steps of k.
struct DirPlace {
  int64_t m0, n0, s0, s1;
  int part;
  __device__ DirPlace(const DirProduct& p, int64_t w) {
    part = static_cast<int>(w % p.parts);
    const int64_t tile = w / p.parts, steps = (p.K + kDirStep - 1) / kDirStep;
    m0 = tile / p.tiles_n * kDirTile;
    n0 = tile % p.tiles_n * kDirTile;
    s0 = steps * part / p.parts;
    s1 = steps * (part + 1) / p.parts;
  }
};
__device__ __forceinline__ void dir_store(const DirProduct& p, const DirPlace& t, const float (&v)[8]) {
  const int64_t m = t.m0 + (threadIdx.x >> 3);
  const int n = static_cast<int>(t.n0) + (threadIdx.x & 7) * 8;
  if (m < p.M && n < p.N) store8<float, false>(p.out + (t.part * p.M + m) * p.ld, n, p.N, v);
}

// y: x W, then what follows it.
template <int kAct>
__global__ __launch_bounds__(kDirThreads) void lin_direct_kernel(const DirProduct p, const LinOut<float> o) {
  __shared__ float lds[kDirLds];
  const DirPlace t(p, xcd_remap(blockIdx.x, gridDim.x));
  float v[8];
  dir_tile<kAlong, kAcross, false, false, false>(p.s, p.f, p.K, t.m0, t.n0, t.s0, t.s1, false, lds, nullptr, v);
  if (p.parts > 1) return dir_store(p, t, v);
  const int64_t m = t.m0 + (threadIdx.x >> 3);
  const int n = static_cast<int>(t.n0) + (threadIdx.x & 7) * 8;
  if (m >= p.M || n >= p.N) return;
  float y[8], slope[8], b[8], r[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) b[q] = r[q] = 0.0f;
  if (o.bias) load8<float, false>(o.bias, n, p.N, b);
  if (o.res) load8<float, false>(static_cast<const float*>(o.res) + m * p.N, n, p.N, r);
#pragma unroll
  for (int q = 0; q < 8; ++q) y[q] = lin_act<float, kAct>(v[q] + b[q], &slope[q]) + r[q];
  store8<float, false>(static_cast<float*>(o.y) + m * o.ld, n, p.N, y);
  if (kAct != MOE_ACT_NONE && o.slope.p) o.slope.put8(m, n, slope);
}

// dx = (dy slope) W^T and dW = x^T (dy slope), with the columns' sums for dbias
// (null: not wanted; [parts of dW][pitch of its sums]) from the tiles of dW's first rows.
template <bool kSlope>
__global__ __launch_bounds__(kDirThreads) void lin_direct_bwd_kernel(const DirProduct dx, const DirProduct dw,
                                                                    float* dbias, int64_t ld_bias) {
  __shared__ float lds[kDirLds];
  __shared__ float cols[kDirWaves][64];
  float v[8];
  // the longer tiles first; each product's neighbours on one XCD
  const int first = static_cast<int>(dw.end - dx.end), b = blockIdx.x;
  if (b >= first) {
    const DirPlace t(dx, xcd_remap(b - first, static_cast<int>(dx.end)));
    dir_tile<kAlong, kAlong, kSlope, false, false>(dx.s, dx.f, dx.K, t.m0, t.n0, t.s0, t.s1, false, lds, cols, v);
    return dir_store(dx, t, v);
  }
  const DirPlace t(dw, xcd_remap(b, first));
  const bool columns = dbias && t.m0 == 0;
  dir_tile<kAcross, kAcross, false, kSlope, true>(dw.s, dw.f, dw.K, t.m0, t.n0, t.s0, t.s1, columns, lds, cols, v);
  dir_store(dw, t, v);
  const int64_t n = t.n0 + threadIdx.x;
  if (columns && threadIdx.x < 64 && n < dw.N) {
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kDirWaves; ++u) sum += cols[u][threadIdx.x];
    dbias[t.part * ld_bias + n] = sum;
  }
}

// ------------------------------------------------------------------ layouts

// Whether the forward's tiles read the weights where they are (mm_tile,
// kTurned): as in the gated block, bf16, widths that fill stages and pieces,
// and not so many tokens that turning the weights once is less.
constexpr int64_t kInPlace = int64_t{1} << 23;  // elements of x
bool in_place(const moe_linear& l) {
  return l.dtype == MOE_BF16 && l.inputs % 64 == 0 && l.outputs % 8 == 0 && l.tokens * l.inputs <= kInPlace;
}

// Slices of the rows in which dbias is added up.
int bias_slices(const moe_linear& l) {
  const int64_t across = (l.outputs + kDaCols - 1) / kDaCols;
  int64_t k = (2 * kCUs + across - 1) / across;
  const int64_t most = (l.tokens + kDaRows - 1) / kDaRows;
  if (k > most) k = most;
  return static_cast<int>(k < 1 ? 1 : (k > 64 ? 64 : k));
}

// Products taken from memory as they are (direct.h): fp32, up to so many
// multiplications; a training pass, from memory and in tiles through LDS, us: 100 x
// 100 x 100 (rows, inputs, outputs) 17 and 32, 1000 x 512 x 512 53 and 65, 300 x 1024
// x 1024 62 and 67, 777 x 500 x 1001 53 and 85, 640 x 640 x 960 50 and 76; above it
// 2000 x 512 x 512 79 and 68, 120 x 2048 x 2048 102 and 72, 8192 x 512 x 512 190 and
// 156. Where the tiles' rows are padded the limit is low: 701 x 901 x 803 takes tiles,
// 95, and would take 75 from memory; the rule does not look at padding.
constexpr int64_t kDirect = int64_t{3} << 27;
bool direct(const moe_linear& l) {
  const int64_t n = static_cast<int64_t>(l.inputs) * l.outputs, wide = l.inputs > l.outputs ? l.inputs : l.outputs;
  // operands below 2^32 bytes, rows of four or more
  if (l.dtype != MOE_FP32 || l.inputs < 4 || l.outputs < 4 || n >= int64_t{1} << 29) return false;
  return l.tokens * (wide + 8) < int64_t{1} << 29 && l.tokens * n <= kDirect;
}
// Whether the backward pass is that of few rows.
bool few_bwd(const moe_linear& l) {
  return l.dtype == MOE_BF16 && few_rows(l) && l.inputs <= kFewInputs && l.outputs <= kFewOutputs &&
         l.tokens * l.inputs * l.outputs <= kFewProducts;
}
// Whether da goes into the tiles as two numbers (lin_halves_kernel); without an
// activation it is dy itself.
bool halves(const moe_linear& l) {
  return l.dtype == MOE_BF16 && few_rows(l) && l.act != MOE_ACT_NONE && !few_bwd(l);
}
// Slices of k: a workgroup a CU, of two steps a wave at least.
int64_t dir_tiles(int64_t M, int64_t N) {
  return (M + kDirTile - 1) / kDirTile * ((N + kDirTile - 1) / kDirTile);
}
int64_t dir_steps(int64_t K) { return (K + kDirStep - 1) / kDirStep; }
int dir_parts(int64_t K, int64_t all_steps) {
  const int64_t least = 2 * kDirWaves, each = (all_steps + kCUs - 1) / kCUs;
  const int64_t p = dir_steps(K) / (each > least ? each : least);
  return static_cast<int>(p < 1 ? 1 : (p > 64 ? 64 : p));
}

struct LinLayout {
  size_t wt, xp, sums;                 // forward: turned weights, padded x, sums of slices
  size_t dx_sums, da, wp, part, bias, xt, dat, zero;  // backward
  size_t total;
  int k_parts, dx_parts, grad_parts, bias_parts;
};

// Slices of K of a product in tiles.
int tile_parts(size_t es, int64_t M, int64_t N, int64_t kp) { return parts_of(es, M, N, kp * es / 128); }

LinLayout lin_layout(const moe_linear& l, bool training) {
  LinLayout L{};
  const size_t es = elem_bytes(l), T = l.tokens, K = l.inputs, N = l.outputs;
  const size_t kp = pad128(K), np = pad128(N);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  auto sums = [&](int parts, size_t cells) { return take(parts > 1 ? parts * cells * sizeof(float) : 0); };
  if (few_rows(l)) {
    // slices of a long K so that every CU has a workgroup, of two steps a wave at least
    const int64_t blocks = T == 0 ? 1 : (N + kSkinnyCols - 1) / kSkinnyCols * ((T + 15) / 16);
    const int64_t most = (K + 2 * kSkinnyStep * kSkinnyWaves - 1) / (2 * kSkinnyStep * kSkinnyWaves);
    const int64_t want = (kCUs + blocks - 1) / blocks;
    L.k_parts = K <= static_cast<size_t>(es == 2 ? kShortK : kShortKF32) ? 1 : static_cast<int>(want < most ? want : most);
  } else if (direct(l)) {
    L.k_parts = dir_parts(K, dir_tiles(T, N) * dir_steps(K));
  } else {
    if (!in_place(l)) {
      L.wt = take(N * kp * es);
      L.xp = take(K == kp ? 0 : T * kp * es);
    }
    L.k_parts = tile_parts(es, T, N, in_place(l) ? K : kp);
  }
  L.sums = sums(L.k_parts, T * N);
  L.total = o;
  if (!training) return L;
  // the backward has the place for itself
  o = 0;
  if (few_bwd(l)) return L;
  if (direct(l)) {
    const int64_t all = dir_tiles(T, K) * dir_steps(N) + dir_tiles(K, N) * dir_steps(T);
    L.dx_parts = dir_parts(N, all);
    L.grad_parts = dir_parts(T, all);
    L.dx_sums = sums(L.dx_parts, T * pad4(K));
    L.part = sums(L.grad_parts, K * pad4(N));
    L.bias = sums(L.grad_parts, pad4(N));
    L.total = std::max(L.total, o);
    return L;
  }
  L.zero = take(kTrZeroBytes);
  if (halves(l)) {
    L.da = take(2 * T * np * es);
    L.wp = take(N == np ? 0 : K * np * es);
    L.xp = take(2 * T * kp * es);
    L.dx_parts = tile_parts(es, 2 * T, K, np);
    L.dx_sums = take(L.dx_parts * 2 * T * K * sizeof(float));
    L.grad_parts = 1;
    L.total = std::max(L.total, o);
    return L;
  }
  L.da = take(l.act == MOE_ACT_NONE && N == np ? 0 : T * np * es);
  L.wp = take(N == np ? 0 : K * np * es);
  L.bias_parts = bias_slices(l);
  L.bias = take(L.bias_parts * pad4(N) * sizeof(float));
  L.dx_parts = tile_parts(es, T, K, np);
  if (es == 2) {
    L.xp = take(K == kp ? 0 : T * kp * es);
    L.grad_parts = slices(l.tokens, static_cast<int64_t>(kp / 128) * (np / 128));
  } else {
    const size_t tp = pad128(T);
    L.xt = take(K * tp * es);
    L.dat = take(N * tp * es);
    L.grad_parts = tile_parts(es, K, N, tp);
  }
  // one place for the sums of either product
  L.dx_sums = L.part = o;
  sums(L.dx_parts, T * K);
  L.total = std::max(L.total, o);
  o = L.part;
  sums(L.grad_parts, es == 2 ? kp * np : K * pad4(N));
  L.total = std::max(L.total, o);
  return L;
}

// ----------------------------------------------------------------- launches

template <typename T, typename Cfg, int kAct, bool kPart, bool kTurned>
void lin_tiles_at(const char* name, const MmArgs& a, const LinOut<T>& o, hipStream_t s) {
  MmArgs p = a;
  p.tiles_n = (p.N + Cfg::BN - 1) / Cfg::BN;
  p.nk *= 128 / Cfg::ROW;
  const int64_t grid = (p.M + Cfg::BM - 1) / Cfg::BM * p.tiles_n * (p.parts > 1 ? p.parts : 1);
  MOE_LAUNCH(name, (lin_tile_kernel<T, Cfg, kAct, kPart, kTurned>), dim3(static_cast<unsigned>(grid)),
             dim3(Cfg::NT), 0, s, p, o);
}

template <typename T, int kAct>
void lin_tiles(const char* name, const MmArgs& p, const LinOut<T>& o, hipStream_t s, bool turned) {
  const TileSize size = tile_of(sizeof(T), p.M, p.N, p.nk);
  if constexpr (sizeof(T) == 2) {
    if (turned) {
      if (size == kSmall) return lin_tiles_at<T, MmSmall, kAct, false, true>(name, p, o, s);
      return lin_tiles_at<T, MmMid, kAct, false, true>(name, p, o, s);
    }
    if (size == kBig) return lin_tiles_at<T, MmBig, kAct, false, false>(name, p, o, s);
    if (size == kTall) return lin_tiles_at<T, MmTall, kAct, false, false>(name, p, o, s);
  }
  if (size == kSmall) return lin_tiles_at<T, MmSmall, kAct, false, false>(name, p, o, s);
  lin_tiles_at<T, MmMid, kAct, false, false>(name, p, o, s);
}

// f(the activation as a constant).
template <typename F>
void with_act(int act, F&& f) {
  switch (act) {
    case MOE_ACT_SILU: return f(std::integral_constant<int, MOE_ACT_SILU>{});
    case MOE_ACT_GELU: return f(std::integral_constant<int, MOE_ACT_GELU>{});
    case MOE_ACT_GELU_TANH: return f(std::integral_constant<int, MOE_ACT_GELU_TANH>{});
    case MOE_ACT_RELU: return f(std::integral_constant<int, MOE_ACT_RELU>{});
    default: return f(std::integral_constant<int, MOE_ACT_NONE>{});
  }
}

template <typename T>
void lin_join(const char* name, int act, const float* part, int parts, const LinOut<T>& o, hipStream_t s) {
  with_act(act, [&](auto a) {
    MOE_LAUNCH(name, (lin_join_kernel<T, decltype(a)::value>),
               dim3((o.N + 255) / 256, static_cast<unsigned>(o.M)), dim3(256), 0, s, part, parts, o);
  });
}

// The slopes in `saved`; none without an activation.
template <typename T>
Slopes<T> slopes_at(const moe_linear& l, void* saved) {
  Slopes<T> s{};
  if (l.act == MOE_ACT_NONE || !saved) return s;
  s.p = static_cast<decltype(s.p)>(saved);
  s.ld = slope_pitch(l);
  if constexpr (sizeof(T) == 2) s.low = reinterpret_cast<uint8_t*>(s.p + l.tokens * s.ld);
  return s;
}

// A product in tiles with its epilogue, over slices of K (sums in `part`)
// where it has few tiles.
template <typename T>
void lin_product(const char* name, int act, const MmArgs& a, const LinOut<T>& o, int parts, float* part,
                 hipStream_t s, bool turned = false) {
  MmArgs p = a;
  p.parts = parts;
  if (parts == 1)
    return with_act(act, [&](auto k) { lin_tiles<T, decltype(k)::value>(name, p, o, s, turned); });
  LinOut<T> sums{};
  sums.y = part;
  sums.ld = p.N;
  sums.M = p.M;
  sums.N = p.N;
  sums.zero = o.zero;
  if constexpr (sizeof(T) == 2) {
    if (turned) lin_tiles_at<T, MmSmall, MOE_ACT_NONE, true, true>(name, p, sums, s);
  }
  if (!turned) lin_tiles_at<T, MmSmall, MOE_ACT_NONE, true, false>(name, p, sums, s);
  lin_join<T>("linear_join", act, part, parts, o, s);
}

// A product's tiles behind `start` workgroups; out, or from two slices of k on
// their sums with rows of `ld` (out: of N).
inline void dir_place(DirProduct* p, int64_t start, int64_t K, int64_t M, int N, int parts, float* out, float* sums,
                      int64_t ld) {
  p->K = K;
  p->M = M;
  p->N = N;
  p->tiles_n = (N + kDirTile - 1) / kDirTile;
  p->parts = parts;
  p->end = start + dir_tiles(M, N) * parts;
  p->out = parts > 1 ? sums : out;
  p->ld = parts > 1 ? ld : N;
}

template <typename T>
hipError_t lin_fwd_t(const moe_linear& l, const void* x, const void* w, const float* bias, const void* res,
                     void* saved, void* y, void* ws, hipStream_t s) {
  const LinLayout L = lin_layout(l, false);
  char* W = static_cast<char*>(ws);
  const int K = l.inputs, N = l.outputs;
  const int64_t kp = pad128(K);
  float* part = reinterpret_cast<float*>(W + L.sums);
  const LinOut<T> o{y, N, bias, res, slopes_at<T>(l, saved), l.tokens, N, nullptr};
  if (few_rows(l)) {
    SkinnyArgs<T, 1> a{static_cast<const T*>(x), nullptr, K, {static_cast<const T*>(w)}, l.tokens, K, N, L.k_parts};
    const dim3 grid((N + kSkinnyCols - 1) / kSkinnyCols, static_cast<unsigned>((l.tokens + 15) / 16), L.k_parts);
    if (L.k_parts > 1) {
      MOE_LAUNCH("linear_rows", (lin_rows_kernel<T, MOE_ACT_NONE, 8>), grid, dim3(512), 0, s, a, o, part);
      lin_join<T>("linear_join", l.act, part, L.k_parts, o, s);
    } else {
      with_act(l.act, [&](auto k) {
        MOE_LAUNCH("linear_rows", (lin_rows_kernel<T, decltype(k)::value, kRowsWaves>), grid, dim3(64 * kRowsWaves), 0, s, a, o,
                   nullptr);
      });
    }
    return hipGetLastError();
  }
  if constexpr (sizeof(T) == 4) {
    if (direct(l)) {
      DirProduct p{};
      p.s = DirOperand{static_cast<const float*>(x), K, nullptr, 0, l.tokens};
      p.f = DirOperand{static_cast<const float*>(w), N, nullptr, 0, N};
      dir_place(&p, 0, K, l.tokens, N, L.k_parts, nullptr, part, N);
      with_act(l.act, [&](auto k) {
        MOE_LAUNCH("linear_direct", (lin_direct_kernel<decltype(k)::value>), dim3(static_cast<unsigned>(p.end)),
                   dim3(kDirThreads), 0, s, p, o);
      });
      if (L.k_parts > 1) lin_join<T>("linear_join", l.act, part, L.k_parts, o, s);
      return hipGetLastError();
    }
  }
  if (in_place(l)) {
    lin_product<T>("linear", l.act, rows_of<T>(x, K, w, N, l.tokens, N, K), o, L.k_parts, part, s, true);
    return hipGetLastError();
  }
  TurnJobs jobs{};
  jobs.add(w, W + L.wt, K, N, N);
  turn<T>("linear_turn", jobs, s);
  PadJobs pads{};
  const void* xp = padded<T>(pads, x, W + L.xp, l.tokens, K);
  pad<T>("linear_pad", pads, s);
  lin_product<T>("linear", l.act, rows_of<T>(xp, kp, W + L.wt, kp, l.tokens, N, kp), o, L.k_parts, part, s);
  return hipGetLastError();
}

template <typename T, typename G>
hipError_t lin_bwd_t(const moe_linear& l, const void* x, const void* w, const void* saved, const void* dy,
                     void* dx, void* dw, float* dbias, void* ws, hipStream_t s) {
  const LinLayout L = lin_layout(l, true);
  char* W = static_cast<char*>(ws);
  const int K = l.inputs, N = l.outputs;
  const int64_t kp = pad128(K), np = pad128(N), tok = l.tokens;
  SliceJobs jobs{};
  int64_t end = 0;
  auto job = [&](const float* part, int splits, int64_t stride, int64_t ld, int M, int cols, void* out, bool wide) {
    end += static_cast<int64_t>(M) * ((cols + 3) / 4);
    jobs.job[jobs.n++] = SliceJob{part, splits, stride, ld, M, cols, out, end, wide};
  };

  if constexpr (sizeof(T) == 4) {
    if (direct(l)) {
      const Slopes<float> sl = slopes_at<float>(l, const_cast<void*>(saved));
      const float* g = static_cast<const float*>(dy);
      DirProduct p{}, q{};
      p.s = DirOperand{g, N, sl.p, sl.ld, tok};
      p.f = DirOperand{static_cast<const float*>(w), N, nullptr, 0, K};
      float* dx_sums = reinterpret_cast<float*>(W + L.dx_sums);
      float* dw_sums = reinterpret_cast<float*>(W + L.part);
      float* bias_sums = reinterpret_cast<float*>(W + L.bias);
      dir_place(&p, 0, N, tok, K, L.dx_parts, static_cast<float*>(dx), dx_sums, pad4(K));
      q.s = DirOperand{static_cast<const float*>(x), K, nullptr, 0, K};
      q.f = DirOperand{g, N, sl.p, sl.ld, N};
      dir_place(&q, p.end, tok, K, N, L.grad_parts, static_cast<float*>(dw), dw_sums, pad4(N));
      float* db = dbias && L.grad_parts > 1 ? bias_sums : dbias;
      auto go = [&](auto slope) {
        MOE_LAUNCH("linear_direct_bwd", (lin_direct_bwd_kernel<decltype(slope)::value>),
                   dim3(static_cast<unsigned>(q.end)), dim3(kDirThreads), 0, s, p, q, db, pad4(N));
      };
      if (sl.p) go(std::true_type{});
      else go(std::false_type{});
      if (L.dx_parts > 1) job(dx_sums, L.dx_parts, tok * pad4(K), pad4(K), static_cast<int>(tok), K, dx, true);
      if (L.grad_parts > 1) {
        job(dw_sums, L.grad_parts, K * pad4(N), pad4(N), K, N, dw, true);
        if (dbias) job(bias_sums, L.grad_parts, pad4(N), pad4(N), 1, N, dbias, true);
      }
      if (jobs.n)
        MOE_LAUNCH("linear_slice_sum", slice_sum_kernel<G>, dim3(blocks_for(end)), dim3(256), 0, s, jobs);
      return hipGetLastError();
    }
  }
  if constexpr (sizeof(T) == 2) {
    if (few_bwd(l)) {
      const int first = (K + kFewCols - 1) / kFewCols;
      const int64_t tiles = static_cast<int64_t>((K + kFewTile - 1) / kFewTile) * ((N + kFewTile - 1) / kFewTile);
      const dim3 grid(static_cast<unsigned>(first + (tiles + kFewWaves - 1) / kFewWaves));
      auto go = [&](auto slope) {
        MOE_LAUNCH("linear_few_bwd", (lin_few_bwd_kernel<G, decltype(slope)::value>), grid, dim3(64 * kFewWaves), 0, s,
                   static_cast<const bf16_t*>(x), static_cast<const bf16_t*>(w), static_cast<const bf16_t*>(dy),
                   slopes_at<bf16_t>(l, const_cast<void*>(saved)), static_cast<bf16_t*>(dx), static_cast<G*>(dw), dbias,
                   static_cast<int>(tok), K, N, first);
      };
      if (l.act == MOE_ACT_NONE) go(std::false_type{});
      else go(std::true_type{});
      return hipGetLastError();
    }
    if (halves(l)) {
      const int rows = static_cast<int>(tok);
      bf16_t* da = reinterpret_cast<bf16_t*>(W + L.da);
      bf16_t* xs = reinterpret_cast<bf16_t*>(W + L.xp);
      u32x4* zero = reinterpret_cast<u32x4*>(W + L.zero);
      float* part = reinterpret_cast<float*>(W + L.dx_sums);
      // padded widths are multiples of kHalvesCols
      MOE_LAUNCH("linear_bwd_da", lin_halves_kernel, dim3(static_cast<unsigned>((np + kp) / kHalvesCols)), dim3(256), 0, s,
                 static_cast<const bf16_t*>(dy), slopes_at<bf16_t>(l, const_cast<void*>(saved)), da, dbias,
                 static_cast<const bf16_t*>(x), xs, rows, K, static_cast<int>(kp), N, static_cast<int>(np));
      PadJobs pads{};
      const void* wp = padded<T>(pads, w, W + L.wp, K, N);
      pad<T>("linear_pad", pads, s);
      LinOut<T> sums{};
      sums.y = part;
      sums.ld = K;
      sums.M = 2 * tok;
      sums.N = K;
      sums.zero = zero;
      MmArgs p = rows_of<T>(da, np, wp, np, 2 * tok, K, np);
      p.parts = L.dx_parts;
      lin_tiles_at<T, MmSmall, MOE_ACT_NONE, true, false>("linear_bwd_dx", p, sums, s);
      MOE_LAUNCH("linear_join", lin_join_halves_kernel, dim3((K + 255) / 256, rows), dim3(256), 0, s, part, L.dx_parts,
                 rows, K, static_cast<bf16_t*>(dx));
      grad_direct<G>("linear_bwd_dw", xs, kp, da, np, kp, np, 2 * tok, K, N, np, dw, dw, zero, s);
      return hipGetLastError();
    }
  }
  const bool made = l.act != MOE_ACT_NONE || N != np;
  const void* da = made ? W + L.da : dy;
  if (made || dbias) {
    float* part = dbias ? reinterpret_cast<float*>(W + L.bias) : nullptr;
    const dim3 grid(static_cast<unsigned>((np + kDaCols - 1) / kDaCols), L.bias_parts);
    T* out = made ? reinterpret_cast<T*>(W + L.da) : nullptr;
    auto go = [&](auto slope) {
      MOE_LAUNCH("linear_bwd_da", (lin_da_kernel<T, decltype(slope)::value>), grid, dim3(32 * kDaRows), 0, s,
                 static_cast<const T*>(dy), slopes_at<T>(l, const_cast<void*>(saved)), out, part, tok, N,
                 static_cast<int>(np), static_cast<int>(pad4(N)));
    };
    if (l.act == MOE_ACT_NONE) go(std::false_type{});
    else go(std::true_type{});
    if (dbias) job(part, L.bias_parts, pad4(N), pad4(N), 1, N, dbias, true);
  }
  PadJobs pads{};
  const void* wp = padded<T>(pads, w, W + L.wp, K, N);
  [[maybe_unused]] const void* xp = x;
  if constexpr (std::is_same<T, bf16_t>::value) xp = padded<T>(pads, x, W + L.xp, tok, K);
  pad<T>("linear_pad", pads, s);
  // the weight gradient reads a row of zeros past the last token
  u32x4* zero = reinterpret_cast<u32x4*>(W + L.zero);
  const LinOut<T> o{dx, K, nullptr, nullptr, Slopes<T>{}, tok, K, zero};
  lin_product<T>("linear_bwd_dx", MOE_ACT_NONE, rows_of<T>(da, np, wp, np, tok, K, np), o, L.dx_parts,
                 reinterpret_cast<float*>(W + L.dx_sums), s);

  float* part = reinterpret_cast<float*>(W + L.part);
  if constexpr (std::is_same<T, bf16_t>::value) {
    if (L.grad_parts == 1) {
      grad_direct<G>("linear_bwd_dw", xp, kp, da, np, kp, np, tok, K, N, np, dw, dw, zero, s);
    } else {
      grad_slices<T>("linear_bwd_dw", xp, kp, da, np, kp, np, tok, L.grad_parts, part, zero, s);
      job(part, L.grad_parts, kp * np, np, K, N, dw, false);
    }
  } else {
    // rows of consecutive tokens, as the gated block's weight gradients take them
    TurnJobs turns{};
    turns.add(x, W + L.xt, tok, K, K);
    turns.add(da, W + L.dat, tok, static_cast<int>(N), made ? np : N);
    turn<T>("linear_bwd_turn", turns, s);
    const int64_t tp = pad128(tok);
    MmArgs p = rows_of<T>(W + L.xt, tp, W + L.dat, tp, K, N, tp);
    LinOut<T> g{};
    g.M = K;
    g.N = N;
    if (L.grad_parts == 1) {
      g.y = dw;
      g.ld = N;
      lin_tiles<T, MOE_ACT_NONE>("linear_bwd_dw", p, g, s, false);
    } else {
      g.y = part;
      g.ld = pad4(N);
      p.parts = L.grad_parts;
      lin_tiles_at<T, MmSmall, MOE_ACT_NONE, true, false>("linear_bwd_dw", p, g, s);
      job(part, L.grad_parts, static_cast<int64_t>(K) * pad4(N), pad4(N), K, N, dw, false);
    }
  }
  if (jobs.n)
    MOE_LAUNCH("linear_slice_sum", slice_sum_kernel<G>, dim3(blocks_for(end)), dim3(256), 0, s, jobs);
  return hipGetLastError();
}

}  // namespace

size_t linear_ws_bytes(const moe_linear& l, bool training) {
  // a training workspace serves inference too
  size_t n = lin_layout(l, false).total;
  if (training) n = std::max(n, lin_layout(l, true).total);
  return align_up(n < 256 ? 256 : n, 256);
}
size_t linear_saved_bytes(const moe_linear& l) {
  if (l.act == MOE_ACT_NONE) return 0;
  return align_up(l.tokens * slope_pitch(l) * (l.dtype == MOE_BF16 ? 5 : 8) / 2, 256);
}

hipError_t launch_linear(const moe_linear& l, const void* x, const void* w, const float* bias, const void* res,
                         void* saved, void* y, void* ws, hipStream_t s) {
  return l.dtype == MOE_BF16 ? lin_fwd_t<bf16_t>(l, x, w, bias, res, saved, y, ws, s)
                             : lin_fwd_t<float>(l, x, w, bias, res, saved, y, ws, s);
}

hipError_t launch_linear_bwd(const moe_linear& l, const void* x, const void* w, const void* saved,
                             const void* dy, void* dx, void* dw, float* dbias, void* ws, hipStream_t s) {
  if (l.tokens == 0) {
    const int64_t n = static_cast<int64_t>(l.inputs) * l.outputs;
    if (l.grad_dtype == MOE_BF16)
      MOE_LAUNCH("linear_zero", zero_kernel<bf16_t>, dim3(blocks_for(n)), dim3(256), 0, s,
                 static_cast<bf16_t*>(dw), n);
    else
      MOE_LAUNCH("linear_zero", zero_kernel<float>, dim3(blocks_for(n)), dim3(256), 0, s, static_cast<float*>(dw), n);
    if (dbias)
      MOE_LAUNCH("linear_zero", zero_kernel<float>, dim3(blocks_for(l.outputs)), dim3(256), 0, s, dbias,
                 int64_t{l.outputs});
    return hipGetLastError();
  }
  if (l.dtype != MOE_BF16) return lin_bwd_t<float, float>(l, x, w, saved, dy, dx, dw, dbias, ws, s);
  return l.grad_dtype == MOE_BF16 ? lin_bwd_t<bf16_t, bf16_t>(l, x, w, saved, dy, dx, dw, dbias, ws, s)
                                  : lin_bwd_t<bf16_t, float>(l, x, w, saved, dy, dx, dw, dbias, ws, s);
}

}  // namespace moe
