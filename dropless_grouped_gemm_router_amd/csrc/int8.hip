// Products with weights in 8-bit integers: y = (q_x q_w^T) s_x s_w.
//
// The token's scale is its largest magnitude times 1 / 127 in fp32, its
// integers x / s in an exact fp32 division, rounded to nearest even. The
// product, not the division by 127 (5% of the rows differ in the scale's last
// bit): it is what torch computes on this device for a tensor over a number,
// so weights and inputs quantised by that expression are the same integers
// as in every path below. Sums of products are exact int32 (65536 products
// of 127 * 128 stay under 2^31).
#include "mm.h"

namespace moe {

namespace {

// ------------------------------------------------------------- quantising

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = max(v, dpp_u<0xb1>(v));
  v = max(v, dpp_u<0x4e>(v));
  v = max(v, dpp_u<0x141>(v));
  v = max(v, dpp_u<0x140>(v));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// Magnitudes are compared as bit patterns: infinities and NaN are then
// larger than every number, and a row that holds one is seen.
__device__ __forceinline__ float scale_of(uint32_t most) {
  return most >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(most) * (1.0f / 127.0f);
}
// rint(v / scale), by the scale's reciprocal where that cannot differ: v inv
// is within 127 * 2^-23 of the quotient and the rounded quotient within
// 127 * 2^-24, so unless v inv is that near to a half both round alike (five
// instructions instead of the dozen of a division; 16384 x 4096 bf16 rows 54
// -> 41 us, which is the time of their bytes). NaN takes the division too.
// A row whose scale is not positive (zero or NaN) has q 0.
struct Quantizer {
  float scale, inv;
  __device__ explicit Quantizer(float s) : scale(s), inv(1.0f / s) {}
  // The integer as a float, by the reciprocal; *near: it may differ.
  __device__ float fast(float v, bool* near) const {
    const float t = v * inv, r = rintf(t);
    *near |= !(fabsf(t - r) < 0.4999f);
    return r;
  }
  __device__ int whole(float r) const {
    r = fminf(fmaxf(r, -127.0f), 127.0f);
    return scale > 0.0f ? static_cast<int>(r) : 0;
  }
  __device__ int operator()(float v) const {
    bool near = false;
    float r = fast(v, &near);
    if (near) r = rintf(v / scale);
    return whole(r);
  }
};

template <int V>
__device__ __forceinline__ void store_q(int8_t* p, const float (&f)[V], const Quantizer& quantize) {
  float r[V];
  bool near = false;
#pragma unroll
  for (int q = 0; q < V; ++q) r[q] = quantize.fast(f[q], &near);
  if (near) {  // one branch a piece
#pragma unroll
    for (int q = 0; q < V; ++q) r[q] = rintf(f[q] / quantize.scale);
  }
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[i] |= (static_cast<uint32_t>(quantize.whole(r[4 * i + q])) & 0xffu) << (8 * q);
  }
  if (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[V / 4 - 1]);
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// One row per kTPR threads (rows past the grid in turns). kNV pieces a thread stay in registers between
// the two passes; with kNV 0 the row is read twice (the second time from
// cache).
template <typename T, int kTPR, int kNV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(int64_t rows, int width, int64_t pitch,
                                                            const T* __restrict__ x, int64_t ld,
                                                            int8_t* __restrict__ q,
                                                            float* __restrict__ scale) {
  constexpr int V = Piece<T>::V, kRows = 256 / kTPR;
  __shared__ uint32_t part[2][4];
  const int t = threadIdx.x % kTPR;
  int odd = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTPR; row < rows;
       row += static_cast<int64_t>(gridDim.x) * kRows, odd ^= 1) {
    const T* xr = x + row * ld;
    float f[kNV ? kNV : 1][V];
    uint32_t most = 0;
    if (kNV) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) Piece<T>::widen(load_piece(xr, (i * kTPR + t) * V, width), f[i]);
#pragma unroll
      for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) most = max(most, __float_as_uint(f[i][e]) & 0x7fffffffu);
    } else {
      for (int c = t * V; c < width; c += kTPR * V) {
        Piece<T>::widen(load_piece(xr, c, width), f[0]);
#pragma unroll
        for (int e = 0; e < V; ++e) most = max(most, __float_as_uint(f[0][e]) & 0x7fffffffu);
      }
    }
    most = wave_umax(most);
    if (kTPR > 64) {
      // two sets of maxima: one barrier a row
      if ((threadIdx.x & 63) == 0) part[odd][threadIdx.x >> 6] = most;
      __syncthreads();
      most = max(max(part[odd][0], part[odd][1]), max(part[odd][2], part[odd][3]));
    }
    const float s = scale_of(most);
    if (t == 0) scale[row] = s;
    const Quantizer quantize(s);
    int8_t* qr = q + row * pitch;
    if (kNV) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kTPR + t) * V;
        if (c < pitch) store_q<V>(qr + c, f[i], quantize);
      }
    } else {
      for (int c = t * V; c < pitch; c += kTPR * V) {
        Piece<T>::widen(load_piece(xr, c, width), f[0]);
        store_q<V>(qr + c, f[0], quantize);
      }
    }
  }
}

// Weights [groups][width][outputs] to rows of one output channel each: a
// workgroup takes 64 channels, reads the group's columns twice (largest
// magnitudes, then values) and turns 64 x 64 blocks through LDS.
template <typename T>
__global__ __launch_bounds__(256) void quantize_weight_kernel(int width, int outputs, int64_t pitch,
                                                              const T* __restrict__ w, int64_t q_rows,
                                                              int8_t* __restrict__ q,
                                                              float* __restrict__ scale) {
  __shared__ uint32_t most[4][64];
  __shared__ float sc[64];
  __shared__ int8_t turn[64][68];
  const int c = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int n = blockIdx.x * 64 + c;
  const T* wg = w + static_cast<int64_t>(blockIdx.y) * width * outputs;
  uint32_t m = 0;
  if (n < outputs)
    for (int k = part; k < width; k += 4)
      m = max(m, __float_as_uint(elem(wg + static_cast<int64_t>(k) * outputs + n)) & 0x7fffffffu);
  most[part][c] = m;
  __syncthreads();
  if (part == 0) {
    sc[c] = scale_of(max(max(most[0][c], most[1][c]), max(most[2][c], most[3][c])));
    if (n < outputs) scale[blockIdx.y * q_rows + n] = sc[c];
  }
  __syncthreads();
  const Quantizer quantize(sc[c]);
  int8_t* qg = q + blockIdx.y * q_rows * pitch;
  for (int k0 = 0; k0 < pitch; k0 += 64) {
    for (int k = part; k < 64; k += 4) {
      float v = 0.0f;
      if (n < outputs && k0 + k < width) v = elem(wg + static_cast<int64_t>(k0 + k) * outputs + n);
      turn[c][k] = static_cast<int8_t>(quantize(v));
    }
    __syncthreads();
    // 64 rows of 64 bytes: 16 threads a row, four bytes each
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i >> 4, at = (i & 15) * 4;
      if (blockIdx.x * 64 + r < outputs)
        *reinterpret_cast<uint32_t*>(qg + static_cast<int64_t>(blockIdx.x * 64 + r) * pitch + k0 + at) =
            *reinterpret_cast<const uint32_t*>(&turn[r][at]);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- products

struct I8Out {
  const float* xs;    // scale of an input row
  const float* ws;    // scale of a weight row [groups][outputs]
  const float* bias;
  void* y;
  int64_t ld;         // columns of y
  int outputs;        // weight rows a group
};

__device__ __forceinline__ float as_sum(uint32_t v) { return static_cast<float>(static_cast<int>(v)); }

// Scales, bias and storage of a tile's rows (the callbacks of mm_drain);
// kFull: every column of the tile exists.
template <typename T, typename Cfg, bool kPaired, bool kFull>
struct I8Rows {
  static constexpr int kJ = Cfg::WN / MmStrip<Cfg>::CB;
  const MmArgs& p;
  const I8Out& o;
  const MmTile& t;
  int base, n[kJ];
  float ws[kJ][8], wu[kJ][8], xs[Cfg::WM][mm_passes<Cfg, kPaired>()];  // wu: paired up scales, else bias

  __device__ void cols(int j, int c) {
    n[j] = base + c;
    const float* w = o.ws + static_cast<int64_t>(t.group) * o.outputs;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int at = kFull ? n[j] + q : min(n[j] + q, p.N - 1);
      ws[j][q] = w[at];
      wu[j][q] = kPaired ? w[p.N + at] : (o.bias ? o.bias[at] : 0.0f);
    }
  }
  __device__ void start(int i, int k, int m) {
    const int64_t row = t.row0 + m;
    xs[i][k] = o.xs[p.perm ? mm_token(p, p.perm[row]) : row];
  }
  __device__ void pre(int, int, int, int) {}
  __device__ void row(int, int i, int j, int k, int m, const uint32_t (&v)[8]) {
    float y[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = as_sum(v[q]) * xs[i][k] * ws[j][q] + wu[j][q];
    store8<T, kFull>(static_cast<T*>(o.y) + (t.row0 + m) * o.ld, n[j], p.N, y);
  }
  __device__ void row(int, int i, int j, int k, int m, const uint32_t (&g)[8], const uint32_t (&u)[8]) {
    float y[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      y[q] = silu_f(as_sum(g[q]) * xs[i][k] * ws[j][q]) * (as_sum(u[q]) * xs[i][k] * wu[j][q]);
    store8<T, kFull>(static_cast<T*>(o.y) + (t.row0 + m) * o.ld, n[j], p.N, y);
  }
};

template <typename T, typename Cfg, bool kPaired>
__global__ __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(Cfg::WPE)))
void i8_tile_kernel(const MmArgs p, const I8Out o) {
  __shared__ __attribute__((aligned(1024))) char smem[MmStrip<Cfg>::LDS];
  i32x16 acc[Cfg::WM][Cfg::WN];
  MmTile t;
  if (!mm_find<Cfg>(p, &t)) return;
  constexpr int kCols = kPaired ? Cfg::BN / 2 : Cfg::BN;
  auto go = [&](auto full) {
    I8Rows<T, Cfg, kPaired, decltype(full)::value> rows{p, o, t, t.nt * kCols};
    mm_begin<Cfg, kPaired>(t.rows, rows);
    mm_tile<OpI8, Cfg, kPaired>(p, smem, t, acc);
    mm_drain<Cfg, kPaired>(smem, acc, t.rows, rows);
  };
  if ((t.nt + 1) * kCols <= p.N) go(std::true_type{});
  else go(std::false_type{});
}

// ------------------------------------------------------------------ few rows
//
// Serving form, up to 16 rows of a dense product: the weights' bytes are the
// cost, so they go from memory straight into the operand of mfma
// 16x16x64 (a lane's 16 bytes of one weight row) and are read once. A
// workgroup takes 16 output columns (paired: 16 gate and the 16 up rows) and
// its eight waves share K. Rows that are not yet integers are quantised into
// LDS by every workgroup for itself while its first weights are on their way:
// one launch instead of two, and the rows come from L2. 4 rows of 4096 through
// 4096 x 4096 weights (16.8 MB), one call after another: 9.2 us against 13.9 in
// 64 x 64 tiles. From a graph 8.2 us, and 4.9 with rows that are in 8 bits
// already: above the bytes' 3.5 us are the rows' two passes, which few waves
// make, the launch and the sum over the waves.
constexpr int kRowsWaves = 8, kRowsBatch = 4;

struct I8Few {
  const void* x;
  int64_t ldx;            // elements between rows
  const int8_t* w;
  int64_t pitch;          // bytes between weight rows
  int width;              // elements of an input row
  int rows;               // 1 to 16
  int N;                  // columns of y
};

template <typename T, typename X, bool kPaired>
__global__ __launch_bounds__(64 * kRowsWaves) void i8_few_kernel(const I8Few p, const I8Out o) {
  constexpr int kW = kPaired ? 2 : 1;
  constexpr bool kInt = sizeof(X) == 1;
  extern __shared__ __attribute__((aligned(16))) char rows_q[];  // [rows][pitch + 16], unless kInt
  __shared__ float scale[16];
  __shared__ int sums[kRowsWaves][kW][16 * 16];
  // The wave's number as a scalar: MFMAs run whatever lanes are on, so a step
  // past the end has to be branched over, which is only certain for a scalar
  // condition.
  const int lane = threadIdx.x & 63, wave = mm_wave();
  const int n0 = blockIdx.x * 16;
  const int8_t* w[kW];
#pragma unroll
  for (int m = 0; m < kW; ++m)
    w[m] = p.w + (min(n0 + (lane & 15), p.N - 1) + static_cast<int64_t>(m) * p.N) * p.pitch +
           16 * (lane >> 4);
  const int steps = static_cast<int>(p.pitch / 64);
  const int q_pitch = static_cast<int>(p.pitch) + 16;  // rows of 16 banks apart

  u32x4 wv[2][kRowsBatch][kW], xv[2][kInt ? kRowsBatch : 1];
  // the input row behind this lane's token (the last one again past the end)
  const int mine = min(lane & 15, p.rows - 1);
  const int8_t* xi = kInt ? static_cast<const int8_t*>(p.x) + mine * p.ldx + 16 * (lane >> 4) : nullptr;
  auto load = [&](int set, int s) {
#pragma unroll
    for (int u = 0; u < kRowsBatch; ++u) {
      const int64_t at = static_cast<int64_t>(min(s + u * kRowsWaves, steps - 1)) * 64;
#pragma unroll
      for (int m = 0; m < kW; ++m) wv[set][u][m] = *reinterpret_cast<const u32x4*>(w[m] + at);
      if (kInt) xv[set][u] = *reinterpret_cast<const u32x4*>(xi + at);
    }
  };
  int s = wave;
  load(0, s);
  load(1, s + kRowsBatch * kRowsWaves);
  if constexpr (!kInt) {
    constexpr int V = Piece<X>::V;
    for (int t = wave; t < p.rows; t += kRowsWaves) {
      const X* row = static_cast<const X*>(p.x) + t * p.ldx;
      uint32_t most = 0;
#pragma unroll 4
      for (int c = lane * V; c < p.width; c += 64 * V) {
        float f[V];
        Piece<X>::widen(load_piece(row, c, p.width), f);
#pragma unroll
        for (int e = 0; e < V; ++e) most = max(most, __float_as_uint(f[e]) & 0x7fffffffu);
      }
      const float sc = scale_of(wave_umax(most));
      if (lane == 0) scale[t] = sc;
      const Quantizer quantize(sc);
#pragma unroll 4
      for (int c = lane * V; c < p.pitch; c += 64 * V) {
        float f[V];
        Piece<X>::widen(load_piece(row, c, p.width), f);
        store_q<V>(reinterpret_cast<int8_t*>(rows_q) + t * q_pitch + c, f, quantize);
      }
    }
    __syncthreads();
  }
  i32x4 acc[kW];
#pragma unroll
  for (int m = 0; m < kW; ++m) acc[m] = (i32x4){0, 0, 0, 0};
  const char* xl = rows_q + mine * q_pitch + 16 * (lane >> 4);
  auto multiply = [&](int set, int s) {
#pragma unroll
    for (int u = 0; u < kRowsBatch; ++u) {
      const int st = s + u * kRowsWaves;
      if (st >= steps) break;
      u32x4 x;
      if (kInt) x = xv[set][kInt ? u : 0];
      else x = *reinterpret_cast<const u32x4*>(xl + st * 64);
#pragma unroll
      for (int m = 0; m < kW; ++m)
        acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv[set][u][m]),
                                                       __builtin_bit_cast(i32x4, x), acc[m], 0, 0, 0);
    }
  };
  constexpr int kSpan = kRowsBatch * kRowsWaves;
  for (; s < steps; s += 2 * kSpan) {
    multiply(0, s);
    if (s + 2 * kSpan < steps) load(0, s + 2 * kSpan);
    multiply(1, s + kSpan);
    if (s + 3 * kSpan < steps) load(1, s + 3 * kSpan);
  }
  // lane L holds token L % 16 and columns 4 (L / 16) .. + 3
#pragma unroll
  for (int m = 0; m < kW; ++m)
    *reinterpret_cast<i32x4*>(&sums[wave][m][(lane & 15) * 16 + 4 * (lane >> 4)]) = acc[m];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int t = threadIdx.x >> 4, n = n0 + (threadIdx.x & 15);
    int v[kW];
#pragma unroll
    for (int m = 0; m < kW; ++m) {
      v[m] = 0;
#pragma unroll
      for (int u = 0; u < kRowsWaves; ++u) v[m] += sums[u][m][threadIdx.x];
    }
    if (t < p.rows && n < p.N) {
      const float xs = kInt ? o.xs[t] : scale[t];
      float y = static_cast<float>(v[0]) * xs * o.ws[n];
      if (kPaired) y = silu_f(y) * (static_cast<float>(v[kW - 1]) * xs * o.ws[p.N + n]);
      else y += o.bias ? o.bias[n] : 0.0f;
      put(static_cast<T*>(o.y) + t * o.ld + n, y);
    }
  }
}

template <typename T, typename Cfg>
void i8_tiles(const MmArgs& a, const I8Out& o, bool paired, int64_t row_tiles, hipStream_t s) {
  MmArgs p = a;
  const int per = paired ? Cfg::BN / 2 : Cfg::BN;
  p.tiles_n = (p.N + per - 1) / per;
  p.nk *= 128 / Cfg::ROW;
  p.k_split *= 128 / Cfg::ROW;
  const unsigned grid = static_cast<unsigned>(row_tiles * p.tiles_n);
  if (paired)
    MOE_LAUNCH("linear_i8_gated", (i8_tile_kernel<T, Cfg, true>), dim3(grid), dim3(Cfg::NT), 0, s, p, o);
  else
    MOE_LAUNCH("linear_i8", (i8_tile_kernel<T, Cfg, false>), dim3(grid), dim3(Cfg::NT), 0, s, p, o);
}

template <typename T>
void quantize_rows_t(int64_t rows, int width, const void* x, int64_t ld, int8_t* q, float* scale,
                     hipStream_t s) {
  constexpr int V = Piece<T>::V;
  const int64_t pitch = i8_pitch(width);
  // at most 2^22 workgroups (a launch has to stay under 2^32 threads)
  auto grid = [&](int tpr) {
    const int64_t need = (rows * tpr + 255) / 256, most = int64_t{1} << 22;
    return dim3(static_cast<unsigned>(need < most ? need : most));
  };
#define MOE_Q(TPR, NV)                                                                         \
  MOE_LAUNCH("quantize_rows", (quantize_rows_kernel<T, TPR, NV>), grid(TPR), dim3(256), 0, s, \
             rows, width, pitch, static_cast<const T*>(x), ld, q, scale)
  if (pitch <= 64 * V) MOE_Q(64, 1);
  else if (pitch <= 128 * V) MOE_Q(64, 2);
  else if (pitch <= 256 * V) MOE_Q(256, 1);
  else if (pitch <= 512 * V) MOE_Q(256, 2);
  else if (pitch <= 1024 * V) MOE_Q(256, 4);
  else MOE_Q(256, 0);
#undef MOE_Q
}

struct I8Layout {
  size_t q, scale, total;
  int64_t rows;
};
I8Layout i8_layout(const moe_i8_linear& l) {
  I8Layout L{};
  L.rows = l.groups > 1 && !l.gather ? l.tokens * l.top_k : l.tokens;
  if (l.x_dtype != MOE_I8) {
    L.scale = align_up(static_cast<size_t>(L.rows) * i8_pitch(l.inputs), 256);
    L.total = L.scale + align_up(static_cast<size_t>(L.rows) * sizeof(float), 256);
  }
  return L;
}

}  // namespace

hipError_t launch_quantize_rows(int64_t rows, int width, int dtype, const void* x, int64_t ld_x,
                                int8_t* q, float* scale, hipStream_t s) {
  const int64_t ld = ld_x ? ld_x : width;
  if (dtype == MOE_BF16) quantize_rows_t<bf16_t>(rows, width, x, ld, q, scale, s);
  else quantize_rows_t<float>(rows, width, x, ld, q, scale, s);
  return hipGetLastError();
}

hipError_t launch_quantize_weight(int groups, int width, int outputs, int dtype, const void* w,
                                  int64_t q_rows, int8_t* q, float* scale, hipStream_t s) {
  const dim3 grid((outputs + 63) / 64, groups);
  const int64_t rows = q_rows ? q_rows : outputs;
  if (dtype == MOE_BF16)
    MOE_LAUNCH("quantize_weight", quantize_weight_kernel<bf16_t>, grid, dim3(256), 0, s, width,
               outputs, i8_pitch(width), static_cast<const bf16_t*>(w), rows, q, scale);
  else
    MOE_LAUNCH("quantize_weight", quantize_weight_kernel<float>, grid, dim3(256), 0, s, width,
               outputs, i8_pitch(width), static_cast<const float*>(w), rows, q, scale);
  return hipGetLastError();
}

size_t linear_i8_ws_bytes(const moe_i8_linear& l) {
  const size_t n = i8_layout(l).total;
  return n < 256 ? 256 : n;
}

constexpr int64_t kCUs = 256;
// The serving form's place: up to 16 rows (8 of up to 1024 bytes) and as many
// columns as two workgroups a CU take. In it and in 64 x 64 tiles: 4096 x 4096
// 1 row 8.4 and 13.5 us, 16 rows 9.6 and 14.2; 1024 x 8192 4 rows 8.0 and 7.6,
// 16 rows 12.0 and 8.2; 4096 x 12288 1 row 21.1 and 15.0. Not routed rows,
// whose groups' columns are too many: 128 tokens to 64 groups of 2048 x 2048,
// top-2, 139 and 49 us; 8 tokens 35 and 16, 1 token 11.4 and 10.0.
constexpr int64_t kFewRows = 16, kFewShort = 1024, kFewRowsShort = 8, kFewColumns = 16 * 2 * kCUs;
// The most elements of x that each of its workgroups quantises for itself, and
// of a row, which is one wave's; past them a launch for it is cheaper (8 rows,
// 4096 x 4096: 11.4 us against 9.0; 2 rows, 5000 x 1000: 10.5 against 9.4; but
// 8 rows, 2048 x 4096: 7.4 against 8.0).
constexpr int64_t kOwnElements = 16384, kOwnWidth = 4096;

template <typename T, typename X>
void i8_few(const I8Few& p, const I8Out& o, bool paired, hipStream_t s) {
  const dim3 grid((p.N + 15) / 16);
  const size_t lds = sizeof(X) == 1 ? 0 : p.rows * (p.pitch + 16);
  if (paired)
    MOE_LAUNCH("linear_i8_few", (i8_few_kernel<T, X, true>), grid, dim3(64 * kRowsWaves), lds, s, p, o);
  else
    MOE_LAUNCH("linear_i8_few", (i8_few_kernel<T, X, false>), grid, dim3(64 * kRowsWaves), lds, s, p, o);
}

hipError_t launch_linear_i8(const moe_i8_linear& l, const void* x, const float* xs,
                            const int8_t* wq, const float* ws, const float* bias,
                            const moe_routing* r, void* y, void* work, hipStream_t s) {
  const I8Layout L = i8_layout(l);
  const int64_t pitch = i8_pitch(l.inputs), M = l.tokens * l.top_k;
  const bool paired = l.gated != 0;
  const int N = paired ? l.outputs / 2 : l.outputs;
  const bool few = !r && M <= (pitch <= kFewShort ? kFewRowsShort : kFewRows) && N <= kFewColumns;
  const bool own = few && l.x_dtype != MOE_I8 && pitch <= kOwnWidth && M * pitch <= kOwnElements;
  if (l.x_dtype != MOE_I8 && !own) {
    int8_t* q = static_cast<int8_t*>(work);
    float* sc = reinterpret_cast<float*>(q + L.scale);
    const hipError_t e = launch_quantize_rows(L.rows, l.inputs, l.x_dtype, x, 0, q, sc, s);
    if (e != hipSuccess) return e;
    x = q;
    xs = sc;
  }
  I8Out o{xs, ws, bias, y, N, l.outputs};
  if (few) {
    I8Few p{};
    p.x = x;
    p.ldx = own ? l.inputs : pitch;
    p.w = wq;
    p.pitch = pitch;
    p.width = l.inputs;
    p.rows = static_cast<int>(M);
    p.N = N;
    auto go = [&](auto t) {
      using T = decltype(t);
      if (!own) i8_few<T, int8_t>(p, o, paired, s);
      else if (l.x_dtype == MOE_BF16) i8_few<T, bf16_t>(p, o, paired, s);
      else i8_few<T, float>(p, o, paired, s);
    };
    if (l.dtype == MOE_BF16) go(bf16_t{});
    else go(float{});
    return hipGetLastError();
  }
  MmArgs p{};
  p.a = static_cast<const char*>(x);
  p.a_pitch = pitch;
  p.b = reinterpret_cast<const char*>(wq);
  p.b_pitch = pitch;
  p.b_group = static_cast<int64_t>(l.outputs) * pitch;
  p.nk = static_cast<int>(pitch / 128);
  p.N = N;
  p.half = p.N * pitch;
  p.per_token = 1.0 / l.top_k;
  p.groups = l.groups;
  p.cap = l.capacity;
  if (r) {
    p.offsets = r->expert_offsets;
    if (l.gather) p.perm = r->perm;
  }
  p.M = M;
  auto go = [&](auto t) {
    using T = decltype(t);
    // As for the gated block (tile_of): the largest tiles that give every CU
    // one, 256 x 256 from eight stages on (16384 x 1024 x 2048: 48 us against 51
    // in 256 x 128 and 54 in 128 x 128; with four stages 66, 62 and 61). Routed
    // rows lose less of their last tile in 128 rows (64 experts, 131072 slots
    // of 512: 72 us against 78), few rows in 64 (64 rows, 4096 x 65536: 50 us
    // against 78).
    const int64_t busy = r ? (M < p.groups ? M : p.groups) : 1;  // groups with rows, at most
    auto tiles = [&](int bm) { return (M + busy * (bm - 1)) / bm; };
    const int64_t per_group = M / p.groups;
    auto count = [&](int m, int n) { return (M + m - 1) / m * ((l.outputs + n - 1) / n); };
    if (!r && M <= 64) i8_tiles<T, MmSmall>(p, o, paired, tiles(64), s);
    else if (p.nk >= 8 && per_group >= 512 && count(256, 256) >= kCUs) i8_tiles<T, MmBig>(p, o, paired, tiles(256), s);
    else if (!r && M > 128 && count(256, 128) >= kCUs) i8_tiles<T, MmTall>(p, o, paired, tiles(256), s);
    else if (per_group >= 128 && count(128, 128) >= kCUs) i8_tiles<T, MmMid>(p, o, paired, tiles(128), s);
    else i8_tiles<T, MmSmall>(p, o, paired, tiles(64), s);
  };
  if (l.dtype == MOE_BF16) go(bf16_t{});
  else go(float{});
  return hipGetLastError();
}

}  // namespace moe
