// Layer norm, forward and backward.
//
//   y = (x - mean) rstd w + b
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w, xh = (x - mean) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// Both passes are bound by memory: the forward reads x and writes y, the
// backward reads x and dy and writes dx. A row lives in the registers of one
// wave (or of one workgroup when it is wider), so the variance is the mean
// square about the mean (no cancellation) without a second read. Waves walk
// rows with the next row's loads issued before the current row is reduced;
// weight and bias stay in registers. 131072 x 512 bf16: 48 to 53 us (5.0 to
// 5.6 TB/s; a copy of 1 GiB reaches 4.8). 16384 x 512 bf16, forward and
// backward: 23 us for 84 MB, of which three launches are about 6.
//
// The backward's weight gradients stay in registers too, each thread owning
// its columns over all rows of its wave; a workgroup then writes one partial
// row of dw and db, and a second kernel adds the partials in a fixed order.
#include "block.h"

namespace moe {

namespace {

struct NormArgs {
  int64_t rows;
  int width;
  float eps, count, inv;  // count: width, inv: 1 / width
  int64_t ld_x, ld_y, ld_dy, ld_dx;
};

// Sums of a row over its threads, kTPR of them: 16 lanes, one wave, or a workgroup
// through LDS (slot: this reduction's own array, so that one barrier is
// enough; the next use of the same slot is a later barrier away).
template <int kTPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*slot)[16]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = kTPR == 16 ? row16_sum(v[i]) : wave_sum(v[i]);
  if (kTPR <= 64) return;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i][wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kTPR / 64; ++w) t += slot[i][w];
    v[i] = t;
  }
}

constexpr int block_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

// V parameters from column c on (`fill` where there is no array).
template <int V>
__device__ __forceinline__ void load_param(const float* p, float fill, int c, int n, float (&o)[V]) {
  if (p && c + V <= n) {
#pragma unroll
    for (int h = 0; h < V; h += 4) {
      const u32x4 v = load_any(p + c + h);
#pragma unroll
      for (int q = 0; q < 4; ++q) o[h + q] = __uint_as_float(v[q]);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < V; ++q) o[q] = (p && c + q < n) ? p[c + q] : fill;
}

// Row piece i of thread t: columns (i * kTPR + t) * V.
template <typename T, int kTPR, int NV>
__global__ __launch_bounds__(block_threads(kTPR)) void norm_fwd_kernel(
    const NormArgs a, const T* x, const float* __restrict__ w, const float* __restrict__ b, T* y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int V = Piece<T>::V, kRows = block_threads(kTPR) / kTPR;
  __shared__ float slots[2][1][16];
  const int t = threadIdx.x % kTPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTPR;
  if (row >= a.rows) return;  // all threads of a row together
  u32x4 cur[NV], nxt[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) cur[i] = load_piece(x + row * a.ld_x, (i * kTPR + t) * V, a.width);
  float wv[NV][V], bv[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<V>(w, 1.0f, (i * kTPR + t) * V, a.width, wv[i]);
    load_param<V>(b, 0.0f, (i * kTPR + t) * V, a.width, bv[i]);
  }
  while (true) {
    const int64_t next = row + step;
    if (next < a.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        nxt[i] = load_piece(x + next * a.ld_x, (i * kTPR + t) * V, a.width);
    }
    float f[NV][V], s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Piece<T>::widen(cur[i], f[i]);
#pragma unroll
      for (int q = 0; q < V; ++q) s[0] += f[i][q];  // zeros past the row
    }
    row_sums<kTPR, 1>(s, slots[0]);
    const float mean = s[0] / a.count;  // a division: the mean of a constant row is its value
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        f[i][q] -= mean;
        if ((i * kTPR + t) * V + q < a.width) ss[0] = __builtin_fmaf(f[i][q], f[i][q], ss[0]);
      }
    row_sums<kTPR, 1>(ss, slots[1]);
    const float rstd = 1.0f / sqrtf(ss[0] / a.count + a.eps);
    if (t == 0 && mean_out) {
      mean_out[row] = mean;
      rstd_out[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V];
#pragma unroll
      for (int q = 0; q < V; ++q) o[q] = __builtin_fmaf(f[i][q] * rstd, wv[i][q], bv[i][q]);
      store_piece(y + row * a.ld_y, (i * kTPR + t) * V, a.width, o);
    }
    if (next >= a.rows) break;
    row = next;
#pragma unroll
    for (int i = 0; i < NV; ++i) cur[i] = nxt[i];
  }
}

// partial: [gridDim.x][2][width], dw then db; null when neither is wanted.
template <typename T, int kTPR, int NV>
__global__ __launch_bounds__(block_threads(kTPR)) void norm_bwd_kernel(
    const NormArgs a, const T* x, const float* __restrict__ w, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const T* dy, T* dx, float* __restrict__ partial) {
  constexpr int V = Piece<T>::V, kRows = block_threads(kTPR) / kTPR;
  __shared__ float slots[2][2][16];
  // the waves' column sums of a workgroup that holds several rows
  __shared__ float cols[kRows > 1 ? kRows * NV * kTPR * V : 1];
  const int t = threadIdx.x % kTPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTPR;
  float wv[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<V>(w, 1.0f, (i * kTPR + t) * V, a.width, wv[i]);
#pragma unroll
    for (int q = 0; q < V; ++q) dw[i][q] = db[i][q] = 0.0f;
  }
  u32x4 cx[NV], cd[NV], nx[NV], nd[NV];
  float cm = 0.0f, cr = 0.0f, nm = 0.0f, nr = 0.0f;
  if (first < a.rows) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cx[i] = load_piece(x + first * a.ld_x, (i * kTPR + t) * V, a.width);
      cd[i] = load_piece(dy + first * a.ld_dy, (i * kTPR + t) * V, a.width);
    }
    cm = mean_in[first];
    cr = rstd_in[first];
  }
  int odd = 0;
  for (int64_t row = first; row < a.rows; row += step, odd ^= 1) {
    const int64_t next = row + step;
    if (next < a.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        nx[i] = load_piece(x + next * a.ld_x, (i * kTPR + t) * V, a.width);
        nd[i] = load_piece(dy + next * a.ld_dy, (i * kTPR + t) * V, a.width);
      }
      nm = mean_in[next];
      nr = rstd_in[next];
    }
    float s[2] = {0.0f, 0.0f};
    float xh[NV][V], g[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Piece<T>::widen(cx[i], xh[i]);
      Piece<T>::widen(cd[i], g[i]);  // zeros past the row: they add nothing below
#pragma unroll
      for (int q = 0; q < V; ++q) {
        xh[i][q] = (xh[i][q] - cm) * cr;
        db[i][q] += g[i][q];
        dw[i][q] = __builtin_fmaf(g[i][q], xh[i][q], dw[i][q]);
        g[i][q] *= wv[i][q];
        if ((i * kTPR + t) * V + q < a.width) {
          s[0] += g[i][q];
          s[1] = __builtin_fmaf(g[i][q], xh[i][q], s[1]);
        }
      }
    }
    row_sums<kTPR, 2>(s, slots[odd]);
    const float mg = s[0] * a.inv, mgx = s[1] * a.inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V];
#pragma unroll
      for (int q = 0; q < V; ++q) o[q] = cr * (g[i][q] - mg - xh[i][q] * mgx);
      store_piece(dx + row * a.ld_dx, (i * kTPR + t) * V, a.width, o);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cx[i] = nx[i];
      cd[i] = nd[i];
    }
    cm = nm;
    cr = nr;
  }
  if (!partial) return;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (kRows == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const int c = (i * kTPR + t) * V + q;
          if (c < a.width) out[static_cast<int64_t>(k) * a.width + c] = k ? db[i][q] : dw[i][q];
        }
      continue;
    }
    if (k) __syncthreads();
    // element (i, q) of lane t at ((i V + q) kTPR + t): lanes side by side
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q)
        cols[(threadIdx.x / kTPR * NV * V + i * V + q) * kTPR + t] = k ? db[i][q] : dw[i][q];
    __syncthreads();
    for (int c = threadIdx.x; c < a.width; c += block_threads(kTPR)) {
      const int piece = c / V, at = ((piece / kTPR) * V + c % V) * kTPR + piece % kTPR;
      float v = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) v += cols[r * NV * V * kTPR + at];
      out[static_cast<int64_t>(k) * a.width + c] = v;
    }
  }
}

// dw and db from `parts` partial rows [parts][2 * width]: a workgroup owns 16
// columns, 64 threads to each, thread j adding rows j, j + 64, ... and the 64
// sums then added in order.
constexpr int kSumCols = 16, kSumGroups = 64;
__global__ __launch_bounds__(kSumCols* kSumGroups) void norm_sum_kernel(
    const float* __restrict__ partial, int parts, int width, float* __restrict__ dw,
    float* __restrict__ db) {
  __shared__ float sums[kSumGroups][kSumCols];
  const int c = threadIdx.x % kSumCols, j = threadIdx.x / kSumCols;
  const int col = blockIdx.x * kSumCols + c;
  float v = 0.0f;
  if (col < 2 * width) {
#pragma unroll 4
    for (int p = j; p < parts; p += kSumGroups) v += partial[static_cast<int64_t>(p) * 2 * width + col];
  }
  sums[j][c] = v;
  __syncthreads();
#pragma unroll
  for (int half = kSumGroups / 2; half > 0; half /= 2) {
    if (j < half) sums[j][c] += sums[j + half][c];
    __syncthreads();
  }
  if (j == 0 && col < 2 * width) {
    if (col < width) {
      if (dw) dw[col] = sums[0][c];
    } else if (db) {
      db[col - width] = sums[0][c];
    }
  }
}

__global__ __launch_bounds__(256) void norm_zero_kernel(float* dw, float* db, int width) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= width) return;
  if (dw) dw[c] = 0.0f;
  if (db) db[c] = 0.0f;
}

// Threads of a row and pieces a thread. As few threads as its registers allow:
// the rows of one wave need no barrier and a CU holds more of them (1155 fp32
// columns, 5001 rows, backward: 64 threads with five pieces 22 us, 256 with
// two 23 us). Past 16 bytes x 64 x 3 (bf16; fp32: 5) a workgroup shares a
// row; rows up to 256 bytes (one piece) or 512 take 16 lanes, so that a wave
// holds four.
struct RowShape {
  int threads, pieces;
};
RowShape row_shape(int width, int V) {
  const int n = (width + V - 1) / V;  // pieces of a row
  if (n <= 32) return {16, n <= 16 ? 1 : 2};
  const int wave = V == 8 ? 3 : 5;
  if (n <= 64 * wave) return {64, (n + 63) / 64};
  if (n <= 512) return {256, n <= 256 ? 1 : 2};
  if (n <= 2048) return {512, n <= 1024 ? 2 : 4};
  return {1024, 4};
}

int per_piece(const moe_norm& n) { return n.dtype == MOE_BF16 ? 8 : 4; }

// Workgroups of the backward: enough to fill the chip, at least four row
// steps each (the partial rows cost 8 bytes a column).
int bwd_blocks(const moe_norm& n) {
  const int tpr = row_shape(n.width, per_piece(n)).threads;
  const int64_t steps = (n.rows * tpr + block_threads(tpr) - 1) / block_threads(tpr);
  const int64_t most = static_cast<int64_t>(256) * 1024 / block_threads(tpr);
  const int64_t b = (steps + 3) / 4;
  return static_cast<int>(b < 1 ? 1 : (b > most ? most : b));
}

template <typename F>
void with_shape(int dtype, int width, F&& f) {
  const RowShape r = row_shape(width, dtype == MOE_BF16 ? 8 : 4);
#define MOE_NORM_CASE(T, TPR, NV)           \
  if (r.threads == TPR && r.pieces == NV)   \
  return f(T{}, std::integral_constant<int, TPR>{}, std::integral_constant<int, NV>{})
  if (dtype == MOE_BF16) {
    MOE_NORM_CASE(bf16_t, 16, 1);
    MOE_NORM_CASE(bf16_t, 16, 2);
    MOE_NORM_CASE(bf16_t, 64, 1);
    MOE_NORM_CASE(bf16_t, 64, 2);
    MOE_NORM_CASE(bf16_t, 64, 3);
    MOE_NORM_CASE(bf16_t, 256, 1);
    MOE_NORM_CASE(bf16_t, 256, 2);
    MOE_NORM_CASE(bf16_t, 512, 2);
    MOE_NORM_CASE(bf16_t, 512, 4);
  } else {
    MOE_NORM_CASE(float, 16, 1);
    MOE_NORM_CASE(float, 16, 2);
    MOE_NORM_CASE(float, 64, 1);
    MOE_NORM_CASE(float, 64, 2);
    MOE_NORM_CASE(float, 64, 3);
    MOE_NORM_CASE(float, 64, 4);
    MOE_NORM_CASE(float, 64, 5);
    MOE_NORM_CASE(float, 256, 2);
    MOE_NORM_CASE(float, 512, 2);
    MOE_NORM_CASE(float, 512, 4);
    MOE_NORM_CASE(float, 1024, 4);
  }
#undef MOE_NORM_CASE
}

NormArgs norm_args(const moe_norm& n) {
  auto ld = [&](int64_t v) { return v ? v : static_cast<int64_t>(n.width); };
  return NormArgs{n.rows, n.width, n.eps, static_cast<float>(n.width), static_cast<float>(1.0 / n.width), ld(n.ld_x), ld(n.ld_y),
                  ld(n.ld_grad_out), ld(n.ld_grad_x)};
}

}  // namespace

hipError_t launch_norm(const moe_norm& n, const void* x, const float* w, const float* b, void* y,
                       float* mean, float* rstd, hipStream_t s) {
  const NormArgs a = norm_args(n);
  with_shape(n.dtype, n.width, [&](auto t, auto tpr, auto nv) {
    using T = decltype(t);
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int kRows = block_threads(TPR) / TPR;
    const int64_t need = (n.rows + kRows - 1) / kRows;
    const int64_t most = static_cast<int64_t>(cu_count()) * (2048 / block_threads(TPR));
    MOE_LAUNCH("layer_norm", (norm_fwd_kernel<T, TPR, NV>),
               dim3(static_cast<unsigned>(need < most ? need : most)), dim3(block_threads(TPR)), 0, s,
               a, static_cast<const T*>(x), w, b, static_cast<T*>(y), mean, rstd);
  });
  return hipGetLastError();
}

size_t norm_ws_bytes(const moe_norm& n) {
  return align_up(static_cast<size_t>(bwd_blocks(n)) * 2 * n.width * sizeof(float), 256);
}

hipError_t launch_norm_bwd(const moe_norm& n, const void* x, const float* w, const float* mean,
                           const float* rstd, const void* dy, void* dx, float* dw, float* db,
                           void* ws, hipStream_t s) {
  if (n.rows == 0) {
    if (!dw && !db) return hipSuccess;
    MOE_LAUNCH("layer_norm_zero", norm_zero_kernel, dim3((n.width + 255) / 256), dim3(256), 0, s, dw,
               db, n.width);
    return hipGetLastError();
  }
  const NormArgs a = norm_args(n);
  const int blocks = bwd_blocks(n);
  float* partial = dw || db ? static_cast<float*>(ws) : nullptr;
  with_shape(n.dtype, n.width, [&](auto t, auto tpr, auto nv) {
    using T = decltype(t);
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    MOE_LAUNCH("layer_norm_bwd", (norm_bwd_kernel<T, TPR, NV>), dim3(blocks),
               dim3(block_threads(TPR)), 0, s, a, static_cast<const T*>(x), w, mean, rstd,
               static_cast<const T*>(dy), static_cast<T*>(dx), partial);
  });
  if (partial)
    MOE_LAUNCH("layer_norm_sum", norm_sum_kernel, dim3((2 * n.width + kSumCols - 1) / kSumCols),
               dim3(kSumCols * kSumGroups), 0, s, partial, blocks, n.width, dw, db);
  return hipGetLastError();
}

}  // namespace moe
