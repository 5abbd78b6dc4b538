// The step between two blocks of a residual stream, forward and backward.
//
//   u = norm(z) w1 + b1 (or z), o = scale res + gate u, y = norm(o) w2 + b2
//
//   do = dout + back(dy w2; oh, ostd),  dres = scale do,  du = gate do
//   dz = back(du w1; zh, zstd) (or du)
//   dw2 = sum dy oh, db2 = sum dy, dgate = sum do u, dw1 = sum du zh, db1 = sum du
// with zh and oh the normalised rows and back(g; h, r) = r (g - mean(g) - h
// mean(g h)); without the means for the rms norm.
//
// Bound by memory: the forward reads z and res and writes o and y, the backward
// reads z, res and two gradients and writes two. A row lives in registers, eight
// bf16 or four fp32 columns a thread and piece, so nothing is read twice: the
// forward takes its four statistics from there, and the backward makes o again
// from z and res, unrounded, instead of reading the rounded o. Rows of up to 16
// pieces take 16 lanes, up to 64 (fp32: 128) a wave, wider ones several waves
// that add up through LDS; the next row's loads are issued before the current row
// is reduced.
//
// The five column sums come of four: with A = sum do zh and B = sum do, dw1 =
// gate A, db1 = gate B and dgate = w1 A + b1 B. Each thread keeps those of its
// columns over all of its rows, a workgroup writes one partial row of each, and a
// second kernel adds the partials in a fixed order.
#include "block.h"

namespace moe {

namespace {

// Floats of a partial row.
__host__ __device__ constexpr int step_pitch(int width) { return (width + 3) / 4 * 4; }

// Threads of a workgroup that holds several rows.
constexpr int kFwdThreads = 256, kBwdThreads = 768;

struct StepArgs {
  int64_t rows;
  int width;
  int rms, post;
  float eps, scale, count, inv;  // count: width, inv: 1 / width
  const void *z, *res, *dout, *dy;
  void *o, *y, *dz, *dres;
  int64_t ld_z, ld_res, ld_o, ld_y, ld_dout, ld_dy, ld_dz, ld_dres;
  const float *w1, *b1, *gate, *w2, *b2;
  float* stats;  // [4][rows]: mean and 1 / deviation of z, of o
  float* partial;
  int wanted;    // bit k: column sum k
  int tpr, rpb;  // threads of a row, rows of a workgroup
};

// Sums of a row over its threads: 16 lanes, a wave, or, kRow 0, the waves from
// `first` on, `waves` of them, through LDS. `slot` is this reduction's own array,
// another one in every other row, so that one barrier is enough: whoever writes it
// again has met all waves at a barrier that they reach after reading it.
template <int kRow, int N>
__device__ __forceinline__ void step_sums(float (&v)[N], float (*slot)[16], int first, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = kRow == 16 ? row16_sum(v[i]) : wave_sum(v[i]);
  if (kRow) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i][threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.0f;
    for (int w = 0; w < waves; ++w) t += slot[i][first + w];
    v[i] = t;
  }
}

// V parameters from column c on: `fill` where there is no array, zeros past the
// row, so that what is made of them there is zero.
template <int V>
__device__ __forceinline__ void load_scales(const float* p, float fill, int c, int n, float (&o)[V]) {
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
  for (int q = 0; q < V; ++q) o[q] = c + q < n ? (p ? p[c + q] : fill) : 0.0f;
}

// Whether the backward reads the parameters again for every row (from the
// caches), and no row ahead: a workgroup of 1024 threads has 128 registers a
// thread, beside the sums too few for them. (One piece a thread still puts 44 bytes
// into scratch memory, two of fp32 92; above 8192 columns 524 and 692, at 0.7 to 1.1 TB/s
// where 4096 x 4096 reaches 4.)
template <int kMax>
constexpr bool kAgain = kMax == 1024;

// The thread's place: its column piece within a row and its row of the
// workgroup's; the rows that all workgroups take in one go.
template <int kRow>
struct StepPlace {
  int t, tpr, in, first, waves;
  int64_t row0, step;
  __device__ StepPlace(const StepArgs& a) {
    tpr = kRow ? kRow : a.tpr;
    in = threadIdx.x / tpr;
    t = threadIdx.x - in * tpr;
    waves = tpr / 64;
    first = in * waves;
    row0 = static_cast<int64_t>(blockIdx.x) * a.rpb;
    step = static_cast<int64_t>(gridDim.x) * a.rpb;
  }
};

// Normalises the row in f (zeros past the row going in): f becomes (f - mean)
// rstd, also past the row.
template <int kRow, int NV, int V>
__device__ __forceinline__ void normalise(const StepArgs& a, const StepPlace<kRow>& p, float (&f)[NV][V],
                                          float (*slots)[1][16], float* mean_out, float* rstd_out) {
  float mean = 0.0f;
  if (!a.rms) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) s[0] += f[i][q];
    step_sums<kRow, 1>(s, slots[0], p.first, p.waves);
    mean = s[0] / a.count;  // a division: the mean of a constant row is its value
  }
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < V; ++q) {
      f[i][q] -= mean;
      if ((i * p.tpr + p.t) * V + q < a.width) ss[0] = __builtin_fmaf(f[i][q], f[i][q], ss[0]);
    }
  step_sums<kRow, 1>(ss, slots[1], p.first, p.waves);
  const float rstd = 1.0f / sqrtf(ss[0] / a.count + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < V; ++q) f[i][q] *= rstd;
  *mean_out = mean;
  *rstd_out = rstd;
}

// 131072 x 512 bf16, two norms: 117 us for 537 MB, 4.6 TB/s (a copy 5.1); 5001 x 1155
// fp32, rows of no alignment: 23 us for 92 MB (18). Above 8192 columns registers do not
// suffice (scratch memory: 172 bytes a thread in bf16, 348 in fp32): 1.2 to 2 TB/s.
template <typename T, int kRow, int NV, int kMax>
__global__ __launch_bounds__(kMax) void step_fwd_kernel(const StepArgs a) {
  constexpr int V = Piece<T>::V;
  __shared__ float slots[8][1][16];
  const StepPlace<kRow> p(a);
  int64_t row = p.row0 + p.in;
  int odd = 0;
  if (row >= a.rows) return;  // all threads of a row together; kRow 0: of the workgroup
  const T* z = static_cast<const T*>(a.z);
  const T* res = static_cast<const T*>(a.res);
  auto at = [&](int i) { return (i * p.tpr + p.t) * V; };
  u32x4 cz[NV], cr[NV], nz[NV], nr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    cz[i] = load_near(z + row * a.ld_z, at(i), a.width);
    cr[i] = load_near(res + row * a.ld_res, at(i), a.width);
  }
  float w1[NV][V], b1[NV][V], g[NV][V], w2[NV][V], b2[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_scales<V>(a.w1, 1.0f, at(i), a.width, w1[i]);
    load_scales<V>(a.b1, 0.0f, at(i), a.width, b1[i]);
    load_scales<V>(a.gate, 1.0f, at(i), a.width, g[i]);
    load_scales<V>(a.w2, 1.0f, at(i), a.width, w2[i]);
    load_scales<V>(a.b2, 0.0f, at(i), a.width, b2[i]);
  }
  while (true) {
    const int64_t next = row + p.step;
    if (next < a.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        nz[i] = load_near(z + next * a.ld_z, at(i), a.width);
        nr[i] = load_near(res + next * a.ld_res, at(i), a.width);
      }
    }
    float f[NV][V], r[NV][V], st[4] = {0.0f, 1.0f, 0.0f, 1.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      trim_piece<T>(cz[i], at(i), a.width);
      trim_piece<T>(cr[i], at(i), a.width);
      Piece<T>::widen(cz[i], f[i]);
      Piece<T>::widen(cr[i], r[i]);
    }
    if (a.post) {
      normalise<kRow, NV, V>(a, p, f, slots + odd, &st[0], &st[1]);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) f[i][q] = __builtin_fmaf(f[i][q], w1[i][q], b1[i][q]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int q = 0; q < V; ++q) f[i][q] = __builtin_fmaf(g[i][q], f[i][q], a.scale * r[i][q]);
      store_piece(static_cast<T*>(a.o) + row * a.ld_o, at(i), a.width, f[i]);
    }
    if (a.y) {
      normalise<kRow, NV, V>(a, p, f, slots + odd + 2, &st[2], &st[3]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int q = 0; q < V; ++q) f[i][q] = __builtin_fmaf(f[i][q], w2[i][q], b2[i][q]);
        store_piece(static_cast<T*>(a.y) + row * a.ld_y, at(i), a.width, f[i]);
      }
    }
    if (a.stats && p.t == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) a.stats[k * a.rows + row] = st[k];
    }
    if (next >= a.rows) break;
    row = next;
    odd ^= 4;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cz[i] = nz[i];
      cr[i] = nr[i];
    }
  }
}

// 16384 x 512 bf16: 24 us for 101 MB (20); 5001 x 1155 fp32 34 us for 139 MB (27).
// partial: [gridDim.x][4][pitch], A, B, dw2 and db2, those that are wanted.
template <typename T, int kRow, int NV, int kMax>
__global__ __launch_bounds__(kMax) void step_bwd_kernel(const StepArgs a) {
  constexpr int V = Piece<T>::V;
  __shared__ float slots[4][2][16];
  // column sums of the rows of a workgroup that holds several
  __shared__ float cols[kMax < 1024 ? NV * V * kMax : 1];
  const StepPlace<kRow> p(a);
  auto at = [&](int i) { return (i * p.tpr + p.t) * V; };
  const T* z = static_cast<const T*>(a.z);
  const T* res = static_cast<const T*>(a.res);
  const T* dout = static_cast<const T*>(a.dout);
  const T* dy = static_cast<const T*>(a.dy);
  float w1[NV][V], b1[NV][V], g[NV][V], w2[NV][V], sum[4][NV][V];
  auto params = [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_scales<V>(a.w1, 1.0f, at(i), a.width, w1[i]);
      load_scales<V>(a.b1, 0.0f, at(i), a.width, b1[i]);
      load_scales<V>(a.gate, 1.0f, at(i), a.width, g[i]);
      load_scales<V>(a.w2, 1.0f, at(i), a.width, w2[i]);
    }
  };
  if (!kAgain<kMax>) params();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < V; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k][i][q] = 0.0f;
  struct Row {
    u32x4 z[NV], r[NV], o[NV], y[NV];
    float st[4];
  };
  // a row past the last as zeros, which add nothing
  auto load = [&](Row& v, int64_t row) {
    if (row >= a.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) v.z[i] = v.r[i] = v.o[i] = v.y[i] = (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
      for (int k = 0; k < 4; ++k) v.st[k] = 0.0f;
      return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v.z[i] = load_near(z + row * a.ld_z, at(i), a.width);
      v.r[i] = load_near(res + row * a.ld_res, at(i), a.width);
      v.o[i] = v.y[i] = (u32x4){0u, 0u, 0u, 0u};
      if (dout) v.o[i] = load_near(dout + row * a.ld_dout, at(i), a.width);
      if (dy) v.y[i] = load_near(dy + row * a.ld_dy, at(i), a.width);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v.st[k] = a.stats[k * a.rows + row];
  };
  Row cur, nxt;
  if (!kAgain<kMax>) load(cur, p.row0 + p.in);
  int odd = 0;
  for (int64_t base = p.row0; base < a.rows; base += p.step, odd ^= 2) {
    const int64_t row = base + p.in;
    if (kAgain<kMax>) {
      load(cur, row);
      params();
    } else if (base + p.step < a.rows) {
      load(nxt, row + p.step);
    }
    const float zm = cur.st[0], zr = cur.st[1], om = cur.st[2], ostd = cur.st[3];
    float zh[NV][V], oh[NV][V], d[NV][V], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r[V];
      trim_piece<T>(cur.z[i], at(i), a.width);
      trim_piece<T>(cur.r[i], at(i), a.width);
      trim_piece<T>(cur.o[i], at(i), a.width);
      trim_piece<T>(cur.y[i], at(i), a.width);
      Piece<T>::widen(cur.z[i], zh[i]);
      Piece<T>::widen(cur.r[i], r);
      Piece<T>::widen(cur.y[i], d[i]);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        zh[i][q] = (zh[i][q] - zm) * zr;  // without the norm after the block 0 and 1: z
        const float u = __builtin_fmaf(zh[i][q], w1[i][q], b1[i][q]);
        oh[i][q] = (__builtin_fmaf(g[i][q], u, a.scale * r[q]) - om) * ostd;
        sum[3][i][q] += d[i][q];
        sum[2][i][q] = __builtin_fmaf(d[i][q], oh[i][q], sum[2][i][q]);
        d[i][q] *= w2[i][q];  // zeros past the row
        s[0] += d[i][q];
        s[1] = __builtin_fmaf(d[i][q], oh[i][q], s[1]);
      }
    }
    if (dy) step_sums<kRow, 2>(s, slots[odd], p.first, p.waves);
    float mean = a.rms ? 0.0f : s[0] * a.inv, proj = s[1] * a.inv;
    s[0] = s[1] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dv[V], out[V];
      Piece<T>::widen(cur.o[i], dv);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        if (dy) dv[q] += ostd * (d[i][q] - mean - oh[i][q] * proj);
        if (at(i) + q >= a.width) dv[q] = 0.0f;
        out[q] = a.scale * dv[q];
        sum[1][i][q] += dv[q];
        sum[0][i][q] = __builtin_fmaf(dv[q], zh[i][q], sum[0][i][q]);
        d[i][q] = dv[q] * g[i][q] * w1[i][q];
        s[0] += d[i][q];
        s[1] = __builtin_fmaf(d[i][q], zh[i][q], s[1]);
      }
      if (row < a.rows) store_piece(static_cast<T*>(a.dres) + row * a.ld_dres, at(i), a.width, out);
    }
    if (a.post) {
      step_sums<kRow, 2>(s, slots[odd + 1], p.first, p.waves);
      mean = a.rms ? 0.0f : s[0] * a.inv;
      proj = s[1] * a.inv;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float out[V];
#pragma unroll
      for (int q = 0; q < V; ++q) out[q] = a.post ? zr * (d[i][q] - mean - zh[i][q] * proj) : d[i][q];
      if (row < a.rows) store_piece(static_cast<T*>(a.dz) + row * a.ld_dz, at(i), a.width, out);
    }
    if (!kAgain<kMax>) cur = nxt;
  }
  if (!a.wanted) return;
  const int pitch = step_pitch(a.width);
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 4 * pitch;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(a.wanted >> k & 1)) continue;
    if (a.rpb == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (at(i) + V <= a.width) {
#pragma unroll
          for (int h = 0; h < V; h += 4)
            store_any(out + static_cast<int64_t>(k) * pitch + at(i) + h,
                      (u32x4){__float_as_uint(sum[k][i][h]), __float_as_uint(sum[k][i][h + 1]),
                              __float_as_uint(sum[k][i][h + 2]), __float_as_uint(sum[k][i][h + 3])});
          continue;
        }
#pragma unroll
        for (int q = 0; q < V; ++q)
          if (at(i) + q < a.width) out[static_cast<int64_t>(k) * pitch + at(i) + q] = sum[k][i][q];
      }
      continue;
    }
    if constexpr (kMax < 1024) {
      __syncthreads();
      // element (i, q) of thread t of a row at ((i V + q) tpr + t): threads side by side
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) cols[(p.in * NV * V + i * V + q) * p.tpr + p.t] = sum[k][i][q];
      __syncthreads();
      for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
        const int piece = c / V, from = ((piece / p.tpr) * V + c % V) * p.tpr + piece % p.tpr;
        float v = 0.0f;
        for (int r = 0; r < a.rpb; ++r) v += cols[r * NV * V * p.tpr + from];
        out[static_cast<int64_t>(k) * pitch + c] = v;
      }
    }
  }
}

// The parameters' gradients (each may be null) from `parts` partial rows
// [parts][4][pitch]: a workgroup owns 32 columns, 32 threads to four of them and
// one of the four sums; thread j adds rows j, j + 32, ... (unwanted sums too,
// whatever they hold: conditions would put the loads one after the other) and the
// 32 are then added in order.
struct StepGrads {
  const float *w1, *b1, *gate;
  float *dw1, *db1, *dgate, *dw2, *db2;
  bool post, pre;  // a norm that is not there has gradients of zero, whatever the sums hold
  int wanted() const {
    return ((dw1 && post) || dgate) | ((db1 && post) || (dgate && b1)) << 1 | (dw2 && pre) << 2 | (db2 && pre) << 3;
  }
};
constexpr int kSumCols = 32, kSumGroups = 32;
__global__ __launch_bounds__(1024) void step_sum_kernel(const float* __restrict__ partial, int parts, int width,
                                                        int pitch, const StepGrads g) {
  __shared__ float sums[kSumGroups][4][kSumCols], total[4][kSumCols];
  {
    const int c = threadIdx.x % 8 * 4, k = threadIdx.x / 8 % 4, j = threadIdx.x / 32;
    const int at = min(static_cast<int>(blockIdx.x) * kSumCols + c, pitch - 4);
    f32x4_t v = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
    const float* src = partial + static_cast<int64_t>(k) * pitch + at;
#pragma unroll 8
    for (int p = j; p < parts; p += kSumGroups)
      v += *reinterpret_cast<const f32x4_t*>(src + static_cast<int64_t>(p) * 4 * pitch);
    *reinterpret_cast<f32x4_t*>(&sums[j][k][c]) = v;
  }
  __syncthreads();
  const int c = threadIdx.x % kSumCols, j = threadIdx.x / kSumCols;
  if (j < 4) {
    float t = 0.0f;
#pragma unroll
    for (int u = 0; u < kSumGroups; ++u) t += sums[u][j][c];
    total[j][c] = t;
  }
  __syncthreads();
  const int col = blockIdx.x * kSumCols + c;
  if (j || col >= width) return;
  const float A = total[0][c], B = total[1][c], gate = g.gate ? g.gate[col] : 1.0f;
  if (g.dw1) g.dw1[col] = g.post ? gate * A : 0.0f;
  if (g.db1) g.db1[col] = g.post ? gate * B : 0.0f;
  if (g.dgate) g.dgate[col] = (g.w1 ? g.w1[col] : 1.0f) * A + (g.b1 ? g.b1[col] * B : 0.0f);
  if (g.dw2) g.dw2[col] = g.pre ? total[2][c] : 0.0f;
  if (g.db2) g.db2[col] = g.pre ? total[3][c] : 0.0f;
}

__global__ __launch_bounds__(256) void step_zero_kernel(const StepGrads g, int width) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= width) return;
  for (float* p : {g.dw1, g.db1, g.dgate, g.dw2, g.db2})
    if (p) p[c] = 0.0f;
}

// Threads of a row and pieces a thread, rows of a workgroup. Rows wider than a
// wave's pieces take whole waves. The backward fills a workgroup of up to 768
// threads with rows, so that there are few partial rows of column sums.
struct StepShape {
  int row, tpr, rpb, pieces;  // row: 16, 64, or 0: whole waves
  int threads() const { return tpr * rpb; }
};
StepShape step_shape(const moe_residual_norm& n, bool bwd) {
  const int V = n.dtype == MOE_BF16 ? 8 : 4, p = (n.width + V - 1) / V;  // pieces of a row
  const int most = bwd ? kBwdThreads : kFwdThreads;
  if (p <= 16) return {16, 16, most / 16, 1};
  if (p <= 64) return {64, 64, most / 64, 1};
  if (V == 4 && p <= 128) return {64, 64, most / 64, 2};
  auto waves = [](int pieces) { return (pieces + 63) / 64 * 64; };
  const int one = waves(p), two = waves((p + 1) / 2);
  if (!bwd) return p <= 1024 ? StepShape{0, one, 1, 1} : p <= 2048 ? StepShape{0, two, 1, 2} : StepShape{0, 1024, 1, 4};
  if (one <= most) return {0, one, most / one, 1};
  if (V == 4 && two <= most) return {0, two, most / two, 2};
  return one <= 1024 ? StepShape{0, one, 1, 1} : two <= 1024 ? StepShape{0, two, 1, 2} : StepShape{0, 1024, 1, 4};
}

template <bool kBwd, typename F>
void with_step_shape(int dtype, const StepShape& r, F&& f) {
  // the largest workgroup of a kernel: what its registers are for
  constexpr int kSome = kBwd ? kBwdThreads : kFwdThreads, kWide = kBwd ? kBwdThreads : 512;
#define MOE_STEP_CASE(T, ROW, NV, MAX)                                \
  if (r.row == ROW && r.pieces == NV && r.threads() <= MAX)    \
  return f(T{}, std::integral_constant<int, ROW>{}, std::integral_constant<int, NV>{}, \
           std::integral_constant<int, MAX>{})
  if (dtype == MOE_BF16) {
    MOE_STEP_CASE(bf16_t, 16, 1, kSome);
    MOE_STEP_CASE(bf16_t, 64, 1, kSome);
    MOE_STEP_CASE(bf16_t, 0, 1, kWide);
    MOE_STEP_CASE(bf16_t, 0, 1, 1024);
    MOE_STEP_CASE(bf16_t, 0, 2, 1024);
  } else {
    MOE_STEP_CASE(float, 16, 1, kSome);
    MOE_STEP_CASE(float, 64, 1, kSome);
    MOE_STEP_CASE(float, 64, 2, kSome);
    MOE_STEP_CASE(float, 0, 1, kWide);
    if constexpr (kBwd) {
      MOE_STEP_CASE(float, 0, 2, kWide);
    } else {
      MOE_STEP_CASE(float, 0, 1, 1024);
    }
    MOE_STEP_CASE(float, 0, 2, 1024);
    MOE_STEP_CASE(float, 0, 4, 1024);
  }
#undef MOE_STEP_CASE
}

// Workgroups of the backward: as many as are at once on the chip, one a CU where
// they are full.
int step_bwd_blocks(const moe_residual_norm& n) {
  const StepShape r = step_shape(n, true);
  const int64_t need = (n.rows + r.rpb - 1) / r.rpb;
  return static_cast<int>(need < 1 ? 1 : (need > 256 ? 256 : need));
}

StepArgs step_args(const moe_residual_norm& n) {
  auto ld = [&](int64_t v) { return v ? v : static_cast<int64_t>(n.width); };
  StepArgs a{};
  a.rows = n.rows;
  a.width = n.width;
  a.rms = n.kind == MOE_NORM_RMS;
  a.post = n.post;
  a.eps = n.eps;
  a.scale = n.scale;
  a.count = static_cast<float>(n.width);
  a.inv = static_cast<float>(1.0 / n.width);
  a.ld_z = ld(n.ld_z);
  a.ld_res = ld(n.ld_res);
  a.ld_o = ld(n.ld_out);
  a.ld_y = ld(n.ld_y);
  a.ld_dout = ld(n.ld_grad_out);
  a.ld_dy = ld(n.ld_grad_y);
  a.ld_dz = ld(n.ld_grad_z);
  a.ld_dres = ld(n.ld_grad_res);
  return a;
}

void set_params(StepArgs* a, const moe_norm_params& p, bool post) {
  a->w1 = post ? p.post_weight : nullptr;
  a->b1 = post ? p.post_bias : nullptr;
  a->gate = p.gate;
  a->w2 = p.pre_weight;
  a->b2 = p.pre_bias;
}

}  // namespace

hipError_t launch_residual_norm(const moe_residual_norm& n, const void* z, const void* res,
                                const moe_norm_params& w, void* out, void* y, float* stats, hipStream_t s) {
  StepArgs a = step_args(n);
  set_params(&a, w, n.post != 0);
  a.z = z;
  a.res = res;
  a.o = out;
  a.y = y;
  a.stats = stats;
  const StepShape r = step_shape(n, false);
  a.tpr = r.tpr;
  a.rpb = r.rpb;
  with_step_shape<false>(n.dtype, r, [&](auto t, auto row, auto nv, auto max) {
    const int64_t need = (n.rows + r.rpb - 1) / r.rpb;
    const int64_t most = static_cast<int64_t>(cu_count()) * (1536 / r.threads());
    MOE_LAUNCH("residual_norm", (step_fwd_kernel<decltype(t), decltype(row)::value, decltype(nv)::value, decltype(max)::value>),
               dim3(static_cast<unsigned>(need < most ? need : most)), dim3(r.threads()), 0, s, a);
  });
  return hipGetLastError();
}

size_t residual_norm_ws_bytes(const moe_residual_norm& n) {
  return align_up(static_cast<size_t>(step_bwd_blocks(n)) * 4 * step_pitch(n.width) * sizeof(float), 256);
}

hipError_t launch_residual_norm_bwd(const moe_residual_norm& n, const void* z, const void* res,
                                    const moe_norm_params& w, const float* stats, const void* dout,
                                    const void* dy, void* dz, void* dres, const moe_norm_grads& g, void* ws,
                                    hipStream_t s) {
  StepArgs a = step_args(n);
  set_params(&a, w, n.post != 0);
  const StepGrads grads{a.w1,         a.b1,         a.gate,      g.post_weight, g.post_bias, g.gate,
                        g.pre_weight, g.pre_bias, n.post != 0, n.pre != 0};
  const int wanted = grads.wanted();
  const bool any = g.post_weight || g.post_bias || g.gate || g.pre_weight || g.pre_bias;
  if (n.rows == 0) {
    if (!any) return hipSuccess;
    MOE_LAUNCH("residual_norm_zero", step_zero_kernel, dim3((n.width + 255) / 256), dim3(256), 0, s, grads,
               n.width);
    return hipGetLastError();
  }
  a.z = z;
  a.res = res;
  a.dout = dout;
  a.dy = dy;
  a.dz = dz;
  a.dres = dres;
  a.stats = const_cast<float*>(stats);
  a.partial = static_cast<float*>(ws);
  a.wanted = wanted;
  const StepShape r = step_shape(n, true);
  a.tpr = r.tpr;
  a.rpb = r.rpb;
  const int blocks = step_bwd_blocks(n);
  with_step_shape<true>(n.dtype, r, [&](auto t, auto row, auto nv, auto max) {
    MOE_LAUNCH("residual_norm_bwd", (step_bwd_kernel<decltype(t), decltype(row)::value, decltype(nv)::value, decltype(max)::value>),
               dim3(blocks), dim3(r.threads()), 0, s, a);
  });
  if (any)  // zeros where no sum is wanted
    MOE_LAUNCH("residual_norm_sum", step_sum_kernel, dim3((n.width + kSumCols - 1) / kSumCols),
               dim3(1024), 0, s, a.partial, blocks, n.width, step_pitch(n.width), grads);
  return hipGetLastError();
}

}  // namespace moe
