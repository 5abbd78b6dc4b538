// Internal definitions of the operators around the layer (moe_block.h):
// launchers, and device helpers they share.
#pragma once

#include "common.h"
#include "moe_block.h"

namespace moe {

// ------------------------------------------------------------ row pieces

// Eight bf16 or four fp32 elements as one 16-byte access at the alignment
// of a single element: global memory takes any address, so rows of odd
// width and strided views need no path of their own (an access that
// straddles a cache line costs a second request).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

__device__ __forceinline__ u32x4 load_any(const bf16_t* p) { return *reinterpret_cast<const u32x4_a2*>(p); }
__device__ __forceinline__ u32x4 load_any(const float* p) { return *reinterpret_cast<const u32x4_a4*>(p); }
__device__ __forceinline__ void store_any(bf16_t* p, const u32x4& v) { *reinterpret_cast<u32x4_a2*>(p) = v; }
__device__ __forceinline__ void store_any(float* p, const u32x4& v) { *reinterpret_cast<u32x4_a4*>(p) = v; }

__device__ __forceinline__ float elem(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float elem(const float* p) { return *p; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// A 16-byte piece widened to fp32, and back (rounded to nearest even).
template <typename T>
struct Piece;
template <>
struct Piece<bf16_t> {
  static constexpr int V = 8;
  __device__ static void widen(const u32x4& v, float (&o)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      o[2 * q] = bf16lo(v[q]);
      o[2 * q + 1] = bf16hi(v[q]);
    }
  }
  __device__ static u32x4 narrow(const float (&v)[8]) {
    return (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7])};
  }
};
template <>
struct Piece<float> {
  static constexpr int V = 4;
  __device__ static void widen(const u32x4& v, float (&o)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = __uint_as_float(v[q]);
  }
  __device__ static u32x4 narrow(const float (&v)[4]) {
    return (u32x4){__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                   __float_as_uint(v[3])};
  }
};

// Elements c .. c + V - 1 of a row of n: a whole piece, or the row's last
// elements one by one with zeros behind them (nothing past the row is read).
template <typename T>
__device__ __forceinline__ u32x4 load_piece(const T* row, int c, int n) {
  constexpr int V = Piece<T>::V;
  if (c + V <= n) return load_any(row + c);
  u32x4 v = (u32x4){0u, 0u, 0u, 0u};
  float e[V];
#pragma unroll
  for (int q = 0; q < V; ++q) e[q] = c + q < n ? elem(row + c + q) : 0.0f;
  return c < n ? Piece<T>::narrow(e) : v;
}
// load_piece without a branch, for rows of V or more: a piece that is not whole
// takes the row's last V elements, and where it is used trim_piece moves its own
// to the front, zeros behind them. (A wave with one lane at the row's end had every
// other lane wait for its loads of single elements: 10000 x 1023 bf16, backward, 58
// us against 31 at 1024.)
template <typename T>
__device__ __forceinline__ u32x4 load_near(const T* row, int c, int n) {
  if (n < Piece<T>::V) return load_piece(row, c, n);
  return load_any(row + min(c, n - Piece<T>::V));
}
template <typename T>
__device__ __forceinline__ void trim_piece(u32x4& v, int c, int n) {
  const int past = c + Piece<T>::V - n;  // elements of the piece behind the row
  if (past <= 0 || n < Piece<T>::V) return;
  const int w = sizeof(T) == 2 ? past / 2 : past;
  if (sizeof(T) == 2 && past & 1)
    v = (u32x4){v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  if (w & 1) v = (u32x4){v[1], v[2], v[3], 0u};
  if (w & 2) v = (u32x4){v[2], v[3], 0u, 0u};
  if (w >= 4) v = (u32x4){0u, 0u, 0u, 0u};
}

template <typename T>
__device__ __forceinline__ void store_piece(T* row, int c, int n, const float (&v)[Piece<T>::V]) {
  constexpr int V = Piece<T>::V;
  if (c + V <= n) {
    store_any(row + c, Piece<T>::narrow(v));
    return;
  }
#pragma unroll
  for (int q = 0; q < V; ++q)
    if (c + q < n) put(row + c + q, v[q]);
}

// Eight consecutive columns n.. of a row of `width`, fp32 in, stored as T;
// kFull: all eight exist.
template <typename T, bool kFull>
__device__ __forceinline__ void store8(T* row, int n, int width, const float (&v)[8]) {
  constexpr int V = Piece<T>::V;
#pragma unroll
  for (int h = 0; h < 8 / V; ++h) {
    float e[V];
#pragma unroll
    for (int q = 0; q < V; ++q) e[q] = v[h * V + q];
    if (kFull) store_any(row + n + h * V, Piece<T>::narrow(e));
    else if (n + h * V < width) store_piece(row, n + h * V, width, e);
  }
}

// ------------------------------------------------------------- reductions

// Sum and maximum over the 64 lanes, in every lane: four data-parallel
// moves inside rows of 16 lanes, then the swaps of rows and halves.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane16(float v, float* other) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float lane32(float v, float* other) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float row16_sum(float v) {  // over the lane's row of 16
  v += dpp<0xb1>(v);   // lane ^ 1
  v += dpp<0x4e>(v);   // lane ^ 2
  v += dpp<0x141>(v);  // half row mirrored
  return v + dpp<0x140>(v);  // row mirrored
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  float o;
  v = lane16(v, &o);
  v += o;
  v = lane32(v, &o);
  return v + o;
}

// ---------------------------------------------------------------- launches

hipError_t launch_norm(const moe_norm& n, const void* x, const float* w, const float* b, void* y,
                       float* mean, float* rstd, hipStream_t s);
size_t norm_ws_bytes(const moe_norm& n);
hipError_t launch_norm_bwd(const moe_norm& n, const void* x, const float* w, const float* mean,
                           const float* rstd, const void* dy, void* dx, float* dw, float* db,
                           void* ws, hipStream_t s);

size_t ffn_block_ws_bytes(const moe_ffn& f, bool training);
size_t ffn_block_saved_bytes(const moe_ffn& f);
hipError_t launch_ffn_block(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                            const void* wd, void* saved, void* out, void* ws, hipStream_t s);
hipError_t launch_ffn_block_bwd(const moe_ffn& f, const void* x, const void* wg, const void* wu,
                                const void* wd, const void* saved, const void* dy, void* dx,
                                void* dwg, void* dwu, void* dwd, void* ws, hipStream_t s);

inline int64_t i8_pitch(int64_t width) { return (width + 127) / 128 * 128; }
hipError_t launch_quantize_rows(int64_t rows, int width, int dtype, const void* x, int64_t ld_x,
                                int8_t* q, float* scale, hipStream_t s);
hipError_t launch_quantize_weight(int groups, int width, int outputs, int dtype, const void* w,
                                  int64_t q_rows, int8_t* q, float* scale, hipStream_t s);
size_t linear_i8_ws_bytes(const moe_i8_linear& l);
hipError_t launch_linear_i8(const moe_i8_linear& l, const void* x, const float* xs,
                            const int8_t* wq, const float* ws, const float* bias,
                            const moe_routing* r, void* y, void* work, hipStream_t s);

size_t linear_ws_bytes(const moe_linear& l, bool training);
size_t linear_saved_bytes(const moe_linear& l);
hipError_t launch_linear(const moe_linear& l, const void* x, const void* w, const float* bias,
                         const void* res, void* saved, void* y, void* ws, hipStream_t s);
hipError_t launch_linear_bwd(const moe_linear& l, const void* x, const void* w, const void* saved,
                             const void* dy, void* dx, void* dw, float* dbias, void* ws,
                             hipStream_t s);

hipError_t launch_residual_norm(const moe_residual_norm& n, const void* z, const void* res,
                                const moe_norm_params& w, void* out, void* y, float* stats,
                                hipStream_t s);
size_t residual_norm_ws_bytes(const moe_residual_norm& n);
hipError_t launch_residual_norm_bwd(const moe_residual_norm& n, const void* z, const void* res,
                                    const moe_norm_params& w, const float* stats, const void* dout,
                                    const void* dy, void* dz, void* dres, const moe_norm_grads& g,
                                    void* ws, hipStream_t s);

size_t balance_ws_bytes(const moe_balance& b);
size_t balance_saved_bytes(const moe_balance& b);
hipError_t launch_balance(const moe_balance& b, const void* x, const float* w, const int32_t* idx,
                          const uint8_t* mask, int32_t* counts, float* mean_prob, float* loss,
                          void* saved, void* ws, hipStream_t s);
hipError_t launch_balance_bwd(const moe_balance& b, const void* x, const uint8_t* mask,
                              const void* saved, const float* gloss, bool add,
                              void* dx, float* dw, void* ws, hipStream_t s);

}  // namespace moe
