// Tiled matrix-product engine of the operators around the layer (gfx950).
//
//   C[m][n] = sum_k A[m][k] B[n][k]     bf16 or fp32 -> fp32, int8 -> int32
//
// Both operands are rows of K-contiguous bytes, a stage being 64 or 128 bytes
// of every row (128: 64 bf16, 32 fp32 or 128 int8), so one engine serves all
// types: the fragments of mfma 32x32x16 bf16, of 32x32x32 i8 and of four
// 32x32x2 fp32 steps are the same 16 bytes a lane. Rows come through pointers
// computed once per tile, which is where gathering by the expert permutation,
// clamping at the last row and the pairing of gate and up columns happen.
//
// Stages go from global memory straight into LDS (no staging registers), in a
// ring of buffers; the 16-byte chunks of an LDS row are swizzled so that the
// rows which a fragment read touches spread over all banks. The MFMA takes
// the B fragment first: lane L then holds row L % 32 and runs of four
// consecutive columns, 8 (q / 4) + 4 (L / 32) + q % 4 for register q.
//
// What bounds it: a CU loads 64 bytes a clock, and a 128 x 128 tile needs as
// many clocks for that as for its MFMAs, 256 x 128 three quarters, 256 x 256
// half; the reads from LDS take 1.5, 1.1 and 0.75 of the MFMAs' time. So large
// tiles where there are enough of them: bf16 with K 2048 to 8192 reaches 1.0
// to 1.2 PFLOP/s (the vendor library's product of 8192 x 8192 matrices on the
// same card: 1.13), int8 16384 x 4096 x 4096 1.9 POP/s (library: 2.0). With K
// 512 the epilogue, which writes as many bytes as the loop reads, is half of
// the time (0.35 to 0.65 PFLOP/s).
#pragma once

#include "block.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct OpBf16 {
  static constexpr int kMfma = 1;  // MFMAs a step
  typedef f32x16_t Acc;
  __device__ static void step(const u32x4& w, const u32x4& x, Acc& acc) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                  __builtin_bit_cast(bf16x8_t, x), acc, 0, 0, 0);
  }
};
struct OpF32 {
  static constexpr int kMfma = 4;
  typedef f32x16_t Acc;
  // step e takes element e of each lane group's 16 bytes, on both sides
  __device__ static void step(const u32x4& w, const u32x4& x, Acc& acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w[e]), __uint_as_float(x[e]), acc, 0, 0, 0);
  }
};
struct OpI8 {
  static constexpr int kMfma = 1;
  typedef i32x16 Acc;
  __device__ static void step(const u32x4& w, const u32x4& x, Acc& acc) {
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, w),
                                                __builtin_bit_cast(i32x4, x), acc, 0, 0, 0);
  }
};

struct MmArgs {
  const char* a;
  int64_t a_pitch;   // bytes between rows
  const int32_t* perm;  // gather: row r reads input row perm[r] / top_k
  double per_token;     // 1 / topk
  const char* b;
  int64_t b_pitch, b_group;  // bytes between rows, between groups
  const char* a2;            // stages from k_split on come from a2 and b2, each
  const char* b2;            // with its own k 0 first (null: none)
  int k_split;
  int nk;                    // stages
  int64_t M;                 // dense: rows
  int N;                     // rows of B; paired: of one half
  const int32_t* offsets;    // routed: expert_offsets, else null
  int groups, cap;
  int parts;                 // dense: slices of K, each a workgroup's own sum
  int tiles_n;
  int64_t half;              // paired: bytes from a gate row of B to its up row
};


template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int RING_ = 4, int ROW_ = 64>
struct MmCfg {
  static constexpr int ROW = ROW_;    // bytes of a row in a stage
  static constexpr int CPR = ROW / 16, RPL = 64 / CPR;  // chunks of a row; rows of a load
  static constexpr int STEPS = ROW / 32;
  static constexpr int RING = RING_;  // stage buffers
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int NW = WAVES_M * WAVES_N, NT = 64 * NW;
  static constexpr int WM = BM / WAVES_M / 32, WN = BN / WAVES_N / 32;  // MFMA tiles per wave
  static constexpr int A_LOADS = BM / RPL / NW, B_LOADS = BN / RPL / NW;     // a wave and stage
  static constexpr int WPE = WM * WN == 16 ? 1 : 2;  // waves to a SIMD: 256 accumulators leave room for one
  static constexpr int STAGE = (BM + BN) * ROW, LDS = RING * STAGE;
  static_assert(BM == WAVES_M * WM * 32 && BN == WAVES_N * WN * 32, "tiles");
  static_assert(BM % (RPL * NW) == 0 && BN % (RPL * NW) == 0, "loads");
};

// This wave's number, as a scalar: what is made of it stays off the vector
// units (the LDS addresses of the loads among it).
__device__ __forceinline__ int mm_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Token of a slot: slot / topk without an integer division (a slot plus a half
// is at least a half of 1 / topk from a multiple, far more than a rounding).
__device__ __forceinline__ int mm_token(const MmArgs& p, int32_t slot) {
  return static_cast<int>(__builtin_fma(static_cast<double>(slot), p.per_token, 0.5 * p.per_token));
}

// Position of chunk c of LDS row r: c ^ mm_swizzle(r), which spreads the rows
// that a fragment read touches over all banks.
template <typename Cfg>
__device__ __forceinline__ int mm_swizzle(int r) {
  return Cfg::ROW == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
}

// The tile sizes in use.
using MmBig = MmCfg<256, 256, 2, 2, 2, 128>;   // one wave to a SIMD
using MmTall = MmCfg<256, 128, 2, 2, 3, 64>;   // two workgroups a CU
using MmMid = MmCfg<128, 128, 2, 2, 3, 64>;    // three
using MmSmall = MmCfg<64, 64, 2, 2, 3, 128>;   // three

// A tile's rows: first row, count (0: nothing to do), weight group.
struct MmTile {
  int64_t row0;
  int rows, group, nt;
  int part, k0, k1;  // slice of K and its stages
};

// The workgroup's tile of routed rows: each lane counts one expert's row tiles
// (at most 64 experts), a prefix sum finds the expert. Uniform over the wave.
// The grid is for the most tiles that the rows can make; those that there are
// go to the XCDs in equal ranges: in the order of the grid a few experts' rows
// would keep two of the eight busy (8 tokens, top-2 of 64 experts of 2048 x
// 2048 in int8: 40 us against 16).
__device__ __forceinline__ MmTile mm_routed_tile(const int32_t* offsets, int groups, int cap, int bm,
                                                 int tiles_n, int lane) {
  int first = 0, count = 0;
  if (lane < groups) {
    first = offsets[lane];
    count = offsets[lane + 1] - first;
    if (cap > 0 && count > cap) count = cap;
  }
  const int tiles = (count + bm - 1) / bm;
  int upto = tiles;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  MmTile t{};
  const int total = __shfl(upto, 63) * tiles_n;
  if (static_cast<int>(blockIdx.x) >= total) return t;
  const int w = xcd_remap(blockIdx.x, total), mt = w / tiles_n;
  t.nt = w % tiles_n;
  const uint64_t past = __ballot(upto > mt);
  const int e = __ffsll(static_cast<unsigned long long>(past)) - 1;
  const int local = mt - (__shfl(upto, e) - __shfl(tiles, e));
  t.group = __builtin_amdgcn_readfirstlane(e);
  t.row0 = __builtin_amdgcn_readfirstlane(__shfl(first, e) + local * bm);
  const int left = __builtin_amdgcn_readfirstlane(__shfl(count, e) - local * bm);
  t.rows = left < bm ? left : bm;
  return t;
}

// Order of the dense tiles: bands of eight row tiles, column by column, so
// that the workgroups running together share rows of A and of B in L2.
__device__ __forceinline__ void mm_tile_order(int w, int tiles_m, int tiles_n, int* mt, int* nt) {
  constexpr int kBand = 8;
  const int band = w / (kBand * tiles_n), in = w % (kBand * tiles_n);
  const int high = min(kBand, tiles_m - band * kBand);
  *mt = band * kBand + in % high;
  *nt = in / high;
}

// At most N of this wave's loads left in flight, its LDS reads done.
template <int N>
__device__ __forceinline__ void mm_wait() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

constexpr int mm_gcd(int a, int b) { return b ? mm_gcd(b, a % b) : a; }

// The main loop. The fragments of a step (32 bytes of K) are read while the
// step before is multiplied, the reads spread between the MFMAs, so that no
// wave waits for LDS. One barrier a stage, before its last step: it says that
// the next stage is whole and that nobody reads this one any more, whose
// buffer is then loaded again, RING stages ahead.
template <typename Op, typename Cfg, typename Load>
__device__ __forceinline__ void mm_loop(char* smem, int nk, int a_frag, int b_frag, int sw,
                                        typename Op::Acc (&acc)[Cfg::WM][Cfg::WN], Load&& load) {
  constexpr int WM = Cfg::WM, WN = Cfg::WN, kFrags = WM + WN, kMfma = WM * WN;
  constexpr int kLoads = Cfg::A_LOADS + Cfg::B_LOADS, kSteps = Cfg::STEPS;
  constexpr int G = mm_gcd(mm_gcd(kFrags, kMfma), kLoads);  // groups of a step
  static_assert(kSteps % 2 == 0, "the last step of a stage uses set 1");
  u32x4 x[2][WM], w[2][WN];
  // fragment f of step q: A's, then B's
  auto read = [&](const char* buf, int q, int f, int set) {
    const int at = ((2 * q) ^ sw) << 4;
    if (f < WM) x[set][f < WM ? f : 0] = *reinterpret_cast<const u32x4*>(buf + a_frag + f * 32 * Cfg::ROW + at);
    else w[set][f < WM ? 0 : f - WM] = *reinterpret_cast<const u32x4*>(buf + b_frag + (f - WM) * 32 * Cfg::ROW + at);
  };
  // The MFMAs of one step on `set`, with the reads of step q of `from` into
  // the other set and, where kLoad, the loads of stage st into `into`; the
  // scheduler is given the same order.
  auto step = [&](auto with_loads, int set, const char* from, int q, int st, char* into) {
    constexpr bool kLoad = decltype(with_loads)::value;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if constexpr (kLoad) {
#pragma unroll
        for (int u = 0; u < kLoads / G; ++u) load(st, into, g * (kLoads / G) + u);
        __builtin_amdgcn_sched_group_barrier(0x010, kLoads / G, 0);
      }
#pragma unroll
      for (int f = 0; f < kFrags / G; ++f) read(from, q, g * (kFrags / G) + f, set ^ 1);
      __builtin_amdgcn_sched_group_barrier(0x100, kFrags / G, 0);
#pragma unroll
      for (int m = 0; m < kMfma / G; ++m) {
        const int n = g * (kMfma / G) + m;
        Op::step(w[set][n % WN], x[set][n / WN], acc[n / WN][n % WN]);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, kMfma / G * Op::kMfma, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto stage = [&](auto with_loads, int s) {
    constexpr bool kLoad = decltype(with_loads)::value;
    char* cur = smem + (s % Cfg::RING) * Cfg::STAGE;
    const char* next = smem + ((s + 1) % Cfg::RING) * Cfg::STAGE;
#pragma unroll
    for (int q = 0; q + 1 < kSteps; ++q) step(std::false_type{}, q & 1, cur, q + 1, 0, nullptr);
    // stage s + 1 has landed (those behind it may be in flight), the reads of
    // stage s are done
    mm_wait<kLoad ? kLoads * (Cfg::RING - 2) : 0>();
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    step(with_loads, 1, next, 0, s + Cfg::RING, cur);
  };
#pragma unroll
  for (int st = 0; st < Cfg::RING; ++st)
    if (st < nk) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) load(st, smem + st * Cfg::STAGE, u);
    }
  if (nk >= Cfg::RING) mm_wait<kLoads * (Cfg::RING - 1)>();
  else mm_wait<0>();
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int f = 0; f < kFrags; ++f) read(smem, 0, f, 0);
  int s = 0;
  for (; s + Cfg::RING < nk; ++s) stage(std::true_type{}, s);
  for (; s < nk; ++s) stage(std::false_type{}, s);  // after the last one `next` is read without use
}

// Tile w (of part `part`) of a dense product. False: no such tile.
template <typename Cfg>
__device__ __forceinline__ bool mm_place(const MmArgs& p, int w, int part, MmTile* tile) {
  MmTile t{};
  int mt;
  mm_tile_order(w, static_cast<int>((p.M + Cfg::BM - 1) / Cfg::BM), p.tiles_n, &mt, &t.nt);
  t.row0 = static_cast<int64_t>(mt) * Cfg::BM;
  const int64_t left = p.M - t.row0;
  t.rows = left < Cfg::BM ? static_cast<int>(left) : Cfg::BM;
  t.part = part;
  t.k0 = p.parts > 1 ? static_cast<int>(static_cast<int64_t>(p.nk) * part / p.parts) : 0;
  t.k1 = p.parts > 1 ? static_cast<int>(static_cast<int64_t>(p.nk) * (part + 1) / p.parts) : p.nk;
  *tile = t;
  return t.rows > 0;
}

// One workgroup's tile, from its index.
template <typename Cfg>
__device__ __forceinline__ bool mm_find(const MmArgs& p, MmTile* tile) {
  if (p.offsets) {
    *tile = mm_routed_tile(p.offsets, p.groups, p.cap, Cfg::BM, p.tiles_n, threadIdx.x & 63);
    tile->k1 = p.nk;
    return tile->rows > 0;
  }
  const int w = xcd_remap(blockIdx.x, gridDim.x);
  const int tiles = p.parts > 1 ? gridDim.x / p.parts : gridDim.x;
  return mm_place<Cfg>(p, w % tiles, w / tiles, tile);
}

// Position of chunk c of k row r in a stage of a B that is [K][N]: the four
// rows of a transposing read spread over all banks.
template <typename Cfg>
__device__ __forceinline__ int mm_turned_at(int r, int c) {
  return c ^ (Cfg::BN == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2);
}

// The loop for a B that is [K][N], N contiguous, of bf16, in 64 or 128
// columns: a stage holds as many rows of k as its rows of A have elements. The
// transposing LDS read makes eight k of a column of them: in a group of 16
// lanes, lane s addresses row s / 4, columns 4 (s % 4) .. + 3, and lane j
// receives the four rows of column j. All the reads of a stage are one
// statement with their wait, for the compiler would wait before its builtin
// for every load in flight (200 tokens, 2048 x 2048: 35 us against 24); what
// is not spread between MFMAs, the other workgroups of the CU cover. Loads go
// RING - 1 stages ahead, into the buffer that all waves have read when they
// meet at the one barrier of a stage. Two buffers took 32 us there, four 25.
template <typename Op, typename Cfg, typename Load>
__device__ __forceinline__ void mm_loop_turned(char* smem, int nk, int a_frag, int sw, int col0,
                                               typename Op::Acc (&acc)[Cfg::WM][Cfg::WN], Load&& load) {
  constexpr bool kWide = Cfg::BN == 128;
  static_assert(kWide ? Cfg::ROW == 64 && Cfg::WM == 2 && Cfg::WN == 2
                      : Cfg::BN == 64 && Cfg::ROW == 128 && Cfg::WM == 1 && Cfg::WN == 1, "tiles");
  constexpr int kLoads = Cfg::A_LOADS + Cfg::B_LOADS, kAhead = Cfg::RING - 1;
  constexpr int kSteps = Cfg::STEPS, kB = Cfg::WN;
  const int lane = threadIdx.x & 63, s16 = lane & 15, g16 = lane >> 4;
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
  const int row = 8 * (g16 >> 1) + (s16 >> 2);
  uint32_t a[kSteps], b[kB];
#pragma unroll
  for (int q = 0; q < kSteps; ++q) a[q] = base + a_frag + (((2 * q) ^ sw) << 4);
#pragma unroll
  for (int j = 0; j < kB; ++j) {
    const int col = col0 + 32 * j + 16 * (g16 & 1) + 4 * (s16 & 3);
    b[j] = base + Cfg::BM * Cfg::ROW + row * Cfg::BN * 2 + (mm_turned_at<Cfg>(row, col >> 3) << 4) + (col & 7) * 2;
  }
#pragma unroll
  for (int st = 0; st < kAhead; ++st)
    if (st < nk) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) load(st, smem + st * Cfg::STAGE, u);
    }
  int at = 0, to = kAhead * Cfg::STAGE;
  for (int s = 0; s < nk; ++s) {
    if (s + kAhead <= nk) mm_wait<kLoads * (kAhead - 1)>();
    else mm_wait<0>();
    asm volatile("s_barrier" ::: "memory");
    if (s + kAhead < nk) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) load(s + kAhead, smem + to, u);
    }
    // x[step WM + i], w[2 (step WN + j) + half]: steps are 16 rows of k apart,
    // halves four, A's fragments 32 rows
    u32x4 x[4];
    uint64_t w[8];
    if constexpr (kWide) {
      asm volatile(
          "ds_read_b64_tr_b16 %4, %14\n\t"
          "ds_read_b64_tr_b16 %5, %14 offset:1024\n\t"
          "ds_read_b128 %0, %12\n\t"
          "ds_read_b64_tr_b16 %6, %15\n\t"
          "ds_read_b64_tr_b16 %7, %15 offset:1024\n\t"
          "ds_read_b128 %1, %12 offset:2048\n\t"
          "ds_read_b64_tr_b16 %8, %14 offset:4096\n\t"
          "ds_read_b64_tr_b16 %9, %14 offset:5120\n\t"
          "ds_read_b128 %2, %13\n\t"
          "ds_read_b64_tr_b16 %10, %15 offset:4096\n\t"
          "ds_read_b64_tr_b16 %11, %15 offset:5120\n\t"
          "ds_read_b128 %3, %13 offset:2048\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]),
            "=&v"(w[3]), "=&v"(w[4]), "=&v"(w[5]), "=&v"(w[6]), "=&v"(w[7])
          : "v"(a[0] + at), "v"(a[1] + at), "v"(b[0] + at), "v"(b[kB - 1] + at)
          : "memory");
    } else {
      asm volatile(
          "ds_read_b64_tr_b16 %4, %16\n\t"
          "ds_read_b64_tr_b16 %5, %16 offset:512\n\t"
          "ds_read_b128 %0, %12\n\t"
          "ds_read_b64_tr_b16 %6, %16 offset:2048\n\t"
          "ds_read_b64_tr_b16 %7, %16 offset:2560\n\t"
          "ds_read_b128 %1, %13\n\t"
          "ds_read_b64_tr_b16 %8, %16 offset:4096\n\t"
          "ds_read_b64_tr_b16 %9, %16 offset:4608\n\t"
          "ds_read_b128 %2, %14\n\t"
          "ds_read_b64_tr_b16 %10, %16 offset:6144\n\t"
          "ds_read_b64_tr_b16 %11, %16 offset:6656\n\t"
          "ds_read_b128 %3, %15\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]),
            "=&v"(w[3]), "=&v"(w[4]), "=&v"(w[5]), "=&v"(w[6]), "=&v"(w[7])
          : "v"(a[0] + at), "v"(a[1] + at), "v"(a[kSteps - 2] + at), "v"(a[kSteps - 1] + at), "v"(b[0] + at)
          : "memory");
    }
#pragma unroll
    for (int q = 0; q < kSteps; ++q)
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const uint64_t lo = w[2 * (q * kB + j)], hi = w[2 * (q * kB + j) + 1];
        const u32x4 v = {static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                         static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
#pragma unroll
        for (int i = 0; i < Cfg::WM; ++i) Op::step(v, x[q * Cfg::WM + i], acc[i][j]);
      }
    at = at + Cfg::STAGE == Cfg::LDS ? 0 : at + Cfg::STAGE;
    to = to + Cfg::STAGE == Cfg::LDS ? 0 : to + Cfg::STAGE;
  }
}

// The tile's sums. kPaired: B's tile holds gate rows and up rows in turns of
// 16 (column p of the tile is gate column 16 (p / 32) + p % 16 of the pair
// block when p % 32 < 16, else the same up column), so a lane's registers
// 0-7 and 8-15 of an MFMA tile are matching gate and up values.
//
// kTurned (mm_loop_turned): B is [K][N], N contiguous, K a multiple of 64 and N of 8.
template <typename Op, typename Cfg, bool kPaired, bool kTurned = false>
__device__ __forceinline__ void mm_tile(const MmArgs& p, char* smem, const MmTile& t,
                                        typename Op::Acc (&acc)[Cfg::WM][Cfg::WN]) {
  const int lane = threadIdx.x & 63, wave = mm_wave();
  // Load i of a wave covers rows (wave LOADS + i) RPL + lane / CPR of an
  // operand's tile, lane l's 16 bytes landing at position l % CPR of the row:
  // the chunk that belongs there is (l % CPR) ^ mm_swizzle(row). Rows past the
  // tile repeat its last row; what they compute is not stored.
  const char* a[Cfg::A_LOADS];
  const char* b[Cfg::B_LOADS];
#pragma unroll
  for (int i = 0; i < Cfg::A_LOADS; ++i) {
    const int r = (wave * Cfg::A_LOADS + i) * Cfg::RPL + lane / Cfg::CPR;
    const int chunk = ((lane % Cfg::CPR) ^ mm_swizzle<Cfg>(r)) << 4;
    int64_t src = t.row0 + min(r, t.rows - 1);
    if (p.perm) src = mm_token(p, p.perm[src]);
    a[i] = p.a + src * p.a_pitch + chunk;
  }
#pragma unroll
  for (int i = 0; i < Cfg::B_LOADS; ++i) {
    if constexpr (kTurned) {
      constexpr int kChunks = Cfg::BN / 8;  // of a k row
      const int r = (wave * Cfg::B_LOADS + i) * (64 / kChunks) + lane / kChunks;
      const int c = mm_turned_at<Cfg>(r, lane % kChunks);
      const int col = kPaired ? t.nt * (Cfg::BN / 2) + 16 * (c >> 2) + 8 * (c & 1) : t.nt * Cfg::BN + 8 * c;
      b[i] = p.b + r * p.b_pitch + min(col, p.N - 8) * 2 + (kPaired && (c & 2) ? p.half : 0);
      continue;
    }
    const int r = (wave * Cfg::B_LOADS + i) * Cfg::RPL + lane / Cfg::CPR;
    const int chunk = ((lane % Cfg::CPR) ^ mm_swizzle<Cfg>(r)) << 4;
    int64_t off;
    if (kPaired) {
      const int c = t.nt * (Cfg::BN / 2) + 16 * (r >> 5) + (r & 15);
      off = min(c, p.N - 1) * p.b_pitch + ((r & 16) ? p.half : 0);
    } else {
      off = min(t.nt * Cfg::BN + r, p.N - 1) * p.b_pitch;
    }
    b[i] = p.b + t.group * p.b_group + off + chunk;
  }
  const int nk = t.k1 - t.k0;
  const int split = p.b2 ? p.k_split : p.nk;
  const int64_t a2 = p.b2 ? (p.a2 - p.a) - static_cast<int64_t>(split) * Cfg::ROW : 0;
  const int64_t b2 = p.b2 ? (p.b2 - p.b) - static_cast<int64_t>(split) * Cfg::ROW : 0;

  const int g = lane >> 5, r32 = lane & 31;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  const int a_frag = (wm * Cfg::WM * 32 + r32) * Cfg::ROW;
  const int b_frag = (Cfg::BM + wn * Cfg::WN * 32 + r32) * Cfg::ROW;
  const int sw = g ^ mm_swizzle<Cfg>(r32);
#pragma unroll
  for (int i = 0; i < Cfg::WM; ++i)
#pragma unroll
    for (int j = 0; j < Cfg::WN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;

  auto load = [&](int st, char* buf, int u) {
    const int64_t off = static_cast<int64_t>(st + t.k0) * Cfg::ROW;
    const int64_t off_b = kTurned ? static_cast<int64_t>(st + t.k0) * (Cfg::ROW / 2) * p.b_pitch : off;
    const bool first = st + t.k0 < split;
    if (u < Cfg::A_LOADS) {
      const char* src = a[u < Cfg::A_LOADS ? u : 0] + off + (first ? 0 : a2);
      char* dst = buf + (wave * Cfg::A_LOADS + u) * 1024;
      __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
    } else {
      const char* src = b[u < Cfg::A_LOADS ? 0 : u - Cfg::A_LOADS] + off_b + (first ? 0 : b2);
      char* dst = buf + Cfg::BM * Cfg::ROW + (wave * Cfg::B_LOADS + u - Cfg::A_LOADS) * 1024;
      __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
    }
  };
  if constexpr (kTurned) mm_loop_turned<Op, Cfg>(smem, nk, a_frag, sw, wn * Cfg::WN * 32, acc, load);
  else mm_loop<Op, Cfg>(smem, nk, a_frag, b_frag, sw, acc, load);
}

// Hands a finished tile out by rows. Stored straight from the accumulators,
// a store instruction would touch 32 rows with a few bytes each; instead each
// wave writes strips of 32 rows into LDS of its own (the stage buffers, free
// by now) and every lane takes eight consecutive columns of a row, so eight
// (paired: four) lanes cover whole cache lines. Callbacks, all inlined:
//   f.cols(j, n)      strip column j's first column of this lane (within the
//                     tile; paired: within the tile's hidden columns)
//   f.start(i, k, m)  row m of strip row i, pass k
//   f.pre(set, k, m)  the same before strip `set`'s rows are handed out
//   f.row(set, i, j, k, m, v), or (.., gate, up): the eight sums
// Vector memory completes in issue order, loads behind stores: a load that
// is issued after a strip's stores costs the wait for all of them (24 us a
// tile, more than the product took at 8 stages). So everything that does not
// change is read first, and pre runs one strip ahead of the stores. For the
// same reason nothing branches: a row past the tile repeats its last row's
// bits (its operands were that row's) and is stored over it.
constexpr int kMmStripPad = 16;  // bytes behind a strip row: spreads the rows over the banks
template <typename Cfg>
struct MmStrip {
  static constexpr int CB = Cfg::WN < 2 ? Cfg::WN : 2;  // MFMA tiles side by side in a strip
  static constexpr int PITCH = CB * 128 + kMmStripPad, BYTES = 32 * PITCH;
  // the workgroup's LDS: the ring, or the strips where they are larger
  static constexpr int LDS = Cfg::LDS > Cfg::NW * BYTES ? Cfg::LDS : Cfg::NW * BYTES;
};

// Passes over a strip: rows of it that a lane hands out.
template <typename Cfg, bool kPaired>
constexpr int mm_passes() {
  return 32 / (64 / (MmStrip<Cfg>::CB * (kPaired ? 16 : 32) / 8));
}

// The callbacks that read what does not change; called before the main loop,
// whose first wait covers them.
template <typename Cfg, bool kPaired, typename F>
__device__ __forceinline__ void mm_begin(int rows, F&& f) {
  using S = MmStrip<Cfg>;
  constexpr int COLS = S::CB * (kPaired ? 16 : 32), LPR = COLS / 8, RPP = 64 / LPR, PASSES = 32 / RPP;
  const int lane = threadIdx.x & 63, wave = mm_wave();
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
#pragma unroll
  for (int j = 0; j < Cfg::WN / S::CB; ++j)
    f.cols(j, (wn * Cfg::WN + j * S::CB) * (kPaired ? 16 : 32) + (lane % LPR) * 8);
#pragma unroll
  for (int i = 0; i < Cfg::WM; ++i)
#pragma unroll
    for (int k = 0; k < PASSES; ++k)
      f.start(i, k, min((wm * Cfg::WM + i) * 32 + lane / LPR + k * RPP, rows - 1));
}

template <typename Cfg, bool kPaired, typename Acc, typename F>
__device__ __forceinline__ void mm_drain(char* smem, const Acc (&acc)[Cfg::WM][Cfg::WN], int rows, F&& f) {
  using S = MmStrip<Cfg>;
  constexpr int COLS = S::CB * (kPaired ? 16 : 32);  // columns handed out per strip row
  constexpr int LPR = COLS / 8, RPP = 64 / LPR, PASSES = 32 / RPP;
  constexpr int NJ = Cfg::WN / S::CB, STRIPS = NJ * Cfg::WM;
  const int lane = threadIdx.x & 63, wave = mm_wave();
  const int g = lane >> 5, r32 = lane & 31;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  char* strip = smem + wave * S::BYTES;
  const int c8 = (lane % LPR) * 8, r0 = lane / LPR;
  // byte of the lane's first column in a strip row (paired: of its gate columns)
  const int at = kPaired ? (c8 / 16) * 128 + (c8 % 16) * 4 : c8 * 4;
  auto m_of = [&](int i, int k) { return min((wm * Cfg::WM + i) * 32 + r0 + k * RPP, rows - 1); };
#pragma unroll
  for (int k = 0; k < PASSES; ++k) f.pre(0, 0, k, m_of(0, k));
  // every wave is done with the stages
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int n = 0; n < STRIPS; ++n) {
    const int i = n % Cfg::WM, j = n / Cfg::WM;
    if (n + 1 < STRIPS) {
#pragma unroll
      for (int k = 0; k < PASSES; ++k)
        f.pre((n + 1) & 1, (n + 1) / Cfg::WM, k, m_of((n + 1) % Cfg::WM, k));
    }
#pragma unroll
    for (int c = 0; c < S::CB; ++c)
#pragma unroll
      for (int rr = 0; rr < 4; ++rr) {
        u32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const auto e = acc[i][j * S::CB + c][4 * rr + q];  // a value: bit_cast takes no vector element
          v[q] = __builtin_bit_cast(uint32_t, e);
        }
        *reinterpret_cast<u32x4*>(strip + r32 * S::PITCH + c * 128 + rr * 32 + g * 16) = v;
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      const char* src = strip + (r0 + k * RPP) * S::PITCH + at;
      u32x4 lo = *reinterpret_cast<const u32x4*>(src), hi = *reinterpret_cast<const u32x4*>(src + 16);
      const uint32_t v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      if constexpr (kPaired) {
        lo = *reinterpret_cast<const u32x4*>(src + 64);
        hi = *reinterpret_cast<const u32x4*>(src + 80);
        const uint32_t u[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        f.row(n & 1, i, j, k, m_of(i, k), v, u);
      } else {
        f.row(n & 1, i, j, k, m_of(i, k), v);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

}  // namespace moe
