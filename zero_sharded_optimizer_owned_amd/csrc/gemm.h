// Matrix products on the matrix cores: out[m][n] = sum over k of P[m][k] Q[n][k],
// operands in 16 bits, sums in fp32.
//
// A block of 512 threads makes an M x 256 tile, k in steps of 64.  With M = 256 its
// eight wavefronts take 128 x 64 each (two in m, four in n).  Up to 128 rows take
// M = 128 (64 x 64 each): those products are bound by the reading of Q, and the
// smaller tile leaves LDS for one more step under way.  A step's tiles (128 bytes
// for each m and n) are loaded straight into LDS, 16 bytes to a lane, one step
// (M = 256) or two ahead.
//
// An operand is laid out either with k contiguous (Rows: element (r, k) at r
// stride + k) or with r contiguous (Columns: at k stride + r).  Rows' tiles hold
// 64 k of a row in 128 bytes and are read by ds_read_b128; Columns' tiles hold
// 256 r of a k in 512 bytes and are read by the transposing read
// (ds_read_b64_tr_b16: 16 lanes fetch 4 k by 16 r and get 4 k of one r each).
// Either way a lane then holds 8 consecutive k of one r.  The direct load
// writes LDS in lane order, so the exclusive-or that spreads the banks is
// applied to the global address: 16-byte piece c of a row lies at piece
// c ^ swizzle(row).
//
// The products are formed with Q first, so that a lane's four results are four
// consecutive n of one m.
//
// Measured in a training step of 6962 rows that count, 128,000 x 4096, bf16 (7.3
// TFLOP each): logits 6.2 to 6.4 ms, dhidden 5.8, dweight 6.4, 1.15 to 1.25 PFLOP/s, the
// matrix cores busy in 56 to 64% of the cycles (a library product of the first
// shape alone: 1.43).  What bounds it is the way of the tiles into LDS, 64 KB a
// step: in scores of 4096 such rows an earlier form took 3.21 ms, 2.94 with half of
// the products left out, 2.49 without the loads.  256 x 256 is the largest tile whose sums fit the
// registers.  Slower: 128 rows to a tile for all (13%: half as much again to load),
// 32 x 32 products (4%), four wavefronts of 128 x 128 (7 to 10%: sums moved between
// register files).  Steps of 32 k with five under way, in requests of 64 bytes, were
// no faster.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vec.h"

namespace zs {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t wave_of_block() { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

constexpr int kGemmThreads = 512;
constexpr int kWaves = kGemmThreads / 64;
constexpr int kTileN = 256, kTileK = 64;

// threadIdx.x, not to be recognised as such: what is computed from it behind a
// product would otherwise be computed before it and kept in registers meanwhile,
// of which the sums leave few.
__device__ __forceinline__ uint32_t thread_anew() {
  uint32_t t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// Tiles of M rows with `Slots` steps in LDS.
template <int M, int Slots>
struct Tile {
  static constexpr int kM = M, kSlots = Slots;
  static constexpr int kBytesP = M * kTileK * 2, kSlotBytes = kBytesP + kTileN * kTileK * 2, kLds = Slots * kSlotBytes;
  static constexpr int kWavesM = 2, kWavesN = kWaves / kWavesM;
  static constexpr int kWaveM = M / kWavesM, kWaveN = kTileN / kWavesN;  // of one wavefront
  static constexpr int kI = kWaveM / 16, kJ = kWaveN / 16;
  static constexpr int kLoads = M / 64 + kTileN / 64;  // a wavefront's, of a step
  typedef f32x4 Acc[kI][kJ];
  // acc[i][j][x] of thread t is m = row(i, t), n = column(j, t) + x of the tile
  static __device__ __forceinline__ uint32_t row(int i, uint32_t t) {
    return wave_of_block() / kWavesN * kWaveM + 16 * i + t % 16;
  }
  static __device__ __forceinline__ uint32_t column(int j, uint32_t t) {
    return wave_of_block() % kWavesN * kWaveN + 16 * j + t % 64 / 16 * 4;
  }
};
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every buffer: reads zero

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4 a, const u32x4 b, const f32x4 c) {
  if constexpr (DT == ZERO_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) char lds_char;

// The next 16 bytes of each lane from base + offset to LDS address `to` + 16 lane.
// Written in assembly because the compiler, which cannot tell the slots apart,
// would let every read of LDS wait for all loads under way; gemm_tile waits for
// the step that it reads.  The instruction has no output register.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t offset, uint32_t to) {
  const u32x4 buffer = {(uint32_t)(uintptr_t)base, (uint32_t)((uintptr_t)base >> 32), 0x7FFFFFFFu, 0x00020000u};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(offset), "s"(buffer)
               : "m0");
}

// R rows, k contiguous.  `base`: row 0 of the tile; rows from `rows` on and k from
// `depth` (a multiple of 8) on are zero.  256 rows are under 2 GB.
template <int R>
struct Rows {
  static constexpr int kLoads = R / 64;  // of each wavefront: 8 rows of 128 bytes
  const char* base;
  uint32_t offset[kLoads], k;
  uint32_t depth;

  __device__ __forceinline__ void begin(const void* p, uint64_t row0, uint32_t n_rows, uint64_t stride, uint32_t depth_) {
    base = static_cast<const char*>(p) + row0 * stride * 2;
    depth = depth_;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t rows = n_rows > row0 ? (uint32_t)min((uint64_t)n_rows - row0, (uint64_t)R) : 0;
    k = ((lane % 8) ^ (lane / 8)) * 8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t row = (wave * kLoads + i) * 8 + lane / 8;
      offset[i] = row < rows ? (uint32_t)(row * stride * 2) + k * 2 : kNowhere;
    }
  }
  __device__ __forceinline__ void load(uint32_t k0, uint32_t tile, int i) const {
    load_to_lds(base + (uint64_t)k0 * 2, k0 + k < depth ? offset[i] : kNowhere, tile + (wave_of_block() * kLoads + i) * 1024);
  }
  // Eight k from 32 kk + 8 (lane / 16) on of row r0 + lane % 16.
  static __device__ __forceinline__ u32x4 fragment(const lds_char* tile, uint32_t r0, uint32_t kk, uint32_t lane) {
    const uint32_t row = r0 + lane % 16, piece = (lane / 16 + 4 * kk) ^ (row % 8);
    return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(tile + row * 128 + piece * 16);
  }
};

// R columns, r contiguous.  `base`: column r0 of row 0; columns from `columns` (a
// multiple of 8) on and k from `depth` on are zero.
template <int R>
struct Columns {
  static constexpr int kLoads = R / 64, kPieces = R / 8;  // of each wavefront; of a row of 2 R bytes
  const char* base;
  uint64_t stride;
  uint32_t offset[kLoads];
  uint32_t depth;

  static __device__ __forceinline__ uint32_t row_of(int i) {
    return (wave_of_block() * kLoads + i) * (64 / kPieces) + threadIdx.x % 64 / kPieces;
  }
  __device__ __forceinline__ void begin(const void* p, uint64_t column0, uint32_t n_columns, uint64_t stride_, uint32_t depth_) {
    base = static_cast<const char*>(p) + column0 * 2;
    stride = stride_;
    depth = depth_;
    const uint32_t columns = n_columns > column0 ? (uint32_t)min((uint64_t)n_columns - column0, (uint64_t)R) : 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t row = row_of(i), c = (threadIdx.x % kPieces) ^ swizzle(row);
      offset[i] = c * 8 < columns ? (uint32_t)(row * stride * 2) + c * 16 : kNowhere;
    }
  }
  // A transposing read takes 32 bytes of each of 4 rows, and two groups of 16
  // lanes at a time rows 8 apart: all in different banks.
  static __device__ __forceinline__ uint32_t swizzle(uint32_t row) {
    return (row % 4) << 1 | (row / 8 % 2) << 3;
  }
  __device__ __forceinline__ void load(uint32_t k0, uint32_t tile, int i) const {
    load_to_lds(base + k0 * stride * 2, k0 + row_of(i) < depth ? offset[i] : kNowhere,
                tile + (wave_of_block() * kLoads + i) * 1024);
  }
  static __device__ __forceinline__ u32x4 fragment(const lds_char* tile, uint32_t r0, uint32_t kk, uint32_t lane) {
    u32x4 f;
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) {
      const uint32_t row = 32 * kk + 8 * (lane / 16) + 4 * h + lane % 16 / 4;
      const uint32_t piece = (r0 / 8 + lane % 4 / 2) ^ swizzle(row);
      const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(tile + row * (2 * R) + piece * 16 + lane % 2 * 8));
      const u32x2 w = __builtin_bit_cast(u32x2, q);
      f[2 * h] = w[0];
      f[2 * h + 1] = w[1];
    }
    return f;
  }
};

// Until at most N of this wavefront's loads are under way, and its reads of LDS are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N == 0 || N == 6, "a count the assembly is written for");
  if constexpr (N == 0) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)" ::: "memory");
}

template <class T>
__device__ __forceinline__ void clear(typename T::Acc& acc) {
#pragma unroll
  for (int i = 0; i < T::kI; ++i)
#pragma unroll
    for (int j = 0; j < T::kJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
}

// Adds to acc.  k runs over [k_begin, k_end), k_begin a multiple of 64; both
// operands are zero from k_end on.
template <int DT, class T, class P, class Q>
__device__ __forceinline__ void gemm_tile(const P& p, const Q& q, uint32_t k_begin, uint32_t k_end, lds_char* lds,
                                          typename T::Acc& acc) {
  constexpr int I = T::kI, J = T::kJ;
  static_assert(P::kLoads + Q::kLoads == T::kLoads, "operands of the tile's sizes");
  const uint32_t m0 = wave_of_block() / T::kWavesN * T::kWaveM, n0 = wave_of_block() % T::kWavesN * T::kWaveN;
  if (k_begin >= k_end) return;
  // Half steps of 32 k.  A half step's fragments are read during the one
  // before: those of Q into registers of their own, those of P each behind the
  // last product of the one it replaces.  In the second half the next step's
  // tiles are read, behind a barrier at which they have arrived and this step's
  // are no longer read, so that the loads of a later step can take its slot.
  u32x4 a[2][J], b[I];
  const uint32_t base = (uint32_t)(uintptr_t)lds, lane = threadIdx.x & 63;
  const auto load = [&](uint32_t k, uint32_t slot, int i) {  // this wavefront's i-th load of a step
    if (i < P::kLoads) p.load(k, base + slot, i);
    else q.load(k, base + slot + T::kBytesP, i - P::kLoads);
  };
  const auto arrive = [&]() {
    wait_loads<(T::kSlots - 2) * T::kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  uint32_t k_load = k_begin;
#pragma unroll
  for (int s = 0; s < T::kSlots - 1; ++s) {
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) load(k_load, s * T::kSlotBytes, i);
    k_load += kTileK;
  }
  arrive();
#pragma unroll
  for (int i = 0; i < T::kLoads; ++i) load(k_load, (T::kSlots - 1) * T::kSlotBytes, i);
  k_load += kTileK;
#pragma unroll
  for (int j = 0; j < J; ++j) a[0][j] = Q::fragment(lds + T::kBytesP, n0 + 16 * j, 0, lane);
#pragma unroll
  for (int i = 0; i < I; ++i) b[i] = P::fragment(lds, m0 + 16 * i, 0, lane);
  uint32_t now = 0;
  const auto half = [&](uint32_t h, const lds_char* from, uint32_t free) {
#pragma unroll
    for (int j = 0; j < J; ++j) a[h ^ 1][j] = Q::fragment(from + T::kBytesP, n0 + 16 * j, h ^ 1, lane);
#pragma unroll
    for (int i = 0; i < I; ++i) {
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = mfma16<DT>(a[h][j], b[i], acc[i][j]);
      b[i] = P::fragment(from, m0 + 16 * i, h ^ 1, lane);
      if (h == 1) {
        constexpr int kEach = (T::kLoads + I / 2 - 1) / (I / 2);  // within the first half of the products
#pragma unroll
        for (int l = i * kEach; l < (i + 1) * kEach; ++l)
          if (l < T::kLoads) load(k_load, free, l);
      }
      __builtin_amdgcn_sched_barrier(0);  // in this order: left to itself the compiler reads just before the use
    }
  };
  for (uint32_t k = k_begin; k < k_end; k += kTileK) {
    half(0, lds + now, 0);
    arrive();
    const uint32_t free = now;
    now = now + T::kSlotBytes == T::kLds ? 0 : now + T::kSlotBytes;
    half(1, lds + now, free);  // behind the last step, of zeros that are not used
    k_load += kTileK;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

// A tile in 16 bits goes to memory by way of LDS, so that a row's 512 bytes are
// stored by 32 lanes in one go (a lane of the products holds 8 of them).  16-byte
// piece c of row m lies at piece c ^ m % 32: all banks at once, both ways.
template <int DT>
__device__ __forceinline__ void put_quad(char* lds, uint32_t m, uint32_t n, const f32x4 x) {
  *reinterpret_cast<u32x2*>(lds + m * 512 + ((n / 8) ^ (m % 32)) * 16 + n % 8 * 2) =
      u32x2{Vec<DT>::pack(x[0], x[1]), Vec<DT>::pack(x[2], x[3])};
}

// `row(m)`: where row m of the tile begins, NULL for none; columns from `columns`
// (a multiple of 8) on are left out.
template <int M, typename F>
__device__ __forceinline__ void store_rows(const char* lds, uint32_t columns, uint32_t t, F row) {
  const uint32_t c = t % 32;
#pragma unroll 4
  for (uint32_t m = t / 32; m < M; m += kGemmThreads / 32) {
    uint16_t* to = row(m);
    if (to && c * 8 < columns)
      *reinterpret_cast<u32x4*>(to + c * 8) = *reinterpret_cast<const u32x4*>(lds + m * 512 + (c ^ (m % 32)) * 16);
  }
}

// The tile times f.  The caller's wavefronts are done with LDS.
template <int DT, class T, typename F>
__device__ __forceinline__ void store_tile(const typename T::Acc& acc, float f, uint32_t columns, char* lds, uint32_t t, F row) {
  static_assert(T::kM * kTileN * 2 <= T::kLds, "the tile in 16 bits");
#pragma unroll
  for (int i = 0; i < T::kI; ++i)
#pragma unroll
    for (int j = 0; j < T::kJ; ++j) put_quad<DT>(lds, T::row(i, t), T::column(j, t), acc[i][j] * f);
  __syncthreads();
  store_rows<T::kM>(lds, columns, t, row);
}

}  // namespace zs
