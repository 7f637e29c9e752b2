// What the row kernels of the model's two ends share: reductions over a
// wavefront and over the wavefronts of a row, and vectors of a row whose last
// one may be cut.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vec.h"

namespace zs {

template <int CTRL>
__device__ __forceinline__ double dpp_add(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over a wavefront, in every lane: four rotations inside the rows of 16
// lanes, then the other rows.
__device__ __forceinline__ double wave_sum(double x) {
  x = dpp_add<0x128>(x);  // row_ror:8, 4, 2, 1
  x = dpp_add<0x124>(x);
  x = dpp_add<0x122>(x);
  x = dpp_add<0x121>(x);
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// Sum over the W wavefronts of a row, in every thread.  `part` holds the row's W
// numbers; a block's rows begin at multiples of W wavefronts.  SYNC: part may still be
// read from a sum before.
template <int W, bool SYNC = true>
__device__ __forceinline__ double row_sum(double x, double* part) {
  x = wave_sum(x);
  if constexpr (W > 1) {
    if constexpr (SYNC) __syncthreads();
    if ((threadIdx.x & 63) == 0) part[(threadIdx.x >> 6) % W] = x;
    __syncthreads();
    x = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) x += part[i];
  }
  return x;
}

// Largest of a DPP row's 16 values, in every lane of it.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t x) {
  x = dpp_max<0x128>(x);
  x = dpp_max<0x124>(x);
  x = dpp_max<0x122>(x);
  return dpp_max<0x121>(x);
}

// Elements [v N, v N + N) of a row of `dim` elements at `row`, N = Lane<DT>::N;
// those past the row's end are zero and are not touched.  WHOLE: dim is a
// multiple of N (the loads of single elements cost registers even where none runs).
template <int DT, bool WHOLE = false>
__device__ __forceinline__ u32x4 load_cut(const void* row, uint32_t v, uint32_t dim) {
  constexpr uint32_t N = Lane<DT>::N;
  const uint32_t e = v * N;
  if (e + N <= dim) return load16_any(row, v);
  u32x4 r = {0, 0, 0, 0};
  if (!WHOLE && e < dim) {
    const typename Vec<DT>::T* p = static_cast<const typename Vec<DT>::T*>(row);
#pragma unroll
    for (uint32_t k = 0; k < N; ++k) {
      if (e + k < dim) {
        if constexpr (DT == ZERO_F32) r[k] = __float_as_uint(p[e + k]);
        else r[k >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, p[e + k]) << (16 * (k & 1));
      }
    }
  }
  return r;
}

template <int DT, bool NT = false, bool WHOLE = false>
__device__ __forceinline__ void store_cut(void* row, uint32_t v, uint32_t dim, const float (&x)[Lane<DT>::N]) {
  constexpr uint32_t N = Lane<DT>::N;
  const uint32_t e = v * N;
  if (e + N <= dim) store16_any<DT, NT>(row, v, x);
  else if (!WHOLE)
#pragma unroll
    for (uint32_t k = 0; k < N; ++k)
      if (e + k < dim) Vec<DT>::store1(row, e + k, x[k]);
}

inline uint32_t dtype_bytes(int dtype) { return dtype == ZERO_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype == ZERO_F16 || dtype == ZERO_BF16 || dtype == ZERO_F32; }
inline bool multiple_of(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Calls fn with the storage type as a compile-time constant.
template <typename F>
void with_dtype(int dtype, F fn) {
  if (dtype == ZERO_F16) fn(std::integral_constant<int, ZERO_F16>{});
  else if (dtype == ZERO_BF16) fn(std::integral_constant<int, ZERO_BF16>{});
  else fn(std::integral_constant<int, ZERO_F32>{});
}

}  // namespace zs
