// Element access of the 8-bit step and the losses: eight elements at a time
// in fp32 registers, whatever their storage.  Conversions to 16 bits are the
// hardware's round-to-nearest-even of one fp32 value (NaN stays NaN).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"

namespace zs {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// One storage type: `Raw` is eight elements as loaded, kPer of them to 16 bytes.
template <int DT>
struct Vec;

template <>
struct Vec<ZERO_F16> {
  typedef _Float16 T;
  struct Raw {
    u32x4 q;
  };
  static __device__ __forceinline__ float get(const Raw& r, int k) {
    const uint32_t w = r.q[k >> 1];
    return (float)__builtin_bit_cast(f16x2, w)[k & 1];
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  }
  static __device__ __forceinline__ float load1(const void* p, uint64_t e) { return (float)static_cast<const T*>(p)[e]; }
  static __device__ __forceinline__ void store1(void* p, uint64_t e, float x) { static_cast<T*>(p)[e] = (T)x; }
};

template <>
struct Vec<ZERO_BF16> {
  typedef uint16_t T;
  struct Raw {
    u32x4 q;
  };
  static __device__ __forceinline__ float get(const Raw& r, int k) {
    const uint32_t w = r.q[k >> 1];
    return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
  }
  static __device__ __forceinline__ float load1(const void* p, uint64_t e) {
    return __uint_as_float((uint32_t)static_cast<const T*>(p)[e] << 16);
  }
  static __device__ __forceinline__ void store1(void* p, uint64_t e, float x) {
    static_cast<T*>(p)[e] = (uint16_t)pack(x, 0.0f);
  }
};

template <>
struct Vec<ZERO_F32> {
  typedef float T;
  struct Raw {
    f32x4 lo, hi;
  };
  static __device__ __forceinline__ float get(const Raw& r, int k) { return k < 4 ? r.lo[k] : r.hi[k - 4]; }
  static __device__ __forceinline__ float load1(const void* p, uint64_t e) { return static_cast<const T*>(p)[e]; }
  static __device__ __forceinline__ void store1(void* p, uint64_t e, float x) { static_cast<T*>(p)[e] = x; }
};

// Eight elements from index e, 16-byte aligned.  NT: the nontemporal hint
// (data touched once).
template <int DT, bool NT = false>
__device__ __forceinline__ typename Vec<DT>::Raw load8(const void* base, uint64_t e) {
  const typename Vec<DT>::T* p = static_cast<const typename Vec<DT>::T*>(base) + e;
  if constexpr (DT == ZERO_F32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(p);
    if constexpr (NT) return {__builtin_nontemporal_load(q), __builtin_nontemporal_load(q + 1)};
    else return {q[0], q[1]};
  } else {
    const u32x4* q = reinterpret_cast<const u32x4*>(p);
    if constexpr (NT) return {__builtin_nontemporal_load(q)};
    else return {*q};
  }
}

template <int DT, bool NT = false>
__device__ __forceinline__ void store8(void* base, uint64_t e, const float (&x)[8]) {
  typename Vec<DT>::T* p = static_cast<typename Vec<DT>::T*>(base) + e;
  if constexpr (DT == ZERO_F32) {
    f32x4* q = reinterpret_cast<f32x4*>(p);
    const f32x4 lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
    if constexpr (NT) {
      __builtin_nontemporal_store(lo, q);
      __builtin_nontemporal_store(hi, q + 1);
    } else {
      q[0] = lo;
      q[1] = hi;
    }
  } else {
    u32x4* q = reinterpret_cast<u32x4*>(p);
    const u32x4 v = {Vec<DT>::pack(x[0], x[1]), Vec<DT>::pack(x[2], x[3]), Vec<DT>::pack(x[4], x[5]),
                     Vec<DT>::pack(x[6], x[7])};
    if constexpr (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
  }
}

// Four elements from index e, a multiple of 4.
template <int DT>
__device__ __forceinline__ void store4(void* base, uint64_t e, float a, float b, float c, float d) {
  typename Vec<DT>::T* p = static_cast<typename Vec<DT>::T*>(base) + e;
  if constexpr (DT == ZERO_F32) *reinterpret_cast<f32x4*>(p) = f32x4{a, b, c, d};
  else *reinterpret_cast<u32x2*>(p) = u32x2{Vec<DT>::pack(a, b), Vec<DT>::pack(c, d)};
}

// Rows of logits: 16 bytes to a lane, N elements, at any address that suits
// the elements (rows start where an odd vocabulary puts them; gfx950 loads and
// stores 16 bytes at any such address in one instruction).  A row is addressed
// by a base that is the same in every thread and a 32-bit vector number, so
// that one register holds a thread's place in all of them.  fp32 lanes take
// four elements and not two halves of eight: a wavefront's instruction then
// covers 1 KB without gaps.
constexpr uint32_t kMaxRowVecs = 1u << 26;  // a row's byte offsets fit 32 bits

typedef u32x4 __attribute__((aligned(2))) u32x4_any;

template <int DT>
struct Lane {
  static constexpr int N = DT == ZERO_F32 ? 4 : 8;
  static __device__ __forceinline__ float get(const u32x4& r, int k) {
    if constexpr (DT == ZERO_F32) return __uint_as_float(r[k]);
    else return Vec<DT>::get(typename Vec<DT>::Raw{r}, k);
  }
};

template <bool NT = false>
__device__ __forceinline__ u32x4 load16_any(const void* base, uint32_t v) {
  const u32x4_any* q = reinterpret_cast<const u32x4_any*>(static_cast<const char*>(base) + v * 16u);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  else return *q;
}

template <int DT, bool NT = false>
__device__ __forceinline__ void store16_any(void* base, uint32_t v, const float (&x)[Lane<DT>::N]) {
  u32x4_any* q = reinterpret_cast<u32x4_any*>(static_cast<char*>(base) + v * 16u);
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == ZERO_F32) w[i] = __float_as_uint(x[i]);
    else w[i] = Vec<DT>::pack(x[2 * i], x[2 * i + 1]);
  }
  if constexpr (NT) __builtin_nontemporal_store((u32x4_any)w, q);
  else *q = w;
}

// Eight e4m3 codes (8 bytes) to and from fp32, by the hardware's conversions:
// decoding is exact, encoding rounds to nearest even.  Values beyond 464 do
// not occur (the callers scale by the block's largest magnitude).
__device__ __forceinline__ void decode8(const u32x2 c, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], true);
    x[4 * h] = a[0];
    x[4 * h + 1] = a[1];
    x[4 * h + 2] = b[0];
    x[4 * h + 3] = b[1];
  }
}

__device__ __forceinline__ u32x2 encode8(const float (&x)[8]) {
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h], x[4 * h + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2], x[4 * h + 3], w, true);
    c[h] = (uint32_t)w;
  }
  return c;
}

}  // namespace zs
